"""The calls of speculative decoding on streams and in captures: the first call of a process inside a capture, a side
stream of a capture with the outputs' memory allocated there, and two streams at once, each with the bits of the plain
call."""
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from context_causal_attention_gb300 import ops as F

pytestmark = pytest.mark.gpu

NAMES = ["plan", "tree_plan", "append_at", "keep", "attn_items", "attn_clusters", "attn_line"]


def calls(seed=0, dev="cuda"):
    """name -> a call on inputs of its own that gives its results anew (stream: None or a stream); the keep's caches are
    made equal before it."""
    g = torch.Generator().manual_seed(seed)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    rows = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)  # noqa: E731
    N, Nkv, D, page, B, new = 8, 2, 64, 16, 3, 20
    R = B * new
    table = torch.randperm(192, generator=g).to(torch.int32).view(B, 64).to(dev)
    wide = torch.cat([table, torch.full((B, 9000), -1, dtype=torch.int32, device=dev)], 1)
    short = table[:, :40].contiguous()
    cu, kv_len = i32([0, 20, 40, 60]), i32([300, 620, 20 + seed])
    kc, vc = rows(192, page, Nkv, D), rows(192, page, Nkv, D)
    q, k = rows(R, N, D), rows(R, Nkv, D)
    parent = i32([max(-1, j // 2 - seed % 3) if j else -1 for _ in range(B) for j in range(new)])
    mask, pos = F.cp_tree_plan(parent, cu, kv_len, 1, 7)
    slots = torch.randperm(192 * page, generator=g)[:R].to(torch.int32).to(dev)
    rope = F.cp_rope_freqs(D, device=dev)
    free = torch.arange(192, dtype=torch.int32, device=dev)
    kept, n_kept = i32([[0, 2, 5, 9 + seed]] * B), i32([4, 3, -1])
    first = [kc.clone(), vc.clone()]
    shared = F.CpCaches([kc.clone(), vc.clone()])

    def plan(s):
        t, f = table.clone(), free.clone()
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        got = F.cp_cache_plan(i32_had, i32_keep, i32_new, t, f, i32_free, page, R, 3, stream=s)
        if s is not None:
            torch.cuda.current_stream().wait_stream(s)
        return (*got, t.clone())

    i32_had, i32_keep, i32_new, i32_free = i32([300, 50, 20]), i32([280, 50, 0]), i32([20, 19, 21]), i32([150, 0])

    def keep(s):
        for c, o in zip(shared.caches, first):
            c.copy_(o)
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        got = F.cp_cache_keep(shared, table, cu, kv_len, kept, n_kept, stream=s)
        if s is not None:
            torch.cuda.current_stream().wait_stream(s)
        return (got, *(c.clone() for c in shared.caches))

    attn = lambda t: lambda s: F.cp_tree_attn_fwd(q, kc, vc, mask, None, 0, t, cu, kv_len, new, stream=s)  # noqa: E731
    return {
        "plan": plan,
        "tree_plan": lambda s: F.cp_tree_plan(parent, cu, kv_len, 1, 7, stream=s),
        "append_at": lambda s: (F.cp_cache_append_at(k, k, *shared.caches, slots, pos, rope=rope, q=q, stream=s),),
        "keep": keep,
        "attn_items": attn(short),
        "attn_clusters": attn(table),
        "attn_line": attn(wide),
    }


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
def test_stream_argument_inside_a_capture(cuda_dev, name):
    call = calls(1)[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        call(s)  # dropped: its memory goes to later work of s
        got = call(s)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for t in got:
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_two_streams_at_once(cuda_dev, name):
    """Two sets of inputs, a stream each, ten calls in a row on both: nothing of one reaches the other."""
    both = [calls(seed)[name] for seed in (2, 5)]
    want = [[t.clone() for t in c(None)] for c in both]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, c in enumerate(both):
            with torch.cuda.stream(streams[i]):
                got[i].append(c(None))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(x, want[i]) for x in got[i])


FIRST = """
import sys, torch
sys.path.insert(0, "tests")
from test_gpu_tree_streams import calls, same
from context_causal_attention_gb300 import ops as F
plan = F.cp_tree_plan
# (masks and positions of any kind: the call of interest is the first)
F.cp_tree_plan = lambda parent, *a, **k: (parent.view(-1, 1).clone(), parent.clamp(min=0))
call = calls()[sys.argv[1]]
F.cp_tree_plan = plan
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call(None)
graph.replay()
torch.cuda.synchronize()
assert same(got, call(None))
assert F.cp_device_status() == 0
print("same")
"""


@pytest.mark.parametrize("name", NAMES)
def test_first_call_of_a_process_may_be_captured(cuda_dev, name):
    r = subprocess.run([sys.executable, "-c", FIRST, name], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
