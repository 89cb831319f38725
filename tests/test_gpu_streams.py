"""Streams, CUDA graphs and concurrent host threads.

Every call is asynchronous on the stream it is given; the prefetch path of the
ring adds a pooled side stream joined back with events.  These tests check that
  * a ring captured in a CUDA graph (side stream included) and replayed on new
    inputs gives exactly the eager results, in every ring mode and with the work
    plan in the workspace;
  * the same call on a non-default stream gives exactly the default stream's
    results;
  * two host threads running prefetched rings at once on their own streams each
    get exactly their single-threaded results (no shared side stream or event).
"""
import subprocess
import sys
import threading

import pytest
import torch

import cp_synth as SY
from conftest import ROOT
from context_causal_attention_gb300 import ops as F

pytestmark = pytest.mark.gpu

CASES = {
    "s4k": SY.WORKLOADS["s4k"],
    # the plan in the workspace: its two pre-pass kernels are captured too
    "global_plan": SY.Workload("st_plan", B=1, S=32 * 4224, N=2, Nkv=1, D=64, C=32),
}


def _shards(w, dev, seed):
    g = torch.Generator().manual_seed(seed)
    mk = lambda n: F.cp_zigzag_shard(torch.randn(w.B, w.S, n, w.D, generator=g).to(torch.bfloat16).to(dev), w.C)  # noqa: E731
    return mk(w.N), mk(w.Nkv), mk(w.Nkv)


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("prefetch,fused", [(1, False), (1, True), (0, False)])
def test_ring_in_a_cuda_graph_matches_eager(cuda_dev, name, prefetch, fused):
    w = CASES[name]
    qs, ks, vs = _shards(w, cuda_dev, 1)
    pos = F.cp_zigzag_positions(w.S, w.C, device=cuda_dev)
    ws = torch.empty(max(256, F.cp_ring_workspace_size(w.B, w.S, w.N, w.Nkv, w.D, w.C, prefetch, F.CP_F32, fused)),
                     dtype=torch.uint8, device=cuda_dev)
    o = torch.empty((w.C, w.B, w.S // w.C, w.N, w.D), dtype=torch.float32, device=cuda_dev)
    lse = torch.empty((w.C, w.B, w.N, w.S // w.C), dtype=torch.float32, device=cuda_dev)

    def ring():
        F.cp_ring_attention_fwd(qs, ks, vs, pos, prefetch=prefetch, fused_merge=fused, workspace=ws, o=o, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ring()  # warm-up outside the capture (lazy set-up of the side stream and kernel attributes)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ring()
    for seed in (2, 3):
        q2, k2, v2 = _shards(w, cuda_dev, seed)
        qs.copy_(q2)
        ks.copy_(k2)
        vs.copy_(v2)
        graph.replay()
        torch.cuda.synchronize()
        o_g, l_g = o.clone(), lse.clone()
        o_e, l_e = F.cp_ring_attention_fwd(qs, ks, vs, pos, prefetch=prefetch, fused_merge=fused)
        torch.cuda.synchronize()
        assert torch.equal(o_g, o_e) and torch.equal(l_g, l_e), seed
    assert F.cp_device_status() == 0


def test_non_default_stream_matches_default(cuda_dev):
    w = SY.WORKLOADS["s4k"]
    qs, ks, vs = _shards(w, cuda_dev, 4)
    pos = F.cp_zigzag_positions(w.S, w.C, device=cuda_dev)
    o_d, l_d = F.cp_ring_attention_fwd(qs, ks, vs, pos, prefetch=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o_s, l_s = F.cp_ring_attention_fwd(qs, ks, vs, pos, prefetch=1, stream=s)
        o_u = F.cp_zigzag_unshard(o_s, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(o_s, o_d) and torch.equal(l_s, l_d)
    assert torch.equal(o_u, F.cp_zigzag_unshard(o_d))


def test_two_host_threads_run_rings_at_once(cuda_dev):
    w = SY.WORKLOADS["s4k"]
    pos = F.cp_zigzag_positions(w.S, w.C, device=cuda_dev)
    inputs = [_shards(w, cuda_dev, 10 + i) for i in range(2)]
    ref = [F.cp_ring_attention_fwd(*x, pos, prefetch=1) for x in inputs]
    torch.cuda.synchronize()
    out, errs = [None, None], []

    def worker(i):
        try:
            torch.cuda.set_device(cuda_dev)
            s = torch.cuda.Stream()
            res = []
            with torch.cuda.stream(s):
                for _ in range(4):
                    res.append(F.cp_ring_attention_fwd(*inputs[i], pos, prefetch=1, stream=s))
            s.synchronize()
            out[i] = res
        except Exception as e:  # reported below
            errs.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert not errs, errs
    for i in range(2):
        assert out[i] is not None
        for o, l in out[i]:
            assert torch.equal(o, ref[i][0]) and torch.equal(l, ref[i][1])
    assert F.cp_device_status() == 0


def _side_calls(dev):
    """Calls that allocate outputs and scratch: name -> (call(stream), bytes of its scratch)."""
    g = torch.Generator().manual_seed(9)
    mk = lambda *shape: torch.randn(*shape, generator=g).to(torch.bfloat16).to(dev)  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    q, k, v = mk(1, 512, 4, 64), mk(1, 512, 2, 64), mk(1, 512, 2, 64)
    pos = torch.arange(512, dtype=torch.int32, device=dev)
    w = [torch.ones(64, device=dev) for _ in range(2)]
    rope = F.cp_rope_freqs(64, device=dev)
    kc, vc = mk(64, 16, 2, 64), mk(64, 16, 2, 64)
    table = torch.arange(64, dtype=torch.int32, device=dev).view(2, 32)
    cu, kv_len, new = i32(0, 20, 40), i32(400, 500), mk(40, 8, 64)
    pages = i32(*range(64))
    qs, ks, vs = (F.cp_zigzag_shard(t, 4) for t in (q, k, v))
    zz = F.cp_zigzag_positions(512, 4, device=dev)
    o, lse = F.cp_attn_partial(q, k, v, pos, pos)
    return {
        "shard": (lambda s: F.cp_zigzag_shard(q, 4, stream=s), 0),
        "rope": (lambda s: F.cp_rope_fwd(q, k, pos, rope, stream=s), 0),
        "norm_bwd": (lambda s: F.cp_qk_norm_rope_bwd(q, k, q, k, *w, pos, rope, stream=s),
                     F.cp_qk_norm_rope_bwd_workspace_size(1, 1, 512, 4, 2, 64)),
        "append": (lambda s: F.cp_cache_append(new[:, :2], new[:, 2:4], kc, vc, table, cu, kv_len, rope=rope, q=new,
                                               stream=s), 0),
        "prefix": (lambda s: F.cp_prefix_attn_fwd(new, kc, vc, pages, 1000, table, cu, kv_len, 20, stream=s),
                   F.cp_prefix_attn_workspace_size(40, 2, 20, 1000, 8, 2, 64, 16, 32)),
        "ring": (lambda s: F.cp_ring_attention_fwd(qs, ks, vs, zz, prefetch=1, stream=s),
                 F.cp_ring_workspace_size(1, 512, 4, 2, 64, 4, 1)),
        "bwd": (lambda s: F.cp_attn_bwd_partial(q, k, v, o, q, lse, pos, pos, stream=s), 256),
    }


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("name", ["shard", "rope", "norm_bwd", "append", "prefix", "ring", "bwd"])
def test_memory_of_a_call_on_another_stream(cuda_dev, name, keep):
    """stream= with nothing given to write into.  The other stream is held back: what the
    current one allocates after the call (the sizes of its outputs, dropped or not, and of its
    scratch) is not what the call still uses.  Then the current stream is held back:
    what it has yet to read is not what the call writes into, though it has been given back."""
    call, scratch = _side_calls(cuda_dev)[name]
    many = lambda x: [t for t in (x if isinstance(x, (tuple, list)) else [x]) if t is not None]  # noqa: E731
    want = [t.clone() for t in many(call(None))]
    sizes = [t.numel() * t.element_size() for t in want] + [max(256, scratch)] * 2
    s = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)  # about 10 ms
        got = many(call(s))
        if not keep:
            got = None
        after = [torch.full((n,), 0xA5, dtype=torch.uint8, device=cuda_dev) for n in sizes]
        torch.cuda.synchronize()
        assert all((t == 0xA5).all() for t in after)
        assert not keep or all(torch.equal(a, b) for a, b in zip(got, want))
        del after, got
        torch.cuda.synchronize()
        before = [torch.full((n,), i + 1, dtype=torch.uint8, device=cuda_dev) for i, n in enumerate(sizes)]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        late = [t.clone() for t in before]
        del before
        got = many(call(s))
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        torch.cuda.synchronize()
        assert all((t == i + 1).all() for i, t in enumerate(late))


@pytest.mark.parametrize("name", ["rope", "norm_bwd", "append", "prefix", "ring"])
def test_stream_argument_inside_a_capture(cuda_dev, name):
    """A call on a side stream of a capture, its outputs and scratch allocated there: each replay
    gives the eager bits, over whatever the memory held."""
    call, _ = _side_calls(cuda_dev)[name]
    many = lambda x: [t for t in (x if isinstance(x, (tuple, list)) else [x]) if t is not None]  # noqa: E731
    want = [t.clone() for t in many(call(None))]
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        call(s)  # dropped: its memory goes to later work of s
        got = many(call(s))
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for t in got:
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


FIRST = """
import sys, torch
from context_causal_attention_gb300 import ops as F
dev, bf, i32 = "cuda", torch.bfloat16, torch.int32
q, k = (torch.randn(40, h, 64, device=dev).to(bf) for h in (8, 2))
pos = torch.arange(40, dtype=i32, device=dev)
w = [torch.ones(64, device=dev)] * 2
rope = F.cp_rope_freqs(64, device=dev)
kc, vc = (torch.randn(64, 16, 2, 64, device=dev).to(bf) for _ in range(2))
table, pages = torch.arange(64, dtype=i32, device=dev).view(2, 32), torch.arange(64, dtype=i32, device=dev)
cu, kv_len = torch.tensor([0, 20, 40], dtype=i32, device=dev), torch.tensor([300, 400], dtype=i32, device=dev)
calls = {
    "norm_bwd": lambda: F.cp_qk_norm_rope_bwd(q, k, q, k, *w, pos, rope),
    "append": lambda: (F.cp_cache_append(k, k, kc, vc, table, cu, kv_len, rope=rope, q=q),),
    "prefix": lambda: F.cp_prefix_attn_fwd(q, kc, vc, pages, 1000, table, cu, kv_len, 20),
}
call = calls[sys.argv[1]]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, call()))
print("same")
"""


@pytest.mark.parametrize("name", ["norm_bwd", "append", "prefix"])
def test_first_call_of_a_process_may_be_captured(cuda_dev, name):
    """What a kernel sets up at its first call is allowed inside a capture."""
    r = subprocess.run([sys.executable, "-c", FIRST, name], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
