"""Appending to the paged cache against the 64-bit forms of rows_ref.py: ragged
and empty sequences, pages that end inside a sequence, padding rows, long
offsets, wrong tables.  Tolerances as in test_gpu_rope.py (bf16 outputs)."""
import numpy as np
import pytest
import torch

import rows_ref as R
from context_causal_attention_gb300 import ops as F
from test_gpu_rope import DT, f64, rand, rope_of, within

pytestmark = pytest.mark.gpu


class Batch:
    """Sequences with `new` new tokens of `length` in all, over pages in random order."""

    def __init__(self, g, new, length, page, spare=2):
        self.new, self.length, self.page = new, length, page
        counts = [-(-m // page) for m in length]
        self.total = sum(counts) + spare
        order = torch.randperm(self.total, generator=g).tolist()
        self.table = torch.full((len(new), max(counts + [1])), -7, dtype=torch.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
            at += c
        self.cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        self.kv_len = torch.tensor(length, dtype=torch.int32)

    def slots(self, b, first, last):
        return [int(self.table[b, i // self.page]) * self.page + i % self.page for i in range(first, last)]

    def new_slots(self):
        return sum((self.slots(b, m - n, m) for b, (n, m) in enumerate(zip(self.new, self.length))), [])

    def new_index(self):
        return np.concatenate([np.arange(m - n, m) for n, m in zip(self.new, self.length)] + [np.zeros(0, int)])


CASES = {
    # one token of one sequence; page edge at the token
    "one": dict(new=[1], length=[17], page=16, N=1, Nkv=1, D=64),
    # decode with a sequence that gets nothing, heads that do not fill a warp
    "decode": dict(new=[1, 0, 1, 1, 1], length=[1, 0, 64, 65, 300], page=64, N=15, Nkv=3, D=128),
    # ragged prompts, padding behind them
    "prompts": dict(new=[40, 1, 0, 129, 16], length=[40, 33, 5, 150, 16], page=32, N=4, Nkv=4, D=64, pad=5),
    # more sequences than one level of the search holds
    "many": dict(new=[1, 0, 2] * 400, length=[3, 1, 20] * 400, page=16, N=2, Nkv=1, D=64, pad=1),
    # only keys and values
    "no_q": dict(new=[100, 100], length=[100, 400], page=256, N=0, Nkv=2, D=128),
}


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("norm", [False, True])
def test_append(cuda_dev, name, dt, norm):
    c = dict(CASES[name])
    g = torch.Generator().manual_seed(len(name))
    b = Batch(g, c["new"], c["length"], c["page"])
    N, Nkv, D, rows, base = c["N"], c["Nkv"], c["D"], sum(c["new"]), 70001
    total = rows + c.get("pad", 0)
    order = "interleaved" if norm else "half"
    rope, th, amp = rope_of(D // 2, order, "by_parts")
    qkv = rand(g, (total, N + 2 * Nkv, D), dt, 2.0)
    q, k, v = qkv[:, :N], qkv[:, N:N + Nkv], qkv[:, N + Nkv:]
    wq, wk = [1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)]
    caches = [rand(g, (b.total, b.page, Nkv, D), "bf16") for _ in range(2)]
    kc, vc = [x.to(cuda_dev) for x in caches]
    d = qkv.to(cuda_dev)
    qo = torch.full((total, N, D), 7.0, dtype=torch.bfloat16, device=cuda_dev) if N else None
    got = F.cp_cache_append(d[:, N:N + Nkv], d[:, N + Nkv:], kc, vc, b.table.to(cuda_dev), b.cu.to(cuda_dev),
                            b.kv_len.to(cuda_dev), rope=rope, q=d[:, :N] if N else None, q_out=qo,
                            wq=wq.to(cuda_dev) if norm and N else None, wk=wk.to(cuda_dev) if norm else None, eps=1e-5,
                            pos_base=base)
    assert got is qo
    at, pos = b.new_slots(), b.new_index() + base

    def want(x, w):
        y = f64(x[:rows])
        y = R.norm(y, f64(w), 1e-5) if norm else y
        return R.turn(y, pos, th, amp, order), 24 * R.U32 * amp * R.pair_size(y, th, order)

    for cache, old, x, w in ((kc, caches[0], k, wk), (vc, caches[1], v, None)):
        flat, before = cache.view(-1, Nkv, D).cpu(), old.view(-1, Nkv, D)
        rest = np.setdiff1d(np.arange(len(flat)), at)
        assert torch.equal(flat[rest], before[rest]), "a slot that got no token changed"
        if w is None:
            assert torch.equal(flat[at], x[:rows].to(torch.bfloat16))
        else:
            within(flat[at], *(lambda y, s: (y, "bf16", s))(*want(x, w)), name + " keys")
    if N:
        y, s = want(q, wq)
        within(qo[:rows], y, "bf16", s, name + " queries")
        assert (qo[rows:] == 7).all()


def test_no_rotation_and_q_in_place(cuda_dev):
    g = torch.Generator().manual_seed(1)
    b = Batch(g, [3, 2], [3, 20], 16)
    q, k, v = (rand(g, (5, h, 64), "bf16").to(cuda_dev) for h in (4, 2, 2))
    kc, vc = (torch.zeros(b.total, 16, 2, 64, dtype=torch.bfloat16, device=cuda_dev) for _ in range(2))
    lists = [t.to(cuda_dev) for t in (b.table, b.cu, b.kv_len)]
    F.cp_cache_append(k, v, kc, vc, *lists)
    assert torch.equal(kc.view(-1, 2, 64)[b.new_slots()], k) and torch.equal(vc.view(-1, 2, 64)[b.new_slots()], v)
    rope, _, _ = rope_of(64, "half")
    want = F.cp_cache_append(k, v, kc, vc, *lists, rope=rope, q=q)
    keys = kc.clone()
    q2 = q.clone()
    F.cp_cache_append(k, v, kc, vc, *lists, rope=rope, q=q2, q_out=q2)
    assert torch.equal(q2, want) and torch.equal(kc, keys)
    # the same rows by cp_rope_fwd
    pos = torch.tensor(b.new_index(), dtype=torch.int32, device=cuda_dev)
    assert torch.equal(F.cp_rope_fwd(q, None, pos, rope)[0], want)


def test_slots_past_32_bits_of_offset(cuda_dev):
    """A cache of more than 2^32 elements: the last page is written, its
    neighbours and the places an overflow would reach are not."""
    pages, page, Nkv, D = 20500, 256, 8, 128  # 5.4e9 elements
    kc = torch.zeros(pages, page, Nkv, D, dtype=torch.bfloat16, device=cuda_dev)
    vc = torch.zeros_like(kc)
    k, v = (torch.ones(2, Nkv, D, dtype=torch.bfloat16, device=cuda_dev) * x for x in (3, 5))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    F.cp_cache_append(k, v, kc, vc, i32(pages - 1, 17000).view(1, 2), i32(0, 2), i32(257))
    torch.cuda.synchronize()
    assert (kc[pages - 1, 255] == 3).all() and (vc[pages - 1, 255] == 5).all()
    assert (kc[17000, 0] == 3).all() and (vc[17000, 0] == 5).all()
    assert int((kc.view(torch.int16).view(-1, Nkv * D)[:, 0] != 0).sum()) == 2
    assert int((vc.view(torch.int16).view(-1, Nkv * D)[:, 0] != 0).sum()) == 2


@pytest.mark.parametrize("what", ["page", "negative_page", "index", "long", "none_bad"])
def test_bad_lists_are_reported_and_write_nothing(cuda_dev, what):
    """A page number or an index out of range: those tokens are skipped, the others
    stored, and the status word says so."""
    g = torch.Generator().manual_seed(2)
    b = Batch(g, [2, 3], [20, 3], 16)
    table, kv_len = b.table.clone(), b.kv_len.clone()
    if what == "page":
        table[0, 1] = b.total
    elif what == "negative_page":
        table[0, 1] = -1
    elif what == "index":
        kv_len[0] = 1     # fewer tokens than new ones: the first has index -1
    elif what == "long":
        kv_len[0] = 16 * table.shape[1] + 2
    k, v = (rand(g, (5, 2, 64), "bf16").to(cuda_dev) for _ in range(2))
    kc, vc = (torch.zeros(b.total, 16, 2, 64, dtype=torch.bfloat16, device=cuda_dev) for _ in range(2))
    F.cp_cache_append(k, v, kc, vc, table.to(cuda_dev), b.cu.to(cuda_dev), kv_len.to(cuda_dev))
    assert F.cp_device_status() == (0 if what == "none_bad" else 11)
    assert F.cp_device_status() == 0
    flat = kc.view(-1, 2, 64)
    assert torch.equal(flat[b.slots(1, 0, 3)], k[2:])
    stored = int((flat != 0).flatten(1).any(1).sum())
    assert stored == {"none_bad": 5, "index": 4}.get(what, 3)


def test_append_in_a_graph_reads_new_lengths(cuda_dev):
    """A captured decode step: kv_len is advanced between replays and each replay
    writes the next slots, from new rows in the same buffers."""
    g = torch.Generator().manual_seed(3)
    rope, th, amp = rope_of(64, "half")
    b = Batch(g, [1, 1], [40, 24], 16)
    k, v, q = (torch.zeros(2, h, 64, dtype=torch.bfloat16, device=cuda_dev) for h in (2, 2, 4))
    kc, vc = (torch.zeros(b.total, 16, 2, 64, dtype=torch.bfloat16, device=cuda_dev) for _ in range(2))
    qo, kv_len = torch.empty_like(q), torch.tensor([29, 13], dtype=torch.int32, device=cuda_dev)
    table, cu = b.table.to(cuda_dev), b.cu.to(cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.cp_cache_append(k, v, kc, vc, table, cu, kv_len, rope=rope, q=q, q_out=qo, pos_base=100)
    want = {}
    for step in range(6):
        rows = [rand(g, (2, h, 64), "bf16") for h in (2, 2, 4)]
        for t, r in zip((k, v, q), rows):
            t.copy_(r)
        kv_len += 1
        graph.replay()
        idx = (kv_len.cpu() - 1).tolist()
        for s, i in enumerate(idx):
            want[b.slots(s, i, i + 1)[0]] = (rows[1][s], R.turn(f64(rows[0][s:s + 1]), [i + 100], th, amp, "half")[0])
    torch.cuda.synchronize()
    fk, fv = kc.view(-1, 2, 64).cpu(), vc.view(-1, 2, 64).cpu()
    assert sorted(want) == torch.nonzero((fv != 0).flatten(1).any(1)).flatten().tolist()
    for s, (rv, rk) in want.items():
        assert torch.equal(fv[s], rv)
        within(fk[s], rk, "bf16", 8 * R.U32 * 10, "keys")


LONG = {
    # new tokens (empty sequences among them, beginnings and the padding's inside units of several tokens), what
    # was there before, heads of q and of k, D, page, padding
    "units_of_2": ([700, 0, 1, 0, 999, 3, 0, 820], 5, 3, 2, 64, 16, 7),
    "units_of_10": ([4096, 1, 0, 4095, 33, 4000, 0, 0, 2, 4001, 4096, 3053], 90, 2, 1, 128, 32, 1),
    "units_of_10_keys_alone": ([4096, 1, 0, 4095, 33, 4000, 0, 0, 2, 4001, 4096, 3053], 0, 0, 3, 64, 128, 3),
    "units_of_32": ([30001, 0, 0, 31, 1, 49000, 97, 2000], 3, 1, 1, 64, 256, 19),
    # more units than all warps take at once
    "units_of_32_in_rounds": ([60001, 7, 0, 70000, 32, 31, 33, 30011], 0, 1, 1, 64, 64, 5),
}


@pytest.mark.parametrize("name", sorted(LONG))
@pytest.mark.parametrize("dt,order,norm", [("bf16", "half", True), ("fp32", "interleaved", False)])
def test_append_of_many_tokens(cuda_dev, name, dt, order, norm):
    """Prompts so long that a warp takes several tokens: every key, value and query against
    64 bits, the slots that got no token and the padding as they were."""
    new, before, N, Nkv, D, page, pad = LONG[name]
    g = torch.Generator().manual_seed(len(name))
    b = Batch(g, new, [n + (before if i % 3 else 0) for i, n in enumerate(new)], page)
    rows, base = sum(new), 1234567
    rope, th, amp = rope_of(D, order, "by_parts")
    x = rand(g, (rows + pad, N + 2 * Nkv, D), dt, 2.0)
    wq, wk = [1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)]
    d = x.to(cuda_dev)
    kc, vc = (torch.full((b.total, page, Nkv, D), 9.0, dtype=torch.bfloat16, device=cuda_dev) for _ in range(2))
    qo = torch.full((rows + pad, N, D), 7.0, dtype=torch.bfloat16, device=cuda_dev) if N else None
    w = dict(wq=wq.to(cuda_dev) if N else None, wk=wk.to(cuda_dev)) if norm else {}
    F.cp_cache_append(d[:, N:N + Nkv], d[:, N + Nkv:], kc, vc, b.table.to(cuda_dev), b.cu.to(cuda_dev),
                      b.kv_len.to(cuda_dev), rope=rope, q=d[:, :N] if N else None, q_out=qo, eps=1e-5, pos_base=base, **w)
    assert F.cp_device_status() == 0
    at, pos = np.array(b.new_slots()), b.new_index() + base
    rest = np.ones(b.total * page, bool)
    rest[at] = False
    keys, values = (c.view(-1, Nkv, D).cpu() for c in (kc, vc))
    assert (keys[rest] == 9).all() and (values[rest] == 9).all()
    assert torch.equal(values[at], x[:rows, N + Nkv:].to(torch.bfloat16))

    def check(got, cut, w, what):
        y = f64(x[:rows, cut])
        y = R.norm(y, f64(w), 1e-5) if norm else y
        within(got, R.turn(y, pos, th, amp, order), "bf16", 24 * R.U32 * amp * R.pair_size(y, th, order), what)

    check(keys[at], slice(N, N + Nkv), wk, "keys")
    if N:
        check(qo[:rows], slice(0, N), wq, "queries")
        assert (qo[rows:] == 7).all()
