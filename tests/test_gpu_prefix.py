"""Attention over a shared prefix and paged sequences, against the 64-bit form of
rows_ref.py.

Tolerance.  Scores: products of bf16 values are exact in fp32, and a sum of D of
them is off by at most D u sum|q k| (u = 2^-24); with unit-normal values and scale
1/sqrt(D) that is under 2^-14 in the score for D = 128, so every weight, and lse,
is right to 2^-13 with the exponential's own 2^-22 and the sums' length / 2^24
(lengths here stay under 2^10 tiles a thread).  Each weight is then rounded to
bf16: off by at most 2^-8 (half a step) of itself, so o is off by at most (2^-8 + 2^-12)
sum p|v| / sum p, and by half a step of its own type."""
import math

import numpy as np
import pytest
import torch

import rows_ref as R
from context_causal_attention_gb300 import ops as F
from test_gpu_cache import Batch
from test_gpu_rope import f64, rand, rope_of, within

pytestmark = pytest.mark.gpu


class Call:
    """A batch with caches, prefix and queries, on the device, and its 64-bit result."""

    def __init__(self, seed, new, length, prefix, N, Nkv, D, page, pad=0, garbage=None, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        # the prefix is one more list of the batch's pages
        b = Batch(g, list(new) + [0], list(length) + [prefix], page)
        self.b, self.N, self.Nkv, self.D, self.prefix, self.new, self.length = b, N, Nkv, D, prefix, new, length
        self.rows, self.R = sum(new), sum(new) + pad
        self.k, self.v = (rand(g, (b.total, page, Nkv, D), "bf16") for _ in range(2))
        self.q = rand(g, (self.R, N, D), "bf16", gain)
        used = np.zeros(b.total * page, bool)
        for s, m in enumerate(b.length):
            used[b.slots(s, 0, m)] = True
        if garbage is not None:
            free = torch.tensor(~used).view(b.total, page)
            self.k[free], self.v[free] = garbage, garbage
            self.q[self.rows:] = garbage
        self.table = b.table[:-1].contiguous()
        self.pages = b.table[-1, :max(1, -(-prefix // page))].contiguous()
        self.cu, self.kv_len = b.cu[:-1].contiguous(), b.kv_len[:-1].contiguous()

    def run(self, dev, **kw):
        self.dev = [t.to(dev) for t in (self.q, self.k, self.v, self.pages, self.table, self.cu, self.kv_len)]
        q, k, v, pages, table, cu, kv_len = self.dev
        return F.cp_prefix_attn_fwd(q, k, v, pages, self.prefix, table, cu, kv_len,
                                    max(1, max(self.new)), **kw)

    def want(self):
        b, n, P = self.b, len(self.new), self.prefix
        k, v = f64(self.k).reshape(-1, self.Nkv, self.D), f64(self.v).reshape(-1, self.Nkv, self.D)
        o, a = (np.zeros((self.rows, self.N, self.D)) for _ in range(2))
        lse, r = np.zeros((self.N, self.rows)), 0
        for s in range(n):
            at = b.slots(n, 0, P) + b.slots(s, 0, self.length[s])
            m, L = self.new[s], self.length[s]
            seen = np.ones((m, P + L), bool)
            seen[:, P:] = np.arange(L) <= np.arange(L - m, L)[:, None]
            o[r:r + m], lse[:, r:r + m], a[r:r + m] = R.attention(f64(self.q[r:r + m]), k[at], v[at], seen,
                                                                 1 / math.sqrt(self.D))
            r += m
        return o, lse, a

    def check(self, o, lse, dt="bf16", what="", gain=1.0):
        wo, wl, a = self.want()
        n = self.rows
        within(o[:n], wo, dt, (2.0 ** -8 + 2.0 ** -12 * gain) * a, what + " o")
        got = f64(lse)[:, :n]
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(got), empty)
        assert (f64(o[:n]).transpose(1, 0, 2)[empty] == 0).all()
        assert np.abs(got[~empty] - wl[~empty]).max(initial=0) <= 2.0 ** -12 * gain, what + " lse"


# new tokens, own lengths, prefix, N, Nkv, D, page, padding
CASES = {
    "one_key": ([1], [1], 0, 1, 1, 64, 16, 0),
    "one_and_prefix": ([1], [1], 1, 4, 1, 128, 16, 0),
    "tile_edges": ([1, 1, 1, 1], [63, 64, 65, 128], 64, 8, 2, 64, 64, 0),
    "page_edges": ([1, 1, 1], [15, 16, 17], 33, 8, 8, 128, 16, 0),
    "draft": ([5, 1, 3, 5], [5, 700, 3, 130], 1000, 12, 4, 64, 32, 3),
    "odd_groups": ([2, 1, 4], [2, 90, 400], 257, 21, 3, 128, 128, 0),
    "one_kv_head": ([3, 3], [3, 77], 500, 40, 1, 64, 256, 0),
    "no_prefix": ([1, 7, 0, 2], [1000, 7, 12, 33], 0, 16, 4, 128, 16, 1),
    "empty_sequences": ([0, 1, 0, 0], [0, 9, 300, 0], 70, 4, 2, 64, 16, 2),
    "prompts": ([150, 1, 64, 33], [150, 40, 264, 33], 300, 8, 2, 128, 64, 5),
    "many": ([1] * 300, list(range(1, 301)), 200, 4, 2, 64, 16, 0),
    "half_tile": ([5, 5], [5, 9], 100, 8, 2, 64, 16, 0),
    "half_tile_long": ([6, 1], [70, 2900], 5000, 24, 3, 128, 64, 0),
    "half_tiles_mixed": ([70, 20, 1, 90], [900, 20, 333, 1200], 400, 16, 4, 64, 32, 3),
    # more pieces than blocks: every block goes from piece to piece, of one, of an odd
    # and of an even number of key tiles, of up to 128 and of more rows
    "short_prompts": ([20] * 400, [20 + 7 * i % 109 for i in range(400)], 100, 4, 1, 64, 16, 0),
    "mixed_prompts": ([1 + 13 * i % 60 for i in range(300)], [61 + 37 * i % 700 for i in range(300)], 130, 4, 1, 128,
                      64, 2),
    "mixed_prompts_small_pages": ([1 + 29 * i % 90 for i in range(200)], [91 + 53 * i % 500 for i in range(200)], 0, 6,
                                  2, 64, 16, 0),
    "most_sequences": ([1] * 4096, [1 + i % 40 for i in range(4096)], 30, 2, 1, 64, 16, 0),
    "most_sequences_wide": ([i % 4 for i in range(4096)], [3 + i % 40 for i in range(4096)], 0, 8, 1, 64, 32, 0),
    "long": ([1, 2], [3000, 9000], 20000, 8, 2, 128, 64, 0),
    # a KV head for nearly every SM: one or two blocks work on a head's line, of both launches
    "heads_152": ([1] * 20, [1 + 9 * i for i in range(20)], 300, 152, 152, 64, 16, 0),
    "heads_76": ([1, 2] * 6, [2 + 9 * i for i in range(12)], 200, 152, 76, 128, 32, 1),
    "heads_157": ([1] * 18, [1 + 9 * i for i in range(18)], 130, 157, 157, 64, 64, 0),
}


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_against_64_bits(cuda_dev, name, dt):
    new, length, prefix, N, Nkv, D, page, pad = CASES[name]
    c = Call(len(name), new, length, prefix, N, Nkv, D, page, pad)
    T = {"bf16": torch.bfloat16, "fp32": torch.float32}[dt]
    o = torch.full((c.R, N, D), 7.0, dtype=T, device=cuda_dev)
    lse = torch.full((N, c.R), 7.0, device=cuda_dev)
    c.run(cuda_dev, o=o, lse=lse)
    c.check(o, lse, dt, name)
    assert (o[c.rows:] == 7).all() and (lse[:, c.rows:] == 7).all()


@pytest.mark.parametrize("garbage", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("name", ["draft", "page_edges", "prompts", "one_key"])
def test_what_unused_slots_hold_does_not_matter(cuda_dev, name, garbage):
    """Slots past a length (in a used page too), spare pages and padding queries hold
    NaN, infinities or the largest values: the same bits come out."""
    new, length, prefix, N, Nkv, D, page, pad = CASES[name]
    clean = Call(3, new, length, prefix, N, Nkv, D, page, pad)
    dirty = Call(3, new, length, prefix, N, Nkv, D, page, pad, garbage=garbage)
    n = clean.rows
    a, b = clean.run(cuda_dev), dirty.run(cuda_dev)
    assert torch.equal(a[0][:n], b[0][:n]) and torch.equal(a[1][:, :n], b[1][:, :n])
    clean.check(*a)


def test_rows_that_see_nothing(cuda_dev):
    """Fewer cached tokens than new ones: rows with a negative index see the prefix
    alone, and without one nothing (o = 0, lse = -inf)."""
    for prefix in (0, 40):
        c = Call(4, [6, 1], [6, 20], prefix, 4, 2, 64, 16)
        c.kv_len[0] = 2
        c.length = [2, 20]
        o, lse = c.run(cuda_dev)
        k, v = f64(c.k).reshape(-1, 2, 64), f64(c.v).reshape(-1, 2, 64)
        at = c.b.slots(2, 0, prefix) + c.b.slots(0, 0, 2)
        seen = np.ones((6, prefix + 2), bool)
        seen[:, prefix:] = np.arange(2) <= (np.arange(6) - 4)[:, None]
        wo, wl, a = R.attention(f64(c.q[:6]), k[at], v[at], seen, 0.125)
        within(o[:6], wo, "bf16", (2.0 ** -8 + 2.0 ** -12) * a, "few keys")
        none = np.isneginf(wl)
        assert none.sum() == (16 if prefix == 0 else 0)
        assert np.array_equal(np.isneginf(f64(lse)[:, :6]), none)
        assert np.abs(f64(lse)[:, :6][~none] - wl[~none]).max() <= 2.0 ** -12
    # no key at all anywhere
    c = Call(5, [1], [1], 0, 2, 1, 128, 16)
    c.kv_len[0] = 0
    o, lse = c.run(cuda_dev)
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["draft", "page_edges", "prompts", "half_tile_long", "short_prompts", "mixed_prompts",
                                  "heads_152", "no_prefix"])
def test_a_query_that_is_not_a_number_stays_alone(cuda_dev, name, value):
    """Every score of a query row of NaN (or of infinities of both signs) is NaN: so are its o and
    lse, and no other row's.  The rows that share its warp may take the sums l of their
    weights in another order: two sums of positive values, each off by at most 34
    additions of u = 2^-24 a tile, so l moves by 68 u < 2^-17 of itself.  o = sum_i f_i o_i / l over
    the pieces: the quotient moves by as much, and each of the products and sums
    rounds relative to its own size, which is at most sum p|v| / sum p, not |o| (pieces of
    opposite sign cancel): a few u of that.  Together under 2^-17 + 2^-21 of sum p|v| / sum p."""
    new, length, prefix, N, Nkv, D, page, pad = CASES[name]
    c = Call(13, new, length, prefix, N, Nkv, D, page, pad)
    n = c.rows
    good = [t.clone() for t in c.run(cuda_dev, o_dtype=F.CP_F32)]
    size = torch.from_numpy(c.want()[2]).to(cuda_dev)
    at = [(r, (7 * r) % N) for r in range(0, n, 11)]
    for r, h in at:
        c.q[r, h] = value
        c.q[r, h, ::2] *= -1
    o, lse = c.run(cuda_dev, o_dtype=F.CP_F32)
    sick = torch.zeros((n, N), dtype=torch.bool, device=cuda_dev)
    for r, h in at:
        sick[r, h] = True
    sick &= ~torch.isneginf(good[1][:, :n].T)  # a row that sees no key has no score
    assert sick.any()
    o, lse, wo, wl = o[:n], lse[:, :n].T, good[0][:n], good[1][:, :n].T
    assert torch.isnan(o[sick]).all() and torch.isnan(lse[sick]).all()
    assert ((o[~sick] - wo[~sick]).abs() <= (2.0 ** -17 + 2.0 ** -21) * size[~sick]).all()
    same = torch.isneginf(wl) & torch.isneginf(lse)
    assert ((lse - wl).abs() <= 2.0 ** -17)[~sick & ~same].all()


@pytest.mark.parametrize("gain", [30.0, 300.0])
def test_large_scores(cuda_dev, gain):
    """Scores in the hundreds and thousands, growing along the keys: the running
    maximum moves.  The score's error scales with the queries (the bound of the
    header times the gain), which the weights share."""
    c = Call(6, [2, 1], [500, 900], 1500, 8, 4, 64, 16, gain=gain)
    # keys grow along the sequence
    for s, m in enumerate(c.b.length):
        at = c.b.slots(s, 0, m)
        k = c.k.view(-1, 4, 64)
        k[at] = (k[at].float() * torch.linspace(0.01, 1, max(m, 1)).view(-1, 1, 1)).to(torch.bfloat16)
    o, lse = c.run(cuda_dev, o_dtype=F.CP_F32)
    c.check(o, lse, "fp32", "gain", gain)


def test_same_bits_twice_and_by_graph(cuda_dev):
    """The same call twice, on another stream, and as a captured graph whose lists
    and caches change between replays: each the bits of an eager call."""
    c = Call(7, [1, 3, 2], [200, 400, 61], 3000, 16, 4, 128, 16)
    a = c.run(cuda_dev)
    b = c.run(cuda_dev)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q, k, v, pages, table, cu, kv_len = c.dev
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        d = F.cp_prefix_attn_fwd(q, k, v, pages, 3000, table, cu, kv_len, 3)
    s.synchronize()
    assert torch.equal(a[0], d[0]) and torch.equal(a[1], d[1])
    o, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
    ws = torch.empty(F.cp_prefix_attn_workspace_size(6, 3, 3, 3000, 16, 4, 128, 16, table.shape[1]), dtype=torch.uint8,
                     device=cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.cp_prefix_attn_fwd(q, k, v, pages, 3000, table, cu, kv_len, 3, o=o, lse=lse, workspace=ws)
    for step in range(3):
        ws.random_(0, 256)
        kv_len.copy_(torch.tensor([200 - 50 * step, 400 - 133 * step, 61 - step], dtype=torch.int32))
        q.copy_(q.flip(0))
        graph.replay()
        want = F.cp_prefix_attn_fwd(q, k, v, pages, 3000, table, cu, kv_len, 3)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), step


@pytest.mark.parametrize("new,N,Nkv,D,page", [(6, 64, 8, 128, 64), (21, 40, 8, 128, 128), (6, 64, 8, 128, 16),
                                               (40, 16, 4, 64, 64)])
def test_repeated_calls_agree(cuda_dev, new, N, Nkv, D, page):
    """Many blocks, pieces and last tiles that are not full, over and over with other work
    between: the bits never change (a wait that passes too early shows as a
    call that differs now and then), and they are right."""
    g = torch.Generator().manual_seed(new * page)
    lens = [new + int(x) for x in torch.randint(0, 1300, (24,), generator=g)]
    c = Call(11, [1 + (new - 1) * (i % 3) // 2 for i in range(24)], lens, 777, N, Nkv, D, page)
    o, lse = c.run(cuda_dev)
    c.check(o, lse)
    junk = torch.empty(64 << 20, device=cuda_dev)
    q, k, v, pages, table, cu, kv_len = c.dev
    for i in range(40):
        if i % 2:
            junk.fill_(i)
        o2, lse2 = F.cp_prefix_attn_fwd(q, k, v, pages, 777, table, cu, kv_len, new)
        assert torch.equal(o, o2) and torch.equal(lse, lse2), i


@pytest.mark.parametrize("B,top,most,N,Nkv,D,page,prefix,hint", [
    (300, 200, 2, 24, 8, 64, 16, 0, 196), (300, 200, 2, 128, 8, 128, 128, 127, 2), (130, 190, 1, 85, 5, 128, 128, 3151, 1),
    (300, 30, 4, 21, 3, 128, 128, 2573, 4), (300, 190, 4, 16, 16, 128, 256, 1000, 400), (300, 20, 4, 9, 3, 64, 64, 0, 400)])
def test_many_short_sequences_on_wide_tiles(cuda_dev, B, top, most, N, Nkv, D, page, prefix, hint):
    """Blocks that go through many pieces of one key tile, where only one half has work,
    and a few of two: each piece has its own queries, over and over."""
    g = torch.Generator().manual_seed(B + N)
    new = torch.randint(0, most + 1, (B,), generator=g).tolist()
    c = Call(16, new, [n + int(x) for n, x in zip(new, torch.randint(0, top, (B,), generator=g))], prefix, N, Nkv, D, page, 3)
    c.run(cuda_dev)
    q, k, v, pages, table, cu, kv_len = c.dev
    first = F.cp_prefix_attn_fwd(q, k, v, pages, prefix, table, cu, kv_len, hint)
    c.check(*first)
    n = c.rows
    for _ in range(10):
        o, lse = F.cp_prefix_attn_fwd(q, k, v, pages, prefix, table, cu, kv_len, hint)
        assert torch.equal(o[:n], first[0][:n]) and torch.equal(lse[:, :n], first[1][:, :n])
    assert F.cp_device_status() == 0


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("new", [1, 40])
def test_pages_past_32_bits_of_offset(cuda_dev, page, new):
    """Caches of 2.7e9 elements each (byte offsets past 2^32), the pages in use at their
    end: the bits of the same call over small caches."""
    c = Call(14, [new, 1, new], [300 + new, 90, new], 700, 16, 4, 128, page)
    want = c.run(cuda_dev)
    q, k, v, pages, table, cu, kv_len = c.dev
    extra = int(2.7e9) // (page * 4 * 128)
    big = []
    for small in (k, v):
        t = torch.empty(extra + c.b.total, page, 4, 128, dtype=torch.bfloat16, device=cuda_dev)
        t[:2 * c.b.total] = float("nan")  # where a wrapped offset would lead
        t[extra:] = small
        big.append(t)
    ws = torch.empty(F.cp_prefix_attn_workspace_size(c.R, 3, new, 700, 16, 4, 128, page, table.shape[1]),
                     dtype=torch.uint8, device=cuda_dev)
    got = F.cp_prefix_attn_fwd(q, *big, pages + extra, 700, torch.where(table < 0, table, table + extra), cu, kv_len, new,
                               workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("name", ["draft", "prompts", "page_edges"])
def test_two_calls_at_once(cuda_dev, name):
    """Two streams, a workspace each, the same caches: both get their own calls' bits.  Then
    two graphs that share a workspace, replayed one after the other."""
    new, length, prefix, N, Nkv, D, page, pad = CASES[name]
    c = Call(15, new, length, prefix, N, Nkv, D, page, pad)
    c.run(cuda_dev)
    q, k, v, pages, table, cu, kv_len = c.dev
    qs = [q, q.flip(1).contiguous()]
    need = F.cp_prefix_attn_workspace_size(c.R, len(new), max(new), prefix, N, Nkv, D, page, table.shape[1])
    ws = [torch.empty(need, dtype=torch.uint8, device=cuda_dev) for _ in range(2)]
    outs = [(torch.zeros_like(q), torch.zeros(N, c.R, device=cuda_dev)) for _ in range(2)]

    def call(i, w):
        F.cp_prefix_attn_fwd(qs[i], k, v, pages, prefix, table, cu, kv_len, max(new), o=outs[i][0], lse=outs[i][1],
                             workspace=ws[w])

    want = []
    for i in range(2):
        call(i, 0)
        want.append([t.clone() for t in outs[i]])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                for t in outs[i]:
                    t.zero_()
                call(i, i)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            call(i, 0)
    for _ in range(10):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))


@pytest.mark.parametrize("hint", [1, 3, 40])
def test_any_hint_is_right(cuda_dev, hint):
    """max_new chooses the tiles only: one that is far off changes no result but by rounding."""
    c = Call(12, [40, 1, 0, 17], [300, 5, 9, 17], 200, 8, 2, 64, 32)
    c.run(cuda_dev)
    q, k, v, pages, table, cu, kv_len = c.dev
    c.check(*F.cp_prefix_attn_fwd(q, k, v, pages, 200, table, cu, kv_len, hint))


def test_outputs_and_workspace_stay_in_bounds(cuda_dev):
    c = Call(8, [3, 40, 1], [3, 300, 77], 130, 6, 2, 64, 16, pad=2)
    c.run(cuda_dev)
    q, k, v, pages, table, cu, kv_len = c.dev
    need = F.cp_prefix_attn_workspace_size(c.R, 3, 40, 130, 6, 2, 64, 16, table.shape[1])
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=cuda_dev)
    o = torch.full((c.R + 2, 6, 64), 7.0, device=cuda_dev)
    lse = torch.full((6 * c.R + 8,), 7.0, device=cuda_dev)
    F.cp_prefix_attn_fwd(q, k, v, pages, 130, table, cu, kv_len, 40, o=o[1:-1], lse=lse[4:-4].view(6, c.R),
                         workspace=ws[256:256 + need])
    torch.cuda.synchronize()
    assert (o[0] == 7).all() and (o[-1] == 7).all() and (lse[:4] == 7).all() and (lse[-4:] == 7).all()
    assert (ws[:256] == 0xA5).all() and (ws[256 + need:] == 0xA5).all()
    c.check(o[1:-1], lse[4:-4].view(6, c.R), "fp32")


@pytest.mark.parametrize("what", ["page", "prefix_page", "length", "negative_length", "counts", "counts_past_rows"])
def test_bad_lists_are_reported(cuda_dev, what):
    """Lists out of range are reported and not followed; a sequence that they do not
    touch keeps its result."""
    c = Call(9, [2, 3], [50, 40], 70, 4, 2, 64, 16)
    good = c.run(cuda_dev)
    torch.cuda.synchronize()
    if what == "page":
        c.table[0, 1] = c.b.total + 5
    elif what == "prefix_page":
        c.pages[2] = -1
    elif what == "length":
        c.kv_len[0] = 16 * c.table.shape[1] + 1
    elif what == "negative_length":
        c.kv_len[0] = -3
    elif what == "counts":
        c.cu[1] = -2
    else:
        c.cu[2] = 6
    o, lse = c.run(cuda_dev)
    assert F.cp_device_status() == 11
    assert F.cp_device_status() == 0
    if what in ("page", "length", "negative_length"):
        assert torch.equal(o[2:], good[0][2:]) and torch.equal(lse[:, 2:], good[1][:, 2:])


@pytest.mark.parametrize("first,N", [(-(2 ** 29 - 31), 8), (-(2 ** 31), 8), (-(2 ** 31) + 101, 32), (-1, 8)])
def test_counts_far_out_of_range_are_not_followed(cuda_dev, first, N):
    """Counts whose products with the heads of a KV head pass 32 bits: reported, and
    nothing outside the workspace is read into a result (NaN lies around it)."""
    c = Call(17, [100], [200], 70, N, 1, 64, 16)
    c.cu[0] = first
    need = F.cp_prefix_attn_workspace_size(100, 1, 100, 70, N, 1, 64, 16, c.table.shape[1])
    ws = torch.full((need + 8192,), 0xFF, dtype=torch.uint8, device=cuda_dev)
    for _ in range(2):  # the second time, over what the first left
        o, lse = c.run(cuda_dev, workspace=ws[4096:4096 + need])
        assert F.cp_device_status() == 11
        assert F.cp_device_status() == 0
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert (ws[:4096] == 0xFF).all() and (ws[4096 + need:] == 0xFF).all()


def test_append_then_attend_decodes_like_one_causal_attention(cuda_dev):
    """The operators together: a prefix and two prompts are appended (norm, rotation),
    then tokens one at a time; every step's attention equals the 64-bit causal
    attention of the whole sequence so far (inputs rounded where the cache rounds)."""
    g = torch.Generator().manual_seed(10)
    N, Nkv, D, page, P = 8, 2, 64, 16, 37
    prompt, steps, total = [21, 5], 4, 40
    b = Batch(g, [0, 0, 0], [prompt[0] + steps, prompt[1] + steps, P], page)
    rope, th, amp = rope_of(D, "half")
    kc, vc = (torch.full((b.total, page, Nkv, D), float("nan"), dtype=torch.bfloat16, device=cuda_dev) for _ in range(2))
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    table, pages = b.table[:2].to(cuda_dev), b.table[2:, :-(-P // page)].contiguous().to(cuda_dev)
    hist = [[], []]  # each sequence's (q, k, v) rows, as drawn

    def draw(n):
        return [rand(g, (n, h, D), "bf16") for h in (N, Nkv, Nkv)]

    def append(rows, tab, cu, lens, base):
        q, k, v = (t.to(cuda_dev) for t in rows)
        return F.cp_cache_append(k, v, kc, vc, tab, cu, lens, rope=rope, q=q, wq=wq.to(cuda_dev), wk=wk.to(cuda_dev),
                                 pos_base=base)

    shared = draw(P)
    append(shared, pages, i32(0, P), i32(P), 0)
    lens = [0, 0]
    for step in range(steps + 1):
        n = prompt if step == 0 else [1, 1]
        rows = [draw(x) for x in n]
        for h, r in zip(hist, rows):
            h.append(r)
        lens = [x + y for x, y in zip(lens, n)]
        cat = [torch.cat([r[i] for r in rows]) for i in range(3)]
        cu, kv_len = i32(0, n[0], n[0] + n[1]), i32(*lens)
        q = append(cat, table, cu, kv_len, P)
        o, lse = F.cp_prefix_attn_fwd(q, kc, vc, pages.flatten(), P, table, cu, kv_len, max(n))
        at = 0
        for s in range(2):
            every = [torch.cat([shared[i]] + [r[i] for r in hist[s]]) for i in range(3)]
            pos = np.arange(P + lens[s])
            qr, kr = (R.bf16(R.turn(R.norm(f64(every[i]), f64(w), 1e-6), pos, th, amp, "half"))
                      for i, w in ((0, wq), (1, wk)))
            seen = pos <= pos[-n[s]:, None]
            wo, wl, a = R.attention(qr[-n[s]:], kr, f64(every[2]), seen, 1 / math.sqrt(D))
            # a value next to a rounding border may go the other way in q or k: half a
            # step (2^-8) of single values, 2^-5 in a score of size sum|q k| scale < 8
            assert np.abs(f64(lse)[:, at:at + n[s]] - wl).max() <= 2.0 ** -5
            within(o[at:at + n[s]], wo, "bf16", (2.0 ** -8 + 2.0 ** -4) * a, "decode")
            at += n[s]


@pytest.mark.parametrize("N,Nkv", [(10, 5), (21, 7), (4, 1)])
def test_lists_that_change_between_calls(cuda_dev, N, Nkv):
    """A decode loop on the device: one small launch between two calls moves the lengths and
    the counts on in place, and every call sees the new ones on all SMs, also on those that
    the launches between left alone (the lanes of 5 or 7 KV heads do not use every SM)."""
    B, steps = 40, 24
    c = Call(23, [2] * B, [3 + 7 * b % 150 + steps for b in range(B)], 260, N, Nkv, 64, 16)
    c.run(cuda_dev)
    q, k, v, pages, table, cu, kv_len = c.dev
    full = kv_len.clone()
    lists = torch.cat([cu, kv_len])
    cu, kv_len = lists[:B + 1], lists[B + 1:]
    # kinds of rows move too: sequence 0 has between 1 and 3 of the new tokens, the next the rest of 4
    after = []
    for i in range(steps):
        want = torch.cat([c.cu.to(cuda_dev), full - i])
        want[1] = 1 + i % 3
        after.append(want)
    ws = torch.empty(F.cp_prefix_attn_workspace_size(2 * B, B, 3, 260, N, Nkv, 64, 16, table.shape[1]), dtype=torch.uint8,
                     device=cuda_dev)
    outs = [(torch.empty_like(q), torch.empty(N, 2 * B, device=cuda_dev)) for _ in range(steps)]
    for i in range(steps):
        lists.copy_(after[i])
        F.cp_prefix_attn_fwd(q, k, v, pages, 260, table, cu, kv_len, 3, o=outs[i][0], lse=outs[i][1], workspace=ws)
    torch.cuda.synchronize()
    for i in range(steps):
        new = after[i][:B + 1].clone(), after[i][B + 1:].clone()  # lists of their own, never changed
        o, lse = F.cp_prefix_attn_fwd(q, k, v, pages, 260, table, *new, 3)
        assert torch.equal(o, outs[i][0]) and torch.equal(lse, outs[i][1]), i
