"""Attention of drafted trees over the paged cache against the 64-bit form of rows_ref.py, and a run of speculative
steps through all calls.  Tolerances as derived in test_gpu_prefix.py: the kernels are the same but for which scores
are hidden."""
import math

import numpy as np
import pytest
import torch

import rows_ref as R
import tree_ref as T
from context_causal_attention_gb300 import ops as F
from test_gpu_prefix import Call
from test_gpu_rope import f64, rand, rope_of, within

pytestmark = pytest.mark.gpu


class TreeCall(Call):
    """A batch of drafted trees (and of prompts: sequences of more tokens than the mask's words hold)."""

    def __init__(self, seed, new, length, prefix, N, Nkv, D, page, words, kind="random", pad=0, garbage=None, gain=1.0):
        super().__init__(seed, new, length, prefix, N, Nkv, D, page, pad, garbage, gain)
        g = np.random.default_rng(seed)
        self.words, self.seen = words, []
        mask = g.integers(-2 ** 31, 2 ** 31, (self.R, words)).astype(np.int32)  # rows that go by none hold anything
        r = 0
        for n in new:
            if n > 32 * words:
                self.seen.append(np.tril(np.ones((n, n), bool)))
            else:
                if kind == "any":  # any set, not only ancestors: also none, and later tokens
                    seen = g.random((n, n)) < 0.4
                else:
                    seen = T.branches(T.random_parents(g, n, kind))[0]
                self.seen.append(seen)
                bits = g.random((n, 32 * words)) < 0.5  # behind the last token: not looked at
                bits[:, :n] = seen
                mask[r:r + n] = T.packed(bits, words)
            r += n
        self.mask = torch.from_numpy(mask)

    def run(self, dev, hint=None, form=None, **kw):
        if form in ("clusters", "line"):
            # a table for more tokens than a block an item takes, or than a cluster: the same call by other kernels
            wide = (140000 if form == "line" else 700) // self.b.page
            self.table = torch.cat([self.table, torch.full((len(self.new), wide), -3, dtype=torch.int32)], 1)
        self.dev = [t.to(dev) for t in (self.q, self.k, self.v, self.mask, self.pages, self.table, self.cu, self.kv_len)]
        return self.again(hint, **kw)

    def again(self, hint=None, **kw):
        q, k, v, mask, pages, table, cu, kv_len = self.dev
        return F.cp_tree_attn_fwd(q, k, v, mask, pages, self.prefix, table, cu, kv_len,
                                  max(1, max(self.new)) if hint is None else hint, **kw)

    def want(self):
        b, n, P = self.b, len(self.new), self.prefix
        k, v = f64(self.k).reshape(-1, self.Nkv, self.D), f64(self.v).reshape(-1, self.Nkv, self.D)
        o, a = (np.zeros((self.rows, self.N, self.D)) for _ in range(2))
        lse, r = np.zeros((self.N, self.rows)), 0
        for s in range(n):
            at = b.slots(n, 0, P) + b.slots(s, 0, self.length[s])
            m, L = self.new[s], self.length[s]
            seen = np.ones((m, P + L), bool)
            own = min(m, L)  # new tokens that are in the cache: the last ones
            seen[:, P + L - own:] = self.seen[s][:, m - own:]
            o[r:r + m], lse[:, r:r + m], a[r:r + m] = R.attention(f64(self.q[r:r + m]), k[at], v[at], seen,
                                                                 1 / math.sqrt(self.D))
            r += m
        return o, lse, a


# new tokens, own lengths, prefix, N, Nkv, D, page, words, padding
CASES = {
    "one": ([1], [1], 0, 1, 1, 64, 16, 1, 0),
    "token_and_prefix": ([1], [70], 33, 4, 1, 128, 16, 1, 0),
    "narrow": ([4, 1, 3, 0, 4], [4, 64, 130, 9, 67], 0, 4, 1, 64, 16, 1, 2),
    "narrow_edges": ([5, 5, 5, 5, 5], [63, 64, 65, 68, 70], 100, 9, 3, 128, 32, 1, 0),
    "narrow_wide_mask": ([16, 16, 2], [16, 80, 500], 40, 2, 2, 64, 64, 3, 1),
    "half_tile": ([27], [900], 0, 32, 8, 128, 16, 1, 0),
    "half_tile_edges": ([20, 20, 20, 20], [127, 128, 129, 148], 0, 12, 3, 64, 64, 1, 0),
    "half_tile_prefix": ([26, 7, 1, 13], [26, 700, 3, 1300], 1000, 16, 4, 128, 32, 1, 3),
    "wide": ([61, 40, 64, 9], [100, 2000, 64, 70], 300, 24, 3, 64, 64, 2, 0),
    "wide_many_words": ([300, 512, 31, 129], [400, 512, 90, 1000], 0, 4, 2, 128, 128, 16, 4),
    "with_prompts": ([20, 150, 1, 33, 70], [300, 150, 40, 300, 75], 200, 8, 2, 128, 64, 1, 5),
    "one_kv_head": ([9, 3], [9, 300], 77, 40, 1, 64, 256, 1, 0),
    "no_groups": ([13, 6], [200, 13], 500, 16, 16, 64, 16, 1, 0),
    "odd_groups": ([11, 2, 30], [90, 2, 400], 257, 21, 3, 128, 128, 1, 0),
    # more items than find room at once, the longest first, and fewer
    "blocks": ([9 + i % 20 for i in range(30)], [9 + i % 20 + 37 * i % 300 for i in range(30)], 0, 32, 8, 128, 16, 1, 1),
    "blocks_few": ([5 + 7 * i % 60 for i in range(22)], [70 + 91 * i % 900 for i in range(22)], 0, 16, 4, 64, 32, 2, 0),
    "blocks_equal": ([9] * 40 + [1, 0] * 20, [300, 9] * 20 + [300, 0] * 20, 70, 32, 8, 64, 16, 1, 2),
    "many": ([1 + i % 6 for i in range(200)], [10 + 7 * i % 300 for i in range(200)], 130, 8, 2, 64, 16, 1, 0),
    "many_wide": ([5 + 13 * i % 60 for i in range(150)], [70 + 37 * i % 700 for i in range(150)], 0, 8, 1, 128, 64, 2, 0),
    "most_sequences": ([1 + i % 2 for i in range(4096)], [2 + i % 40 for i in range(4096)], 30, 2, 1, 64, 16, 1, 0),
}


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("kind", ["random", "any", "chain"])
@pytest.mark.parametrize("form", ["as_chosen", "clusters", "line"])
def test_against_64_bits(cuda_dev, name, kind, form):
    new, length, prefix, N, Nkv, D, page, words, pad = CASES[name]
    c = TreeCall(len(name), new, length, prefix, N, Nkv, D, page, words, kind, pad)
    dt = "fp32" if kind == "any" else "bf16"
    T_ = {"bf16": torch.bfloat16, "fp32": torch.float32}[dt]
    o = torch.full((c.R, N, D), 7.0, dtype=T_, device=cuda_dev)
    lse = torch.full((N, c.R), 7.0, device=cuda_dev)
    c.run(cuda_dev, form=form, o=o, lse=lse)
    c.check(o, lse, dt, name)
    assert (o[c.rows:] == 7).all() and (lse[:, c.rows:] == 7).all()


@pytest.mark.parametrize("name", ["narrow", "narrow_edges", "half_tile_prefix", "wide", "with_prompts", "many"])
def test_a_chain_is_the_prefix_attention(cuda_dev, name):
    """Trees that are chains: both calls give what 64 bits give."""
    new, length, prefix, N, Nkv, D, page, words, pad = CASES[name]
    c = TreeCall(5, new, length, prefix, N, Nkv, D, page, words, "chain", pad)
    o, lse = c.run(cuda_dev)
    q, k, v, mask, pages, table, cu, kv_len = c.dev
    o2, lse2 = F.cp_prefix_attn_fwd(q, k, v, pages, prefix, table, cu, kv_len, max(new))
    c.check(o, lse)
    c.check(o2, lse2)


@pytest.mark.parametrize("garbage", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("name", ["narrow", "half_tile_prefix", "wide", "with_prompts", "one"])
@pytest.mark.parametrize("form", ["as_chosen", "clusters", "line"])
def test_what_unused_slots_hold_does_not_matter(cuda_dev, name, garbage, form):
    new, length, prefix, N, Nkv, D, page, words, pad = CASES[name]
    clean = TreeCall(3, new, length, prefix, N, Nkv, D, page, words, "random", pad)
    dirty = TreeCall(3, new, length, prefix, N, Nkv, D, page, words, "random", pad, garbage=garbage)
    n = clean.rows
    a, b = clean.run(cuda_dev, form=form), dirty.run(cuda_dev, form=form)
    assert torch.equal(a[0][:n], b[0][:n]) and torch.equal(a[1][:, :n], b[1][:, :n])


@pytest.mark.parametrize("form", ["as_chosen", "clusters", "line"])
@pytest.mark.parametrize("name", ["narrow", "half_tile_prefix", "wide"])
def test_keys_that_a_row_does_not_see_are_hidden_whatever_they_hold(cuda_dev, name, form):
    """NaN, infinities and the lowest value in drafted K rows: rows that do not see them keep their values (to the
    tolerance that test_gpu_prefix.py derives for rows beside a row of NaN)."""
    new, length, prefix, N, Nkv, D, page, words, pad = CASES[name]
    c = TreeCall(8, new, length, prefix, N, Nkv, D, page, words, "star", pad)
    good = [t.clone() for t in c.run(cuda_dev, form=form, o_dtype=F.CP_F32)]
    size = torch.from_numpy(c.want()[2]).to(cuda_dev)
    keep = torch.ones(c.rows, dtype=torch.bool)
    r = 0
    for s, n in enumerate(new):
        for j, bad in zip(range(1, n, 3), [float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min] * 99):
            slot = c.b.slots(s, length[s] - n + j, length[s] - n + j + 1)[0]
            c.k.view(-1, Nkv, D)[slot] = bad
            keep[r + j] = False
        r += n
    o, lse = c.run(cuda_dev, o_dtype=F.CP_F32)
    n = c.rows
    keep = keep.to(cuda_dev)
    assert ((o[:n] - good[0][:n]).abs()[keep] <= (2.0 ** -17 + 2.0 ** -21) * size[keep]).all()
    assert ((lse[:, :n] - good[1][:, :n]).abs()[:, keep] <= 2.0 ** -17).all()


def test_rows_that_see_nothing(cuda_dev):
    """No cached key, no prefix, no bit: o = 0 and lse = -inf; other rows of the tile have theirs.  Fewer cached
    tokens than new ones: those at negative indexes are not there."""
    for D, N, Nkv in ((64, 4, 2), (128, 24, 1)):
        c = TreeCall(4, [6, 3], [6, 20], 0, N, Nkv, D, 16, 1, "any")
        for j in (0, 2, 5):
            c.seen[0][j] = False
        c.seen[0][1, 3] = True
        bits = np.concatenate(c.seen[:1])
        c.mask[:6] = torch.from_numpy(T.packed(bits, 1))
        o, lse = c.run(cuda_dev)
        c.check(o, lse)
        for j in (0, 2, 5):
            assert (o[j] == 0).all() and torch.isneginf(lse[:, j]).all()
        c.kv_len[0], c.length = 4, [4, 20]
        c.check(*c.run(cuda_dev))
        c.kv_len[0], c.length = 0, [0, 20]
        o, lse = c.run(cuda_dev)
        c.check(o, lse)
        assert (o[:6] == 0).all()


@pytest.mark.parametrize("form", ["as_chosen", "clusters", "line"])
@pytest.mark.parametrize("N,n", [(2, 5), (16, 30), (32, 60)])
def test_a_row_that_sees_one_key_gives_its_value(cuda_dev, N, n, form):
    """One weight, whatever its score: o is that key's value to the bit."""
    c = TreeCall(18, [n, 3], [n, 3], 0, N, 2, 64, 16, 2, "roots", gain=40.0)
    o, lse = c.run(cuda_dev, form=form)
    c.check(o, lse, gain=40.0)
    at = c.b.slots(0, 0, n) + c.b.slots(1, 0, 3)
    v = c.v.view(-1, 2, 64)[at].repeat_interleave(N // 2, 1)
    assert torch.equal(o.cpu(), v)


@pytest.mark.parametrize("form", ["as_chosen", "clusters", "line"])
@pytest.mark.parametrize("gain", [1.0, 40.0, 3000.0])
@pytest.mark.parametrize("N,n,D", [(2, 5, 64), (16, 30, 64), (32, 60, 64), (8, 25, 128)])
def test_a_row_that_sees_one_key_gives_its_value_in_32_bits(cuda_dev, N, n, D, gain, form):
    """The same for fp32 outputs, which show what a bf16 one rounds away, up to the scores that the header names; lse is the
    score, to the rounding of its products' sum, of its multiplication and of itself (as check() derives)."""
    c = TreeCall(19, [n, 3], [n, 3], 0, N, 2, D, 16, 2, "roots", gain=gain)
    o, lse = c.run(cuda_dev, form=form, o_dtype=F.CP_F32)
    assert np.abs(f64(lse)).max() < 2 ** 14  # of the one key: lse is the score
    at = c.b.slots(0, 0, n) + c.b.slots(1, 0, 3)
    v = c.v.view(-1, 2, D)[at].repeat_interleave(N // 2, 1)
    assert torch.equal(o.cpu(), v.float())
    c.check(o, lse, "fp32", gain=gain)


@pytest.mark.parametrize("form", ["as_chosen", "clusters", "line"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["narrow", "half_tile_prefix", "half_tile", "wide", "with_prompts", "blocks", "no_groups"])
def test_a_query_that_is_not_a_number_stays_alone(cuda_dev, name, value, form):
    """A query row of NaN (or of infinities of both signs): NaN in its own o and lse alone.  Other rows within what
    test_gpu_prefix.py derives for rows beside such a one."""
    new, length, prefix, N, Nkv, D, page, words, pad = CASES[name]
    c = TreeCall(13, new, length, prefix, N, Nkv, D, page, words, "any", pad)
    n = c.rows
    good = [t.clone() for t in c.run(cuda_dev, form=form, o_dtype=F.CP_F32)]
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


# few sequences of as many tiles a block as a cluster is given (17 to 32 of 128 keys), and many over whole tiles of keys
LONG = {
    "shares_of_a_cluster": ([12, 20, 3, 1, 16, 9, 20, 0, 7], [8190, 5000, 7000, 4097, 300, 6500, 20, 900, 7300], 0, 16, 8, 64, 16, 1),
    "shares_of_a_cluster_128": ([20, 9, 40, 33], [15000, 9000, 12345, 16000], 0, 4, 4, 128, 64, 2),
    "shares_with_a_prefix": ([5, 17, 11, 2], [4000, 3900, 77, 1], 12000, 16, 8, 64, 32, 1),
    "blocks": ([7 + 5 * i % 24 for i in range(12)], [3000 - 211 * i % 2300 for i in range(12)], 0, 16, 8, 128, 32, 1),
    "blocks_64": ([30 - 7 * i % 25 for i in range(16)], [2990 - 333 * i % 2700 for i in range(16)], 0, 16, 8, 64, 16, 1),
}


@pytest.mark.parametrize("kind", ["random", "any"])
@pytest.mark.parametrize("name", sorted(LONG))
def test_long_sequences(cuda_dev, name, kind):
    new, length, prefix, N, Nkv, D, page, words = LONG[name]
    c = TreeCall(17, new, length, prefix, N, Nkv, D, page, words, kind)
    o, lse = c.run(cuda_dev, o_dtype=F.CP_F32)
    c.check(o, lse, "fp32", name)


@pytest.mark.parametrize("gain", [30.0, 300.0])
@pytest.mark.parametrize("N", [2, 16])
@pytest.mark.parametrize("form", ["as_chosen", "clusters", "line"])
def test_large_scores(cuda_dev, gain, N, form):
    c = TreeCall(6, [7, 12], [500, 900], 700, N, 2, 64, 16, 1, gain=gain)
    for s, m in enumerate(c.b.length):
        at = c.b.slots(s, 0, m)
        k = c.k.view(-1, 2, 64)
        k[at] = (k[at].float() * torch.linspace(0.01, 1, max(m, 1)).view(-1, 1, 1)).to(torch.bfloat16)
    o, lse = c.run(cuda_dev, form=form, o_dtype=F.CP_F32)
    c.check(o, lse, "fp32", "gain", gain)


@pytest.mark.parametrize("form", ["as_chosen", "clusters", "line"])
@pytest.mark.parametrize("name", ["narrow_edges", "half_tile_prefix", "wide", "with_prompts"])
def test_same_bits_twice_on_a_stream_and_by_graph(cuda_dev, name, form):
    new, length, prefix, N, Nkv, D, page, words, pad = CASES[name]
    c = TreeCall(7, new, length, prefix, N, Nkv, D, page, words, "random", pad)
    a = [t.clone() for t in c.run(cuda_dev, form=form)]
    n = c.rows
    same = lambda x, y: torch.equal(x[0][:n], y[0][:n]) and torch.equal(x[1][:, :n], y[1][:, :n])  # noqa: E731
    for _ in range(5):
        assert same(a, c.again())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    d = c.again(stream=s)
    s.synchronize()
    assert same(a, d)
    q, k, v, mask, pages, table, cu, kv_len = c.dev
    o, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
    ws = torch.empty(F.cp_tree_attn_workspace_size(c.R, len(new), max(new), words, prefix, N, Nkv, D, page, table.shape[1]),
                     dtype=torch.uint8, device=cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.again(o=o, lse=lse, workspace=ws)
    for step in range(3):
        ws.random_(0, 256)
        mask.copy_(mask.roll(1, 0))
        q.copy_(q.flip(1))
        kv_len.copy_((kv_len - step).clamp(min=0))
        graph.replay()
        assert same((o, lse), c.again()), step


def test_two_calls_at_once(cuda_dev):
    """Two streams with a workspace each, and two graphs over one, each get their own bits."""
    new, length, prefix, N, Nkv, D, page, words, pad = CASES["half_tile_prefix"]
    c = TreeCall(15, new, length, prefix, N, Nkv, D, page, words, "random", pad)
    c.run(cuda_dev)
    q, k, v, mask, pages, table, cu, kv_len = c.dev
    masks = [mask, mask.roll(1, 0).contiguous()]
    need = F.cp_tree_attn_workspace_size(c.R, len(new), max(new), words, prefix, N, Nkv, D, page, table.shape[1])
    ws = [torch.empty(need, dtype=torch.uint8, device=cuda_dev) for _ in range(2)]
    outs = [(torch.zeros_like(q), torch.zeros(N, c.R, device=cuda_dev)) for _ in range(2)]

    def call(i, w):
        F.cp_tree_attn_fwd(q, k, v, masks[i], pages, prefix, table, cu, kv_len, max(new), o=outs[i][0], lse=outs[i][1],
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


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("new", [2, 40])
def test_pages_past_32_bits_of_offset(cuda_dev, page, new):
    c = TreeCall(14, [new, 1, new], [300 + new, 90, new], 700, 16, 4, 128, page, 2)
    want = c.run(cuda_dev)
    q, k, v, mask, pages, table, cu, kv_len = c.dev
    extra = int(2.7e9) // (page * 4 * 128)
    big = []
    for small in (k, v):
        t = torch.empty(extra + c.b.total, page, 4, 128, dtype=torch.bfloat16, device=cuda_dev)
        t[:2 * c.b.total] = float("nan")
        t[extra:] = small
        big.append(t)
    got = F.cp_tree_attn_fwd(q, *big, mask, pages + extra, 700, torch.where(table < 0, table, table + extra), cu, kv_len, new)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("hint", [1, 3, 40])
def test_any_hint_is_right(cuda_dev, hint):
    c = TreeCall(12, [40, 1, 0, 17], [300, 5, 9, 17], 200, 8, 2, 64, 32, 2)
    c.check(*c.run(cuda_dev, hint=hint))


# new tokens, own lengths, prefix, N, Nkv, D, page, words: items of several row tiles (trees and prompts), and few key tiles
# for many blocks
ROW_TILES = {
    "trees_128": ([100, 70, 33], [900, 70, 1500], 0, 8, 1, 128, 16, 4),
    "prompt_128": ([300, 5], [300, 700], 130, 16, 2, 128, 64, 1),
    "trees_64": ([64, 200, 1], [2000, 200, 64], 0, 8, 1, 64, 32, 8),
    "prompt_64": ([400, 20], [1000, 90], 77, 6, 1, 64, 16, 1),
    "two_tiles_of_keys": ([150, 40], [150, 170], 0, 8, 2, 128, 16, 1),
    "one_tile_of_keys": ([90, 3], [90, 100], 0, 8, 2, 64, 16, 3),
}


@pytest.mark.parametrize("hint", [1, 20, None])
@pytest.mark.parametrize("form", ["as_chosen", "clusters", "line"])
@pytest.mark.parametrize("name", sorted(ROW_TILES))
def test_any_hint_is_right_in_every_form(cuda_dev, name, form, hint):
    """Fewer row tiles than an item has: its block, or its cluster, takes one behind the other, over shared memory that
    other blocks have just read.  The same bits every time."""
    new, length, prefix, N, Nkv, D, page, words = ROW_TILES[name]
    c = TreeCall(31, new, length, prefix, N, Nkv, D, page, words, pad=1)
    o, lse = (t.clone() for t in c.run(cuda_dev, hint=hint, form=form))
    c.check(o, lse)
    for _ in range(20):
        o2, lse2 = c.again(hint=hint)
        assert torch.equal(o[:c.rows], o2[:c.rows]) and torch.equal(lse[:, :c.rows], lse2[:, :c.rows])


def test_outputs_and_workspace_stay_in_bounds(cuda_dev):
    c = TreeCall(8, [3, 40, 1], [3, 300, 77], 130, 6, 2, 64, 16, 2, pad=2)
    c.run(cuda_dev)
    table = c.dev[5]
    need = F.cp_tree_attn_workspace_size(c.R, 3, 40, 2, 130, 6, 2, 64, 16, table.shape[1])
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=cuda_dev)
    o = torch.full((c.R + 2, 6, 64), 7.0, device=cuda_dev)
    lse = torch.full((6 * c.R + 8,), 7.0, device=cuda_dev)
    before = [t.clone() for t in c.dev]
    c.again(o=o[1:-1], lse=lse[4:-4].view(6, c.R), workspace=ws[256:256 + need])
    torch.cuda.synchronize()
    assert (o[0] == 7).all() and (o[-1] == 7).all() and (lse[:4] == 7).all() and (lse[-4:] == 7).all()
    assert (ws[:256] == 0xA5).all() and (ws[256 + need:] == 0xA5).all()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, c.dev))
    c.check(o[1:-1], lse[4:-4].view(6, c.R), "fp32")


@pytest.mark.parametrize("what", ["page", "prefix_page", "length", "negative_length", "counts", "counts_past_rows"])
@pytest.mark.parametrize("N", [4, 32])
@pytest.mark.parametrize("form", ["as_chosen", "clusters", "line"])
def test_bad_lists_are_reported(cuda_dev, what, N, form):
    c = TreeCall(9, [2, 3], [50, 40], 70, N, 2, 64, 16, 1)
    good = [t.clone() for t in c.run(cuda_dev, form=form)]
    wo, wl, size = c.want()
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
        if form != "line":  # (a block or a cluster sees one sequence)
            assert torch.equal(o[2:], good[0][2:]) and torch.equal(lse[:, 2:], good[1][:, 2:])
        # The line is cut in other places where the first sequence has another length, and a piece's weights are rounded
        # relative to the piece's own maximum: off by half a step of themselves either way, so within the same bounds.
        within(o[2:], wo[2:], "bf16", (2.0 ** -8 + 2.0 ** -12) * size[2:], "the other sequence")
        assert np.abs(f64(lse)[:, 2:] - wl[:, 2:]).max() <= 2.0 ** -12


def test_speculative_steps_decode_like_one_causal_attention(cuda_dev):
    """All calls as they are used: every step's pages are planned on the device, its drafted trees' ancestors and
    positions formed, their tokens stored by slot and position in the caches of two layers, attended, and one branch
    kept.  Each row's attention equals the 64-bit causal attention of its own branch behind what was kept before
    (inputs rounded where the cache rounds), in both layers, and no page is lost."""
    g = torch.Generator().manual_seed(10)
    rng = np.random.default_rng(10)
    N, Nkv, D, page, P, B, words, layers, n_pages, width = 8, 2, 64, 16, 37, 3, 1, 2, 60, 12
    rope, th, amp = rope_of(D, "half")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    caches = [torch.full((n_pages, page, Nkv, D), float("nan"), dtype=torch.bfloat16, device=cuda_dev)
              for _ in range(2 * layers)]
    handle = F.CpCaches(caches)
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
    wd = [w.to(cuda_dev) for w in (wq, wk)]
    draw = lambda n: [[rand(g, (n, h, D), "bf16") for h in (N, Nkv, Nkv)] for _ in range(layers)]  # noqa: E731
    # the shared prefix is a sequence of its own whose pages are planned like the others'
    table, stack, n_free = i32([[0] * width] * (B + 1)), i32(list(range(n_pages))), i32([n_pages, 0])
    had = i32([0] * (B + 1))
    prefix = draw(P)
    had, cu, slots, pos, _ = F.cp_cache_plan(had, i32([0] * (B + 1)), i32([0] * B + [P]), table, stack, n_free, page, P,
                                             n_free_out=n_free)
    for layer in range(layers):
        q, k, v = (t.to(cuda_dev) for t in prefix[layer])
        F.cp_cache_append_at(k, v, *caches[2 * layer:2 * layer + 2], slots, pos, rope=rope, wk=wd[1])
    pages = table[B, :-(-P // page)].contiguous()
    table, had, free0 = table[:B].contiguous(), had[:B].contiguous(), n_free[0].item()
    keep = had.clone()
    hist = [[] for _ in range(B)]  # each sequence's kept tokens: per layer (q, k, v) rows as drawn
    for step in range(6):
        new = [[20, 5, 33], [9, 1, 32], [7, 20, 5], [1, 1, 1], [16, 30, 2], [3, 0, 8]][step]
        R_ = sum(new) + 2
        parents = [T.random_parents(rng, n, "random") for n in new]
        had, cu, slots, pos, n_free = F.cp_cache_plan(had, keep, i32(new), table, stack, n_free, page, R_, P)
        assert n_free[1].item() == 0
        mask, pos = F.cp_tree_plan(i32(sum(parents, []) + [0, 0]), cu, had, words, P, pos=pos)
        rows = draw(R_)
        for layer in range(layers):
            q, k, v = (t.to(cuda_dev) for t in rows[layer])
            q = F.cp_cache_append_at(k, v, *caches[2 * layer:2 * layer + 2], slots, pos, rope=rope, q=q, wq=wd[0], wk=wd[1])
            o, lse = F.cp_tree_attn_fwd(q, *caches[2 * layer:2 * layer + 2], mask, pages, P, table, cu, had, max(new))
            r = 0
            for s in range(B):
                seen_new, depth = (np.tril(np.ones((new[s],) * 2, bool)), np.arange(new[s])) if new[s] > 32 else \
                    T.branches(parents[s])
                old = [torch.cat([prefix[layer][i]] + [h[layer][i] for h in hist[s]]) for i in range(3)]
                every = [torch.cat([old[i], rows[layer][i][r:r + new[s]]]) for i in range(3)]
                m = len(old[0])
                at = np.concatenate([np.arange(m), m + depth])
                qr, kr = (R.bf16(R.turn(R.norm(f64(every[i]), f64(w), 1e-6), at, th, amp, "half"))
                          for i, w in ((0, wq), (1, wk)))
                seen = np.concatenate([np.ones((new[s], m), bool), seen_new], 1)
                wo, wl, a = R.attention(qr[m:], kr, f64(every[2]), seen, 1 / math.sqrt(D))
                # a value next to a rounding border may go the other way in q or k: half a step (2^-8) of
                # single values, 2^-5 in a score of size sum|q k| scale < 8
                if new[s]:
                    assert np.abs(f64(lse)[:, r:r + new[s]] - wl).max() <= 2.0 ** -5
                within(o[r:r + new[s]], wo, "bf16", (2.0 ** -8 + 2.0 ** -4) * a, "step %d" % step)
                r += new[s]
        # one branch of each tree is accepted; a prompt stays whole
        kept, n_kept, r = [[0] * 32 for _ in range(B)], [], 0
        for s in range(B):
            if new[s] > 32 or new[s] == 0:
                path, count = list(range(new[s])), -1
            else:
                path = np.nonzero(T.branches(parents[s])[0][int(rng.integers(0, new[s]))])[0].tolist()
                count = len(path)
                kept[s][:count] = path
            n_kept.append(count)
            hist[s].append([[t[r:r + new[s]][path] for t in rows[layer]] for layer in range(layers)])
            r += new[s]
        keep = F.cp_cache_keep(handle, table, cu, had, i32(kept), i32(n_kept), R=R_)
        assert keep.tolist() == [sum(len(h[0][0]) for h in hist[s]) for s in range(B)]
    # all sequences end: every page that is not the prefix's is free again
    *_, n_free = F.cp_cache_plan(had, i32([0] * B), i32([0] * B), table, stack, n_free, page, 1)
    assert n_free.tolist() == [free0, 0]
    assert sorted(stack.tolist()[:free0] + pages.tolist()) == list(range(n_pages))
    assert F.cp_device_status() == 0
