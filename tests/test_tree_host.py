"""What the calls of the page plan, the storing by slots, the drafted trees and the kept branch refuse on the
host before anything is launched, and the tests' own plain forms (no GPU needed)."""
import ctypes
import glob
import os

import numpy as np
import pytest
import torch

import tree_ref as T
from conftest import ROOT
from context_causal_attention_gb300 import ops as F

FAKE = 1 << 20  # aligned, never read
FAR = [FAKE + (i << 32) for i in range(16)]


def args(spec, **change):
    names = [n for n, _ in spec]
    for k in change:
        assert k in names, k
    return [change.get(n, v) for n, v in spec]


PLAN = [("had", FAR[0]), ("keep", FAR[1]), ("n_new", FAR[2]), ("B", 4), ("table", FAR[3]), ("max_pages", 8),
        ("page", 16), ("free", FAR[4]), ("n_pages", 100), ("n_free", FAR[5]), ("base", 0), ("R", 64),
        ("kv_len", FAR[6]), ("cu", FAR[7]), ("slots", FAR[8]), ("pos", FAR[9]), ("n_free_out", FAR[10]), ("stream", None)]


def test_plan_refusals(cplib):
    call = lambda **c: cplib.cp_cache_plan(*args(PLAN, **c))  # noqa: E731
    for n in ("had", "keep", "n_new", "table", "free", "n_free", "kv_len", "cu", "slots", "pos", "n_free_out"):
        assert call(**{n: None}) == 1, n
        assert call(**{n: FAR[11] + 2}) == 5, n
    assert call(B=0) == 2 and call(B=4097) == 2 and call(R=0) == 2 and call(R=1 << 30) == 2
    assert call(max_pages=0) == 2 and call(n_pages=0) == 2 and call(max_pages=1 << 28) == 2 and call(n_pages=1 << 28) == 2
    assert call(page=8) == 7 and call(page=48) == 7 and call(page=512) == 7
    assert call(base=1 << 31) == 10 and call(base=-(1 << 31) - 1) == 10
    # results apart from one another and from the lists, but for those that may be in place
    assert call(kv_len=FAR[2]) == 10 and call(cu=FAR[0]) == 10 and call(slots=FAR[1] + 8) == 10
    assert call(pos=FAR[8] + 4 * 63) == 10 and call(n_free_out=FAR[7]) == 10 and call(table=FAR[4]) == 10
    assert call(kv_len=FAR[0] + 4) == 10 and call(n_free_out=FAR[5] - 4) == 10 and call(free=FAR[3] + 4 * 31) == 10
    assert call(had=FAR[3]) == 10 and call(n_free=FAR[4] + 8) == 10 and call(n_new=FAR[9] + 4) == 10


APPEND = [("q", FAR[0]), ("k", FAR[1]), ("v", FAR[2]), ("qs", 4 * 64), ("ks", 2 * 64), ("vs", 2 * 64), ("dtype", 0),
          ("R", 8), ("N", 4), ("Nkv", 2), ("D", 64), ("wq", None), ("wk", None), ("wd", 1), ("eps", 1e-6),
          ("rope", None), ("kc", FAR[3]), ("vc", FAR[4]), ("n_pages", 10), ("page", 16), ("slots", FAR[5]),
          ("pos", FAR[6]), ("q_out", FAR[7]), ("stream", None)]


def test_append_at_refusals(cplib):
    call = lambda **c: cplib.cp_cache_append_at(*args(APPEND, **c))  # noqa: E731
    for n in ("q", "k", "v", "kc", "vc", "slots", "pos", "q_out"):
        assert call(**{n: None}) == 1, n
        assert call(**{n: FAR[9] + 2}) == 5, n
    assert call(R=0) == 2 and call(Nkv=0) == 2 and call(N=-1) == 2 and call(D=96) == 7 and call(page=24) == 7
    assert call(dtype=2) == 4 and call(wd=5) == 4 and call(ks=100) == 2 and call(qs=4 * 64 + 4) == 5
    assert call(wk=FAR[8], eps=-1.0) == 10 and call(wk=FAR[8], eps=float("nan")) == 10
    assert call(vc=FAR[3] + 16) == 10 and call(q_out=FAR[1]) == 10 and call(q_out=FAR[3] + 32) == 10
    assert call(n_pages=1 << 28) == 2


KEEP = [("caches", None), ("n", 2), ("n_pages", 10), ("page", 16), ("Nkv", 2), ("D", 64), ("table", FAR[3]), ("B", 4),
        ("max_pages", 8), ("cu", FAR[4]), ("kv_len", FAR[5]), ("R", 64), ("kept", FAR[6]), ("max_kept", 5),
        ("n_kept", FAR[7]), ("kv_keep", FAR[8]), ("stream", None)]


def test_keep_refusals(cplib):
    def call(caches=(FAR[0], FAR[1]), **c):
        ptrs = None if caches is None else (ctypes.c_void_p * len(caches))(*caches)
        c.setdefault("n", 0 if caches is None else len(caches))
        return cplib.cp_cache_keep(*args(KEEP, caches=ptrs, **c))
    assert call(caches=None, n=2) == 1 and call(caches=(FAR[0], None)) == 1
    for n in ("table", "cu", "kv_len", "kept", "n_kept", "kv_keep"):
        assert call(**{n: None}) == 1, n
        assert call(**{n: FAR[11] + 2}) == 5, n
    assert call(caches=(FAR[0], FAR[1] + 8)) == 5
    assert call(n=0) == 2 and call(caches=[FAKE + (i << 32) for i in range(257)]) == 2
    assert call(max_kept=0) == 2 and call(max_kept=513) == 2 and call(R=0) == 2 and call(B=4097) == 2
    assert call(D=32) == 7 and call(page=100) == 7
    size = 10 * 16 * 2 * 64 * 2
    assert call(caches=(FAR[0], FAR[0] + size - 16)) == 10 and call(caches=(FAR[1], FAR[0], FAR[1])) == 10
    for n in ("table", "cu", "kv_len", "kept", "n_kept"):
        assert call(kv_keep=dict(KEEP)[n]) == 10, n


TREE = [("parent", FAR[0]), ("cu", FAR[1]), ("kv_len", FAR[2]), ("B", 4), ("R", 64), ("words", 2), ("base", 0),
        ("mask", FAR[3]), ("pos", FAR[4]), ("stream", None)]


def test_tree_plan_refusals(cplib):
    call = lambda **c: cplib.cp_tree_plan(*args(TREE, **c))  # noqa: E731
    for n in ("parent", "cu", "kv_len", "mask", "pos"):
        assert call(**{n: None}) == 1, n
        assert call(**{n: FAR[11] + 2}) == 5, n
    assert call(B=0) == 2 and call(B=4097) == 2 and call(R=0) == 2 and call(words=0) == 2 and call(words=17) == 2
    assert call(base=1 << 31) == 10
    # results apart from one another and from the lists
    for n in ("parent", "cu", "kv_len"):
        assert call(mask=dict(TREE)[n]) == 10 and call(pos=dict(TREE)[n] + 4) == 10, n
    assert call(pos=FAR[3] + 4 * 127) == 10


ATTN = [("q", FAR[0]), ("kc", FAR[1]), ("vc", FAR[2]), ("n_pages", 100), ("page", 16), ("pre", FAR[3]), ("P", 32),
        ("table", FAR[4]), ("B", 4), ("max_pages", 8), ("cu", FAR[5]), ("kv_len", FAR[6]), ("mask", FAR[7]),
        ("words", 2), ("max_new", 8), ("R", 64), ("N", 4), ("Nkv", 2), ("D", 64), ("scale", 0.125), ("o", FAR[8]),
        ("od", 0), ("lse", FAR[9]), ("ws", FAR[10]), ("ws_bytes", 1 << 40), ("stream", None)]


def test_tree_attention_refusals(cplib):
    call = lambda **c: cplib.cp_tree_attn_fwd(*args(ATTN, **c))  # noqa: E731
    for n in ("q", "kc", "vc", "pre", "table", "cu", "kv_len", "mask", "o", "lse"):
        assert call(**{n: None}) == 1, n
        assert call(**{n: FAR[11] + 2}) == 5, n
    assert call(words=0) == 2 and call(words=17) == 2 and call(R=0) == 2 and call(max_new=65) == 2 and call(B=0) == 2
    assert call(D=96) == 7 and call(page=8) == 7 and call(N=3) == 3 and call(od=7) == 4
    assert call(scale=0.0) == 10 and call(scale=float("nan")) == 10
    assert call(ws=None) == 6 and call(ws_bytes=100) == 6 and call(ws=FAR[10] + 128) == 5
    n = ctypes.c_size_t(0)
    size = lambda *a: cplib.cp_tree_attn_workspace_size(*a, ctypes.byref(n))  # noqa: E731
    assert size(64, 4, 8, 2, 32, 4, 2, 64, 16, 8) == 0 and n.value > 0
    assert size(64, 4, 8, 0, 32, 4, 2, 64, 16, 8) == 2 and size(64, 4, 8, 17, 32, 4, 2, 64, 16, 8) == 2
    assert size(0, 4, 8, 2, 32, 4, 2, 64, 16, 8) == 2 and size(64, 4, 8, 2, 32, 5, 2, 64, 16, 8) == 3
    assert cplib.cp_tree_attn_workspace_size(64, 4, 8, 2, 32, 4, 2, 64, 16, 8, None) == 1


def test_stalled_tree_attention_checks_as_the_call_does(cplib):
    def call(ns=10_000_000, **c):
        return cplib.cp_selftest_stalled_tree_attn(*args(ATTN, **c)[:-1], ns, None)

    for ns in (0, 999_999, 2_000_000_001):
        assert call(ns) == 10, ns
    assert call(q=None) == 1 and call(mask=None) == 1 and call(words=17) == 2 and call(ws_bytes=1) == 6
    assert call(q=FAR[0] + 8) == 5
    i32, bf = lambda *s: torch.zeros(*s, dtype=torch.int32), lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    for mask in (None, i32(6, 1), i32(5), i32(5, 2).float(), i32(2, 5).t()):
        with pytest.raises(ValueError):
            F.cp_selftest_stalled_tree_attn(10_000_000, bf(5, 4, 64), bf(4, 16, 2, 64), bf(4, 16, 2, 64), mask, None, 0,
                                            i32(3, 2), i32(4), i32(3), 2)


def test_binding_refusals(cplib):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):  # tables of another batch
        F.cp_cache_plan(i32(3), i32(4), i32(4), i32(4, 2), i32(9), i32(2), 16, 8)
    with pytest.raises(ValueError):
        F.cp_cache_plan(i32(4).long(), i32(4), i32(4), i32(4, 2), i32(9), i32(2), 16, 8)
    with pytest.raises(ValueError):
        F.cp_cache_plan(i32(4), i32(4), i32(4), i32(2, 4).t(), i32(9), i32(2), 16, 8)
    with pytest.raises(ValueError):
        F.cp_cache_plan(i32(4), i32(4), i32(4), i32(4, 2), i32(9), i32(2), 16, 8, slots=i32(9))
    with pytest.raises(ValueError):
        F.cp_tree_plan(i32(6), i32(3), i32(3), 1)
    with pytest.raises(ValueError):
        F.cp_tree_plan(i32(6), i32(4), i32(3), 2, mask=i32(6, 1))
    kc, vc = bf(4, 16, 2, 64), bf(4, 16, 2, 64)
    with pytest.raises(ValueError):
        F.cp_cache_append_at(bf(5, 2, 64), bf(5, 2, 64), kc, vc, i32(4), i32(5))
    with pytest.raises(ValueError):
        F.cp_cache_append_at(bf(5, 2, 64), bf(5, 2, 64), kc, vc, i32(5).float(), i32(5))
    with pytest.raises(TypeError):
        F.cp_cache_append_at(bf(5, 2, 64), bf(5, 2, 64), kc.float(), vc.float(), i32(5), i32(5))
    with pytest.raises(ValueError):
        F.CpCaches([])
    with pytest.raises(ValueError):
        F.CpCaches([kc, bf(5, 16, 2, 64)])
    with pytest.raises(TypeError):
        F.CpCaches([kc.float()])
    with pytest.raises(ValueError):
        F.CpCaches([kc, bf(4, 2, 16, 64).transpose(1, 2)])
    with pytest.raises(AttributeError):
        F.CpCaches([kc]).caches = ()
    with pytest.raises(ValueError):
        F.cp_cache_keep([kc, vc], i32(3, 2), i32(4), i32(3), i32(2, 5), i32(3))
    for mask in (None, i32(6, 1), i32(5), i32(5, 2).float(), i32(2, 5).t()):
        with pytest.raises(ValueError):
            F.cp_tree_attn_fwd(bf(5, 4, 64), kc, vc, mask, None, 0, i32(3, 2), i32(4), i32(3), 2)


def test_plain_plan_keeps_every_page_once():
    """The tests' own form: over random steps no page is lost or handed out twice."""
    g = np.random.default_rng(0)
    B, page, n_pages, width = 7, 4, 60, 20
    table, stack, n_free, had = [[-1] * width for _ in range(B)], list(range(n_pages)), n_pages, [0] * B
    for _ in range(300):
        keep = [int(g.integers(0, h + 1)) if g.random() < 0.5 else h for h in had]
        new = [int(g.integers(0, min(12, width * page - k) + 1)) for k in keep]
        r = T.plan(had, keep, new, table, stack, n_free, page, 100)
        had, n_free = r["kv_len"], r["n_free"][0]
        owned = [p for b in range(B) for p in table[b][:-(-had[b] // page)]]
        assert sorted(owned + stack[:n_free]) == list(range(n_pages))


def test_plain_branches():
    seen, depth = T.branches([-1, 0, 0, 1, -1, 4, 3])
    assert depth.tolist() == [0, 1, 1, 2, 0, 1, 3]
    assert np.nonzero(seen[6])[0].tolist() == [0, 1, 3, 6]
    words = T.packed(np.eye(40, dtype=bool), 2)
    assert words[31].tolist() == [-2 ** 31, 0] and words[33].tolist() == [0, 2]


def test_cluster_barriers_order_what_was_read_before_them():
    """Blocks of a cluster read each other's shared memory and then overwrite it or end: a barrier between that arrives
    without release orders none of those reads."""
    sources = glob.glob(os.path.join(ROOT, "context_causal_attention_gb300", "csrc", "*.cu*"))
    assert len(sources) > 20
    for path in sources:
        with open(path) as f:
            assert "barrier.cluster.arrive.relaxed" not in f.read(), path
