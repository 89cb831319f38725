"""Frequencies, and what the rotation, norm and append calls refuse on the host
before anything is launched (no GPU needed)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import rows_ref as R
from context_causal_attention_gb300 import _lib
from context_causal_attention_gb300 import ops as F

FAKE = 1 << 20  # aligned, never read
FAR = [FAKE + (i << 32) for i in range(12)]


@pytest.mark.parametrize("scaling", ["plain", "linear", "base", "by_parts"])
def test_frequencies(cplib, scaling):
    kind = {"plain": 0, "linear": 1, "base": 2, "by_parts": 3}[scaling]
    for rot in (16, 64, 128):
        r = F.cp_rope_freqs(rot, 10000.0, kind, 8.0, 4096, device="cpu")
        th, amp = R.thetas(rot, 10000.0, scaling, 8.0, 4096.0)
        turns = r.freqs.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
        assert np.abs(turns - th / (2 * np.pi)).max() <= 2.0 ** -52
        assert abs(r.amplitude - amp) <= amp * 2.0 ** -23


def test_phases_keep_the_fraction_of_a_turn(cplib):
    r = F.cp_rope_phases([2 * np.pi, np.pi, -np.pi / 2, 0.0], device="cpu")
    assert r.rot_dim == 8
    got = r.freqs.numpy().view(np.uint64)
    assert got.tolist() == [0, 1 << 63, 3 << 62, 0]


def test_phases_are_as_near_as_stated(cplib):
    """The stored turns against the given frequencies in exact fractions: within theta 2^-52 + 2^-62
    radians a position, modulo a turn (pi to 60 digits)."""
    turn = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")
    w = [10000.0 ** (-i / 64) for i in range(64)] + [6.283185307179586, -6.283185307179586, 3.0, -0.1, 1e-12, -1e-300]
    got = F.cp_rope_phases(w, device="cpu").freqs.numpy().view(np.uint64)
    for x, f in zip(w, got):
        off = (Fraction(int(f), 1 << 64) * turn - Fraction(x)) % turn
        off = min(off, turn - off)
        assert off <= abs(Fraction(x)) / 2 ** 52 + Fraction(1, 1 << 62), x


def test_frequency_refusals(cplib):
    f = np.zeros(64, np.uint64)
    a = ctypes.c_float(0)
    call = lambda rot=64, base=1e4, kind=0, factor=1.0, length=1.0: cplib.cp_rope_freqs(  # noqa: E731
        rot, base, kind, factor, length, f.ctypes.data, ctypes.byref(a))
    assert call() == 0
    assert call(rot=0) == 2 and call(rot=7) == 2 and call(rot=2, kind=2, factor=2.0) == 2
    assert call(base=0.5) == 10 and call(base=float("nan")) == 10 and call(kind=4) == 10
    assert call(kind=1, factor=0.5) == 10 and call(kind=3, factor=2.0, length=0.0) == 10
    assert call(kind=2, factor=1e300, rot=4) == 10
    assert cplib.cp_rope_freqs(64, 1e4, 0, 1.0, 1.0, None, ctypes.byref(a)) == 1
    w = np.array([7.0, np.inf])
    assert cplib.cp_rope_phases(w[:1].ctypes.data, 1, f.ctypes.data) == 10
    assert cplib.cp_rope_phases(w[1:].ctypes.data, 1, f.ctypes.data) == 10
    assert cplib.cp_rope_phases(w.ctypes.data, 0, f.ctypes.data) == 2
    assert cplib.cp_rope_phases(None, 1, f.ctypes.data) == 1


def test_a_rotation_stays_with_its_frequencies(cplib):
    """A list shorter than the rotated part is refused (the kernels read rot_dim / 2 entries),
    and what calls would not follow cannot be set."""
    f = torch.zeros(16, dtype=torch.int64)
    assert F.CpRope(f, 32, 0, 1.0).freqs is f and F.CpRope(f, 16, 1, 0.5).rot_dim == 16
    for bad, rot in ((f, 34), (f, 128), (f.int(), 32), (f.double(), 32), (torch.zeros(32, dtype=torch.int64)[::2], 32)):
        with pytest.raises(ValueError):
            F.CpRope(bad, rot, 0, 1.0)
    r = F.cp_rope_freqs(64, device="cpu")
    for name, value in (("freqs", f), ("rot_dim", 16), ("order", 1), ("amplitude", 2.0)):
        with pytest.raises(AttributeError):
            setattr(r, name, value)
    assert (r.rot_dim, r.order, r.amplitude) == (64, F.CP_ROPE_HALF, 1.0)


def spec(freqs=FAKE, rot=64, order=0, amp=1.0):
    return ctypes.byref(_lib.RopeStruct(freqs, rot, order, amp))


def rope(cplib, name="cp_rope_fwd", q=FAR[0], k=FAR[1], pos=FAKE, C=2, B=1, s=8, N=4, Nkv=2, D=64, qs=256, ks=128,
         dt=0, r="default", qo=FAR[2], ko=FAR[3]):
    return getattr(cplib, name)(q, k, pos, C, B, s, N, Nkv, D, qs, ks, dt, spec() if r == "default" else r, qo, ko,
                                None)


@pytest.mark.parametrize("name", ["cp_rope_fwd", "cp_rope_bwd"])
def test_rope_refusals(cplib, name):
    bad = lambda **kw: rope(cplib, name, **kw)  # noqa: E731
    for kw in (dict(q=None), dict(k=None), dict(pos=None), dict(qo=None), dict(ko=None), dict(r=None),
               dict(r=spec(freqs=None))):
        assert bad(**kw) == 1, kw
    for kw in (dict(C=0), dict(B=0), dict(s=0), dict(N=-1), dict(N=0, Nkv=0), dict(qs=255), dict(ks=120),
               dict(s=1 << 31), dict(C=1 << 16, s=1 << 16), dict(r=spec(rot=0)), dict(r=spec(rot=66)),
               dict(r=spec(rot=33)), dict(N=70000, qs=70000 * 64)):
        assert bad(**kw) == 2, kw
    for kw in (dict(D=96, qs=384, ks=192), dict(D=256, qs=1024, ks=512), dict(r=spec(rot=24))):
        assert bad(**kw) == 7, kw
    assert bad(dt=2) == 4
    for kw in (dict(r=spec(order=2)), dict(r=spec(amp=float("inf"))), dict(qo=FAR[0] + 16), dict(qo=FAR[1]),
               dict(ko=FAR[0]), dict(qo=FAR[2], ko=FAR[2] + 64), dict(q=FAR[0], k=FAR[1], ko=FAR[1] - 16)):
        assert bad(**kw) == 10, kw
    for kw in (dict(q=FAR[0] + 8), dict(qo=FAR[2] + 4), dict(pos=FAKE + 2), dict(qs=260), dict(r=spec(freqs=FAKE + 4))):
        assert bad(**kw) == 5, kw


def test_rows_written_over_other_rows_are_refused(cplib):
    """In place is where an output is its own input; an output over the other tensor's rows
    (q and k the same rows, or slices of one buffer that share heads) is not."""
    one, four = 64 * 2, 4 * 64 * 2  # bytes of a head, of q's row
    same = dict(N=4, Nkv=4, ks=256)
    for name in ("cp_rope_fwd", "cp_rope_bwd"):
        for kw in (
                dict(q=FAR[0], k=FAR[0], qo=FAR[0], ko=FAR[0], **same),       # both in place of the same rows
                dict(q=FAR[0], k=FAR[0], qo=FAR[0], ko=FAR[3], **same),       # q in place, k reads those rows
                dict(q=FAR[0], k=FAR[0], qo=FAR[2], ko=FAR[0], **same),
                dict(q=FAR[0], k=FAR[0] + one, qo=FAR[0], ko=FAR[0] + one, qs=512, ks=512),
                dict(q=FAR[0], k=FAR[0] + four - one, qo=FAR[0], ko=FAR[0] + four - one, qs=512, ks=512),
                dict(q=FAR[0] + one, k=FAR[0], qo=FAR[0] + one, ko=FAR[0], qs=512, ks=512),
                # k's last head is q's first of the next token
                dict(q=FAR[0], k=FAR[0] + 7 * one, qo=FAR[0], ko=FAR[0] + 7 * one, qs=512, ks=512),
                dict(q=FAR[0], k=FAR[0] + four, qo=FAR[0], ko=FAR[0] + four, qs=512, ks=384)):
            assert rope(cplib, name, **kw) == 10, kw


def test_norm_refusals(cplib):
    def fwd(q=FAR[0], wq=FAKE, wk=FAKE, pos=FAKE, r="default", eps=1e-6, wd=1, dt=0):
        return cplib.cp_qk_norm_rope_fwd(q, FAR[1], wq, wk, pos, 1, 1, 8, 4, 2, 64, 256, 128, dt, wd, eps,
                                         spec() if r == "default" else r, FAR[2], FAR[3], None)

    assert fwd(q=None) == 1 and fwd(wq=None) == 1 and fwd(wk=None) == 1 and fwd(pos=None) == 1
    assert fwd(eps=-1.0) == 10 and fwd(eps=float("nan")) == 10 and fwd(wd=3) == 4 and fwd(dt=3) == 4
    assert fwd(wq=FAKE + 4) == 5 and fwd(r=spec(rot=24)) == 7
    n = ctypes.c_size_t(0)
    size = cplib.cp_qk_norm_rope_bwd_workspace_size
    assert size(1, 1, 8, 4, 2, 64, ctypes.byref(n)) == 0 and n.value > 0
    assert size(1, 1, 8, 4, 2, 64, None) == 1 and size(1, 1, 0, 4, 2, 64, ctypes.byref(n)) == 2
    assert size(1, 1, 8, 4, 2, 80, ctypes.byref(n)) == 7

    def bwd(gq=FAR[4], gk=FAR[5], dq=FAR[2], dk=FAR[3], dwq=FAR[6], dwk=FAR[7], ws=FAR[8], nb=n.value, wq=FAKE):
        return cplib.cp_qk_norm_rope_bwd(gq, gk, FAR[0], FAR[1], wq, FAKE, FAKE, 1, 1, 8, 4, 2, 64, 256, 128, 0, 1,
                                         1e-6, spec(), dq, dk, dwq, dwk, ws, nb, None)

    for kw in (dict(gq=None), dict(gk=None), dict(dwq=None), dict(dwk=None), dict(wq=None), dict(dq=None)):
        assert bwd(**kw) == 1, kw
    assert bwd(ws=None) == 6 and bwd(nb=n.value - 1) == 6
    assert bwd(ws=FAR[8] + 128) == 5 and bwd(dwq=FAR[6] + 2) == 5 and bwd(gq=FAR[4] + 8) == 5
    assert bwd(dq=FAR[4] + 16) == 10 and bwd(dq=FAR[5]) == 10 and bwd(dk=FAR[4]) == 10


def test_weight_gradients_that_share_memory_are_refused(cplib):
    def bwd(dwq, dwk):
        return cplib.cp_qk_norm_rope_bwd(FAR[4], FAR[5], FAR[0], FAR[1], FAKE, FAKE, FAKE, 1, 1, 8, 4, 2, 64, 256, 128,
                                         0, 1, 1e-6, spec(), FAR[2], FAR[3], dwq, dwk, FAR[8], 1 << 30, None)

    for off in (0, 4, 252, -4, -252):
        assert bwd(FAR[6], FAR[6] + off) == 10, off


def test_append_refusals(cplib):
    def app(q=FAR[0], k=FAR[1], v=FAR[2], qs=256, ks=128, vs=128, dt=0, R_=8, N=4, Nkv=2, D=64, wq=None, wk=None, wd=1,
            eps=1e-6, r="default", base=0, kc=FAR[3], vc=FAR[4], pages=10, page=16, table=FAKE, B=2, most=4, cu=FAKE,
            ln=FAKE, qo=FAR[5]):
        return cplib.cp_cache_append(q, k, v, qs, ks, vs, dt, R_, N, Nkv, D, wq, wk, wd, eps,
                                     spec() if r == "default" else r, base, kc, vc, pages, page, table, B, most, cu,
                                     ln, qo, None)

    for kw in (dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(table=None), dict(cu=None),
               dict(ln=None), dict(q=None), dict(qo=None), dict(r=spec(freqs=None))):
        assert app(**kw) == 1, kw
    for kw in (dict(R_=0), dict(R_=1 << 31), dict(N=-1), dict(Nkv=0), dict(pages=0), dict(B=0), dict(B=4097),
               dict(most=0), dict(pages=1 << 28), dict(most=1 << 28), dict(qs=255), dict(ks=64), dict(vs=64),
               dict(r=spec(rot=65))):
        assert app(**kw) == 2, kw
    for kw in (dict(D=96, qs=384, ks=192, vs=192), dict(page=8), dict(page=48), dict(page=512), dict(r=spec(rot=24))):
        assert app(**kw) == 7, kw
    assert app(dt=5) == 4 and app(wd=5) == 4
    for kw in (dict(wk=FAKE, eps=-1.0), dict(base=1 << 31), dict(vc=FAR[3]), dict(qo=FAR[1]), dict(qo=FAR[0] + 16),
               dict(qo=FAR[0], dt=1), dict(qo=FAR[0], qs=512)):
        assert app(**kw) == 10, kw
    for kw in (dict(k=FAR[1] + 8), dict(cu=FAKE + 2), dict(ks=132), dict(wq=FAKE + 4), dict(kc=FAR[3] + 8)):
        assert app(**kw) == 5, kw


def test_append_refuses_caches_that_overlap(cplib):
    size = 10 * 16 * 2 * 64 * 2  # bytes of a cache

    def app(kc=FAR[3], vc=FAR[4], qo=FAR[5]):
        return cplib.cp_cache_append(FAR[0], FAR[1], FAR[2], 256, 128, 128, 0, 8, 4, 2, 64, None, None, 1, 1e-6, spec(),
                                     0, kc, vc, 10, 16, FAKE, 2, 4, FAKE, FAKE, qo, None)

    for off in (0, 16, size - 16, -16, 16 - size):
        assert app(vc=FAR[3] + off) == 10, off
    for cache in (FAR[3], FAR[4]):
        for off in (0, size - 16, 16 - 8 * 4 * 64 * 2):
            assert app(qo=cache + off) == 10, off


def test_binding_refusals(cplib):
    """Shapes, strides and devices that the binding refuses before the call."""
    rope = F.cp_rope_freqs(64, device="cpu")
    pos = torch.zeros(5, dtype=torch.int32)
    q = torch.zeros(5, 2, 64)
    for bad in (q[:, :, ::2], q.transpose(0, 1), q.transpose(1, 2), q[0]):
        with pytest.raises(ValueError):
            F.cp_rope_fwd(bad, None, pos, rope)
    with pytest.raises(ValueError):
        F.cp_rope_fwd(torch.zeros(2, 6, 2, 64)[:, :5], None, pos, rope)  # tokens at two distances
    with pytest.raises(ValueError):
        F.cp_rope_fwd(q, torch.zeros(4, 2, 64), pos, rope)
    with pytest.raises(ValueError):
        F.cp_rope_fwd(q, None, pos.long(), rope)
    with pytest.raises(ValueError):
        F.cp_rope_fwd(q, None, pos[:4], rope)
    with pytest.raises(ValueError):
        F.cp_rope_fwd(q, None, pos, rope, q_out=torch.zeros(5, 2, 64, dtype=torch.bfloat16))
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        F.cp_rope_fwd(q, None, pos, rope)  # not on a GPU


def test_repeated_tokens_are_refused(cplib):
    """Rows that an expanded dimension repeats lie at no distance from one another: read as
    tokens at the outer dimension's distance they would end far behind the tensor."""
    assert F._head_rows(torch.zeros(3, 2, 4, 64)) == (256, (3, 2), 4, 64)
    assert F._head_rows(torch.zeros(3, 1, 9, 64)[:, :, :4].expand(3, 1, 4, 64)) == (576, (3, 1), 4, 64)
    for lead in ((3, 2), (2, 3, 2), (1, 3, 5)):
        x = torch.zeros(*lead[:-1], 1, 4, 64).expand(*lead, 4, 64)
        with pytest.raises(ValueError, match="one distance"):
            F._head_rows(x)
    for x in (torch.zeros(1, 2, 4, 64).expand(3, 2, 4, 64), torch.zeros(4, 64).expand(5, 4, 64)):
        with pytest.raises(ValueError, match="one distance"):
            F._head_rows(x)


def test_prefix_attention_refusals(cplib):
    n = ctypes.c_size_t(0)

    def size(R_=8, B=2, new=4, P=100, N=8, Nkv=2, D=64, page=16, most=4, out=ctypes.byref(n)):
        return cplib.cp_prefix_attn_workspace_size(R_, B, new, P, N, Nkv, D, page, most, out)

    assert size() == 0 and n.value > 0
    need = n.value
    assert size(P=0) == 0 and size(R_=1, new=1, B=1) == 0 and size(B=4096) == 0
    assert size(out=None) == 1
    for kw in (dict(R_=0), dict(B=0), dict(B=4097), dict(new=0), dict(new=9), dict(P=-1), dict(P=(1 << 31) - 255),
               dict(N=0), dict(Nkv=0), dict(most=0), dict(most=1 << 27), dict(R_=1 << 28, N=64)):
        assert size(**kw) == 2, kw
    assert size(N=9) == 3
    for kw in (dict(D=96), dict(D=256), dict(page=8), dict(page=24), dict(page=512)):
        assert size(**kw) == 7, kw

    def call(q=FAR[0], k=FAR[1], v=FAR[2], pages=10, page=16, pp=FAKE, P=100, table=FAKE, B=2, most=4, cu=FAKE, ln=FAKE,
             new=4, R_=8, N=8, Nkv=2, D=64, scale=0.125, o=FAR[3], od=0, lse=FAKE, ws=FAR[4], nb=need):
        return cplib.cp_prefix_attn_fwd(q, k, v, pages, page, pp, P, table, B, most, cu, ln, new, R_, N, Nkv, D, scale,
                                        o, od, lse, ws, nb, None)

    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(pp=None), dict(table=None), dict(cu=None), dict(ln=None),
               dict(o=None), dict(lse=None)):
        assert call(**kw) == 1, kw
    for kw in (dict(pages=0), dict(pages=1 << 27), dict(R_=0), dict(new=0), dict(new=9)):
        assert call(**kw) == 2, kw
    assert call(N=9) == 3 and call(od=2) == 4
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**kw) == 10, kw
    for kw in (dict(q=FAR[0] + 8), dict(k=FAR[1] + 8), dict(o=FAR[3] + 8), dict(lse=FAKE + 2), dict(cu=FAKE + 1),
               dict(pp=FAKE + 2), dict(ws=FAR[4] + 128)):
        assert call(**kw) == 5, kw
    assert call(ws=None) == 6 and call(nb=need - 1) == 6
    assert call(D=96) == 7 and call(page=48) == 7


def test_stalled_prefix_attention_checks_as_the_call_does(cplib):
    def call(q=FAR[0], ns=10_000_000, nb=1 << 40, ws=FAR[4]):
        return cplib.cp_selftest_stalled_prefix_attn(q, FAR[1], FAR[2], 10, 16, FAKE, 100, FAKE, 2, 4, FAKE, FAKE, 4, 8, 8,
                                                     2, 64, 0.125, FAR[3], 0, FAKE, ws, nb, ns, None)

    for ns in (0, 999_999, 2_000_000_001):
        assert call(ns=ns) == 10, ns
    assert call(q=None) == 1 and call(nb=1) == 6 and call(ws=None) == 6 and call(q=FAR[0] + 8) == 5


def test_prefix_binding_refusals(cplib):
    bf, i32 = torch.bfloat16, torch.int32
    kc = torch.zeros(4, 16, 2, 64, dtype=bf)
    q, pages, table = torch.zeros(3, 8, 64, dtype=bf), torch.zeros(2, dtype=i32), torch.zeros(1, 2, dtype=i32)
    cu, ln = torch.tensor([0, 3], dtype=i32), torch.tensor([3], dtype=i32)
    ok = dict(q=q, k_cache=kc, v_cache=kc.clone(), prefix_pages=pages, prefix_len=20, table=table, cu_new=cu, kv_len=ln,
              max_new=3)
    for kw in (dict(q=q.float()), dict(q=q[:, ::2]), dict(q=q[0]), dict(prefix_pages=pages[:1]),
               dict(prefix_pages=pages.long()), dict(cu_new=cu[:1]), dict(o=torch.zeros(3, 8, 32, dtype=bf)),
               dict(lse=torch.zeros(3, 8)), dict(v_cache=kc[:3])):
        with pytest.raises(ValueError):
            F.cp_prefix_attn_fwd(**dict(ok, **kw))
    for kw in (dict(table=table.long()), dict(k_cache=kc.float(), v_cache=kc.float())):
        with pytest.raises(TypeError):
            F.cp_prefix_attn_fwd(**dict(ok, **kw))


def test_missing_lists_get_the_librarys_error(cplib, monkeypatch):
    """What is left out where it is needed reaches the library, which refuses it (on
    the host, before anything is launched)."""
    monkeypatch.setattr(F, "_here", lambda *ts: 0)
    monkeypatch.setattr(F, "_raw_stream", lambda stream, dev: None)
    bf, i32 = torch.bfloat16, torch.int32
    kc = torch.zeros(4, 16, 2, 64, dtype=bf)
    q, table = torch.zeros(3, 8, 64, dtype=bf), torch.zeros(1, 2, dtype=i32)
    cu, ln = torch.tensor([0, 3], dtype=i32), torch.tensor([3], dtype=i32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    rope, pos, w = F.cp_rope_freqs(64, device="cpu"), torch.zeros(3, dtype=i32), torch.ones(64)
    for call in (lambda: F.cp_prefix_attn_fwd(q, kc, kc.clone(), None, 20, table, cu, ln, 3, workspace=ws),
                 lambda: F.cp_rope_fwd(q, None, None, rope), lambda: F.cp_rope_bwd(q, None, pos, None),
                 lambda: F.cp_qk_norm_rope_fwd(q, None, w, None, None, rope),
                 lambda: F.cp_qk_norm_rope_fwd(q, q, w, None, pos, rope),
                 lambda: F.cp_qk_norm_rope_bwd(q, None, q, None, w, None, None, rope, workspace=ws)):
        with pytest.raises(F.CpError) as e:
            call()
        assert e.value.status == 1
