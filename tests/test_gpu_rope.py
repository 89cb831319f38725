"""Rotary positions and the per-head norm with rotation, forward and backward,
against the 64-bit forms of rows_ref.py.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32): a rotated value
a c - b s is off by at most A (|a| + |b|) 8 u -- the fraction of a turn is rounded
to fp32 (pi 2^-25 radians, under 2 u), sincospif is within 2 ulps (4 u), and the
amplitude and the two products add a rounding each.  The norm adds its sum of D
squares (16 in a lane, log2(D/16) shuffles: under 20 u of the sum, half of it in
r), the root, the division and two products: 16 u more.  The norm's gradient has
the same pieces and a second sum: 48 u of r (|u| + |xh| mean|u xh|).  dw sums n
rows one after the other at worst: (n + 40) u of sum |g xh|.  On top of each, half
a step of the output's type."""
import numpy as np
import pytest
import torch

import rows_ref as R
from context_causal_attention_gb300 import ops as F

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
KIND = {"plain": F.CP_ROPE_PLAIN, "linear": F.CP_ROPE_LINEAR, "base": F.CP_ROPE_BASE, "by_parts": F.CP_ROPE_BY_PARTS}
ORDER = {"half": F.CP_ROPE_HALF, "interleaved": F.CP_ROPE_INTERLEAVED}


def f64(t):
    return t.detach().cpu().double().numpy()


def rand(g, shape, dt, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(DT[dt])


def rope_of(rot, order, scaling="plain", factor=8.0, original=64.0):
    r = F.cp_rope_freqs(rot, scaling=KIND[scaling], factor=factor, original_len=original, order=ORDER[order])
    th, amp = R.thetas(rot, scaling=scaling, factor=factor, original=original)
    return r, th, amp


def within(got, want, dt, slack, what):
    err, tol = np.abs(f64(got) - want), R.HALF[dt] * np.abs(want) + slack + 1e-37
    assert np.isfinite(f64(got)).all(), what
    assert (err <= tol).all(), "%s: %g over its bound" % (what, float((err / tol).max()))


# C, B, s, N, Nkv, D, rot: one token, heads that do not fill a warp's rows, odd
# lengths, several shards, one tensor alone
SHAPES = [
    (1, 1, 1, 1, 1, 64, 64), (1, 1, 1, 32, 8, 128, 128), (2, 3, 5, 3, 1, 64, 32), (4, 1, 16, 5, 5, 128, 64),
    (1, 2, 33, 7, 1, 64, 16), (1, 1, 257, 9, 3, 128, 32), (2, 2, 7, 6, 0, 64, 48),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("order", ["half", "interleaved"])
def test_rows(cuda_dev, shape, dt, order):
    """Every entry point on one shape: rotation and norm, both directions."""
    C, B, s, N, Nkv, D, rot = shape
    g = torch.Generator().manual_seed(C * 1000 + s)
    rope, th, amp = rope_of(rot, order, "by_parts" if s % 2 else "base")
    pos = torch.randint(-5, 1 << 20, (C, s), generator=g, dtype=torch.int32)
    p = pos.numpy()[:, None].repeat(B, 1)
    eps = 1e-5
    xs = [rand(g, (C, B, s, h, D), dt, 3.0) if h else None for h in (N, Nkv)]
    gs = [rand(g, (C, B, s, h, D), dt) if h else None for h in (N, Nkv)]
    ws = [1 + 0.3 * torch.randn(D, generator=g) if h else None for h in (N, Nkv)]
    dev = lambda l: [None if t is None else t.to(cuda_dev) for t in l]  # noqa: E731
    xd, gd, wd, pd = dev(xs), dev(gs), dev(ws), pos.to(cuda_dev)
    fwd, bwd = F.cp_rope_fwd(*xd, pd, rope), F.cp_rope_bwd(*gd, pd, rope)
    nf = F.cp_qk_norm_rope_fwd(*xd, *wd, pd, rope, eps=eps)
    nb = F.cp_qk_norm_rope_bwd(*gd, *xd, *wd, pd, rope, eps=eps)
    for t, what in enumerate("qk"):
        if xs[t] is None:
            assert fwd[t] is None and nb[2 + t] is None
            continue
        x, gr, w = f64(xs[t]), f64(gs[t]), f64(ws[t])
        u = R.U32
        within(fwd[t], R.turn(x, p, th, amp, order), dt, 8 * u * amp * R.pair_size(x, th, order), what + " rotated")
        within(bwd[t], R.turn(gr, p, th, amp, order, True), dt, 8 * u * amp * R.pair_size(gr, th, order),
               what + " rotated back")
        y = R.norm(x, w, eps)
        within(nf[t], R.turn(y, p, th, amp, order), dt, 24 * u * amp * R.pair_size(y, th, order), what + " normed")
        back = R.turn(gr, p, th, amp, order, True)
        dx, dw = R.norm_bwd(x, w, back, eps)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        size = np.abs(w) * amp * R.pair_size(gr, th, order)
        slack = 48 * u * r * (size + np.abs(x * r) * (size * np.abs(x * r)).mean(-1, keepdims=True))
        within(nb[t], dx, dt, slack, what + " norm gradient")
        rows = x.size // D
        big = (amp * R.pair_size(gr, th, order) * np.abs(x * r)).reshape(-1, D).sum(0)
        within(nb[2 + t], dw, "fp32", (rows + 40) * u * big, what + " weight gradient")


@pytest.mark.parametrize("scaling", ["plain", "linear", "base", "by_parts"])
def test_far_positions_lose_nothing(cuda_dev, scaling):
    """Positions up to the ends of int32: the angle is exact to the fp64 frequency."""
    rope, th, amp = rope_of(128, "half", scaling, 4.0, 4096.0)
    pos = torch.tensor([0, 1, -1, 4095, 1 << 20, 16777217, -(1 << 31), (1 << 31) - 1], dtype=torch.int32)
    x = rand(torch.Generator().manual_seed(3), (8, 4, 128), "fp32")
    y, _ = F.cp_rope_fwd(x.to(cuda_dev), None, pos.to(cuda_dev), rope)
    # the fp64 frequency itself is known to 2^-53 of its size on either side
    far = np.abs(pos.numpy().astype(np.float64))[:, None, None] * np.concatenate([th, th]) * 2.0 ** -51
    slack = amp * R.pair_size(f64(x), th, "half") * (8 * R.U32 + far)
    within(y, R.turn(f64(x), pos.numpy(), th, amp, "half"), "fp32", slack, scaling)


def test_phases_from_given_frequencies(cuda_dev):
    w = [1.0, 0.25, 3.0, 1e-9, 0.5, 2.0, 0.125, 6.0]
    rope = F.cp_rope_phases(w, amplitude=0.75)
    x = rand(torch.Generator().manual_seed(4), (3, 2, 64), "fp32")
    pos = torch.tensor([2, 1000, 123456], dtype=torch.int32)
    y, _ = F.cp_rope_fwd(x.to(cuda_dev), None, pos.to(cuda_dev), rope)
    slack = 0.75 * R.pair_size(f64(x), w, "half") * 8 * R.U32 + 123456 * 6 * 2.0 ** -50
    within(y, R.turn(f64(x), pos.numpy(), np.array(w), 0.75, "half"), "fp32", slack, "given frequencies")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("call", ["rope", "norm"])
def test_strided_rows_and_in_place(cuda_dev, dt, call):
    """q and k as slices of a fused projection, into new tensors and in place:
    the same bits as from dense copies; the v heads between them stay."""
    g = torch.Generator().manual_seed(5)
    N, Nkv, D = 6, 2, 128
    qkv = rand(g, (2, 37, N + 2 * Nkv, D), dt).to(cuda_dev)
    q, k = qkv[:, :, :N], qkv[:, :, N:N + Nkv]
    pos = torch.arange(37, dtype=torch.int32, device=cuda_dev)
    rope, _, _ = rope_of(64, "interleaved")
    w = [1 + 0.1 * torch.randn(D, generator=g).to(cuda_dev) for _ in range(2)]
    if call == "rope":
        run = lambda a, b, oa=None, ob=None: F.cp_rope_fwd(a, b, pos, rope, oa, ob)  # noqa: E731
    else:
        run = lambda a, b, oa=None, ob=None: F.cp_qk_norm_rope_fwd(a, b, *w, pos, rope, q_out=oa, k_out=ob)  # noqa: E731
    want = run(q.contiguous(), k.contiguous())
    got = run(q, k)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    v = qkv[:, :, N + Nkv:].clone()
    run(q, k, q, k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, :, N + Nkv:], v)


@pytest.mark.parametrize("which", ["q", "k", "both"])
@pytest.mark.parametrize("order", ["qkv", "kvq", "one_token"])
def test_one_of_two_slices_in_place(cuda_dev, which, order):
    """Slices of one buffer lie side by side, so either may be turned in place while the
    other goes elsewhere; the heads between them stay."""
    g = torch.Generator().manual_seed(12)
    N, Nkv, D = 3, 2, 64
    rows = rand(g, (1 if order == "one_token" else 41, N + 2 * Nkv, D), "bf16").to(cuda_dev)
    at = (2 * Nkv, 0) if order == "kvq" else (0, N)
    cut = lambda t: (t[:, at[0]:at[0] + N], t[:, at[1]:at[1] + Nkv])  # noqa: E731
    pos = torch.arange(len(rows), dtype=torch.int32, device=cuda_dev)
    rope, _, _ = rope_of(32, "half")
    w = [1 + 0.1 * torch.randn(D, generator=g).to(cuda_dev) for _ in range(2)]
    grads = [rand(g, (len(rows), h, D), "bf16").to(cuda_dev) for h in (N, Nkv)]
    calls = [lambda a, b, x=None, y=None: F.cp_rope_fwd(a, b, pos, rope, x, y),
             lambda a, b, x=None, y=None: F.cp_qk_norm_rope_fwd(a, b, *w, pos, rope, q_out=x, k_out=y),
             lambda a, b, x=None, y=None: F.cp_qk_norm_rope_bwd(*grads, a, b, *w, pos, rope, dq=x, dk=y)]
    for i, call in enumerate(calls):
        want = call(*(t.contiguous() for t in cut(rows)))
        buf = rows.clone()
        q, k = cut(buf)
        got = call(q, k, q if which != "k" else None, k if which != "q" else None)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        kept = torch.ones(N + 2 * Nkv, dtype=torch.bool, device=cuda_dev)
        for t, n in ((0, N), (1, Nkv)):
            if which in ("both", "qk"[t]):
                kept[at[t]:at[t] + n] = False
        assert torch.equal(buf[:, kept], rows[:, kept]), i


def test_backward_in_place_and_bf16_weights(cuda_dev):
    g = torch.Generator().manual_seed(6)
    q, k, gq, gk = (rand(g, (1, 1, 50, h, 64), "bf16").to(cuda_dev) for h in (4, 2, 4, 2))
    w = [(1 + 0.1 * torch.randn(64, generator=g)).to(torch.bfloat16).to(cuda_dev) for _ in range(2)]
    pos = torch.arange(50, dtype=torch.int32, device=cuda_dev)
    rope, _, _ = rope_of(64, "half")
    want = F.cp_qk_norm_rope_bwd(gq, gk, q, k, *[x.float() for x in w], pos, rope)
    a, b = gq.clone(), gk.clone()
    got = F.cp_qk_norm_rope_bwd(a, b, q, k, *w, pos, rope, dq=a, dk=b)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    a, b = q.clone(), k.clone()
    got = F.cp_qk_norm_rope_bwd(gq, gk, a, b, *w, pos, rope, dq=a, dk=b)
    assert got[0] is a and all(torch.equal(x, y) for x, y in zip(got, want))


def test_norm_alone_and_special_values(cuda_dev):
    """Without a rotation the norm stands alone; a row of zeros gives zeros; NaN and
    infinities stay in their row, and beside the rotated part in their value."""
    g = torch.Generator().manual_seed(7)
    x = rand(g, (9, 3, 64), "fp32")
    x[2, 1] = 0
    w = 1 + 0.1 * torch.randn(64, generator=g)
    y, _ = F.cp_qk_norm_rope_fwd(x.to(cuda_dev), None, w.to(cuda_dev), None, None, None, eps=1e-6)
    want = R.norm(f64(x), f64(w), 1e-6)
    within(y, want, "fp32", 24 * R.U32 * np.abs(want), "norm alone")
    assert (y[2, 1] == 0).all()
    pos = torch.arange(9, dtype=torch.int32, device=cuda_dev)
    for order in ("half", "interleaved"):
        rope, th, amp = rope_of(16, order)
        z = x.clone()
        z[4, 2, 20] = float("nan")
        z[5, 0, 63] = float("inf")
        z[6, 1, 3] = float("inf")
        t, _ = F.cp_rope_fwd(z.to(cuda_dev), None, pos, rope)
        t = t.cpu()
        assert torch.isnan(t[4, 2, 20]) and torch.isinf(t[5, 0, 63])
        assert torch.equal(t[..., 16:][torch.isfinite(z[..., 16:])], z[..., 16:][torch.isfinite(z[..., 16:])])
        bad = ~torch.isfinite(t[..., :16])
        assert bad.sum() == 2 and bad[6, 1].sum() == 2
        n, _ = F.cp_qk_norm_rope_fwd(z.to(cuda_dev), None, w.to(cuda_dev), None, pos, rope)
        ok = torch.isfinite(n.cpu()).all(-1)
        assert ok.sum() == 27 - 3 and not ok[4, 2] and not ok[5, 0] and not ok[6, 1]


def test_gradient_against_differences(cuda_dev):
    """The kernel's fp32 gradients against central differences of the 64-bit
    forward: step 1e-4 leaves (h^2/6) f''' ~ 1e-8, the kernel's own rounding 1e-5."""
    g = torch.Generator().manual_seed(8)
    rope, th, amp = rope_of(32, "interleaved", "by_parts")
    x, gr, w = rand(g, (3, 2, 64), "fp32"), rand(g, (3, 2, 64), "fp32"), 1 + 0.2 * torch.randn(64, generator=g)
    pos = torch.tensor([5, 70, 900], dtype=torch.int32)
    dq, _, dw, _ = F.cp_qk_norm_rope_bwd(gr.to(cuda_dev), None, x.to(cuda_dev), None, w.to(cuda_dev), None,
                                         pos.to(cuda_dev), rope, eps=1e-5)

    def loss(a, b):
        return float((R.turn(R.norm(a, b, 1e-5), pos.numpy(), th, amp, "interleaved") * f64(gr)).sum())

    X, W, h = f64(x), f64(w), 1e-4
    for at in [(0, 0, 0), (1, 1, 17), (2, 0, 40), (2, 1, 63)]:
        e = np.zeros_like(X)
        e[at] = h
        assert abs((loss(X + e, W) - loss(X - e, W)) / (2 * h) - float(dq[at])) < 1e-5
    for j in (0, 31, 63):
        e = np.zeros(64)
        e[j] = h
        assert abs((loss(X, W + e) - loss(X, W - e)) / (2 * h) - float(dw[j])) < 1e-4


def test_many_rows_are_the_same_twice(cuda_dev):
    """More rows than all blocks take at once, in both directions: the same bits twice
    (weight gradients included), in a graph and on another stream."""
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k, gq, gk = (torch.randn(2, 1, 9001, h, 64, generator=g, device=cuda_dev).to(torch.bfloat16)
                    for h in (5, 2, 5, 2))
    w = [torch.randn(64, generator=g, device=cuda_dev) for _ in range(2)]
    pos = torch.arange(18002, dtype=torch.int32, device=cuda_dev).view(2, 9001)
    rope, _, _ = rope_of(64, "half")
    ref = F.cp_qk_norm_rope_bwd(gq, gk, q, k, *w, pos, rope)
    out = [torch.empty_like(t) for t in ref]
    ws = torch.empty(F.cp_qk_norm_rope_bwd_workspace_size(2, 1, 9001, 5, 2, 64), dtype=torch.uint8, device=cuda_dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        F.cp_qk_norm_rope_bwd(gq, gk, q, k, *w, pos, rope, dq=out[0], dk=out[1], dwq=out[2], dwk=out[3], workspace=ws)
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_outputs_stay_in_bounds(cuda_dev):
    """Guard rows around outputs and workspace stay as they were."""
    g = torch.Generator().manual_seed(10)
    q = rand(g, (77, 3, 64), "bf16").to(cuda_dev)
    w = torch.ones(64, device=cuda_dev)
    pos = torch.arange(77, dtype=torch.int32, device=cuda_dev)
    rope, _, _ = rope_of(64, "half")
    big = torch.full((79, 3, 64), 7.0, dtype=torch.bfloat16, device=cuda_dev)
    F.cp_qk_norm_rope_fwd(q, None, w, None, pos, rope, q_out=big[1:78])
    assert (big[0] == 7).all() and (big[78] == 7).all()
    need = F.cp_qk_norm_rope_bwd_workspace_size(1, 1, 77, 3, 0, 64)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=cuda_dev)
    dw = torch.full((64 + 32,), 7.0, device=cuda_dev)
    big.fill_(7.0)
    F.cp_qk_norm_rope_bwd(q, None, q, None, w, None, pos, rope, dq=big[1:78], dwq=dw[16:80], workspace=ws[256:256 + need])
    assert (big[0] == 7).all() and (big[78] == 7).all() and (dw[:16] == 7).all() and (dw[80:] == 7).all()
    assert (ws[:256] == 0xA5).all() and (ws[256 + need:] == 0xA5).all()


# more units than all resident warps take at once (608 blocks of 8 warps forward, 304 backward), in odd
# numbers; several heads to a lane's walk; B > 1, where positions repeat; one tensor alone
MANY = [(2, 3, 1667, 5, 2, 64, 64), (1, 1, 9001, 20, 3, 64, 32), (3, 1, 2111, 9, 1, 128, 128), (1, 2, 5003, 3, 0, 128, 64),
        (1, 1, 4999, 33, 7, 128, 96)]


@pytest.mark.parametrize("shape", MANY)
@pytest.mark.parametrize("dt,order", [("bf16", "half"), ("bf16", "interleaved"), ("fp32", "half"), ("fp32", "interleaved")])
def test_many_rows(cuda_dev, shape, dt, order):
    """Rotation and norm, both directions, where a warp goes from token to token: every
    value against 64 bits, and the same bits on another stream.  dw: a thread adds the rows
    of its own tokens one after the other, then 3 shuffles, 8 warps, at most 10 blocks a warp and 5
    shuffles follow: (rows of a thread + 26) u of sum |g xh| in the place of all rows, and the
    40 u of the terms."""
    C, B, s, N, Nkv, D, rot = shape
    g = torch.Generator().manual_seed(s)
    rope, th, amp = rope_of(rot, order, "by_parts")
    pos = torch.randint(-9, 1 << 20, (C, s), generator=g, dtype=torch.int32)
    p, eps, u = pos.numpy()[:, None].repeat(B, 1), 1e-5, R.U32
    heads = [h for h in (N, Nkv) if h]
    pad = [None] * (2 - len(heads))
    xs, gs = ([rand(g, (C, B, s, h, D), dt, x) for h in heads] for x in (3.0, 1.0))
    ws = [1 + 0.3 * torch.randn(D, generator=g) for _ in heads]
    xd, gd, wd = ([t.to(cuda_dev) for t in l] + pad for l in (xs, gs, ws))
    pd = pos.to(cuda_dev)

    def calls():
        return [F.cp_rope_fwd(*xd, pd, rope), F.cp_rope_bwd(*gd, pd, rope),
                F.cp_qk_norm_rope_fwd(*xd, *wd, pd, rope, eps=eps), F.cp_qk_norm_rope_bwd(*gd, *xd, *wd, pd, rope, eps=eps)]

    fwd, bwd, nf, nb = got = calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = calls()
    side.synchronize()
    assert all(a is b or torch.equal(a, b) for x, y in zip(got, again) for a, b in zip(x, y))
    for t, h in enumerate(heads):
        x, gr, w = f64(xs[t]), f64(gs[t]), f64(ws[t])
        what = "qk"[t]
        within(fwd[t], R.turn(x, p, th, amp, order), dt, 8 * u * amp * R.pair_size(x, th, order), what + " rotated")
        back, pair = R.turn(gr, p, th, amp, order, True), amp * R.pair_size(gr, th, order)
        within(bwd[t], back, dt, 8 * u * pair, what + " rotated back")
        y = R.norm(x, w, eps)
        within(nf[t], R.turn(y, p, th, amp, order), dt, 24 * u * amp * R.pair_size(y, th, order), what + " normed")
        dx, dw = R.norm_bwd(x, w, back, eps)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        xh, size = np.abs(x * r), np.abs(w) * pair
        within(nb[t], dx, dt, 48 * u * r * (size + xh * (size * xh).mean(-1, keepdims=True)), what + " norm gradient")
        blocks = 304 * h // (N + Nkv) - 1  # at least
        mine = -(-C * B * s // (8 * blocks)) * -(-h // (512 // D))
        within(nb[2 + t], dw, "fp32", (mine + 66) * u * (pair * xh).reshape(-1, D).sum(0), what + " weight gradient")
