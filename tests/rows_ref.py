"""64-bit forms of the rotation, the per-head norm, the paged append and the
attention over a shared prefix, in plain numpy, for the tests."""
import math

import numpy as np

U32 = 2.0 ** -24          # half a step of fp32, relative
HALF = {"bf16": 2.0 ** -8, "fp32": U32}


def thetas(rot, base=10000.0, scaling="plain", factor=1.0, original=0.0):
    """Radians per position of each pair, and the amplitude."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2.0))
    th = base ** (-2.0 * i / rot)
    if scaling == "linear":
        th = th / factor
    if scaling == "by_parts":
        keep = np.clip((original * th / (2 * np.pi) - 1.0) / 31.0, 0.0, 1.0)
        return th * keep + th / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    return th, 1.0


def pair_index(rot, order):
    """Columns of the first and second values of the pairs."""
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if order == "half" else (2 * i, 2 * i + 1)


def turn(x, pos, th, amp, order, back=False):
    """Rows x [..., T, H, D] turned by positions pos [T] (or broadcastable to x's leading dimensions)."""
    ia, ib = pair_index(2 * len(th), order)
    ang = np.asarray(pos, np.float64)[..., None] * th
    c, s = amp * np.cos(ang)[..., None, :], amp * np.sin(ang)[..., None, :]
    if back:
        s = -s
    y = x.copy()
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def pair_size(x, th, order):
    """|a| + |b| of the pair that each value belongs to (its own size outside the rotated part)."""
    ia, ib = pair_index(2 * len(th), order)
    y = np.abs(x)
    both = y[..., ia] + y[..., ib]
    y[..., ia] = both
    y[..., ib] = both
    return y


def norm(x, w, eps):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r * w


def norm_bwd(x, w, g, eps):
    """(dx, dw) of norm() for the gradient g of its result."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh, u = x * r, w * g
    dx = r * (u - xh * (u * xh).mean(-1, keepdims=True))
    return dx, (g * xh).reshape(-1, x.shape[-1]).sum(0)


def bf16(x):
    """Round to the nearest bf16 value, ties to even."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = ((b + 0x7fff + ((b >> 16) & 1)) >> 16) << 16
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def attention(q, k, v, seen, scale):
    """q [n, N, D] over k, v [L, Nkv, D] with seen [n, L] -> (o [n, N, D], lse [N, n], sum p|v| / sum p)."""
    n, N, D = q.shape
    G = N // k.shape[1]
    o, a, lse = np.zeros((n, N, D)), np.zeros((n, N, D)), np.full((N, n), -np.inf)
    some = seen.any(1)
    for h in range(N):
        if not some.any():
            break
        s = np.where(seen, q[:, h] @ k[:, h // G].T * scale, -np.inf)[some]
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        l = p.sum(1, keepdims=True)
        o[some, h] = p @ v[:, h // G] / l
        a[some, h] = p @ np.abs(v[:, h // G]) / l
        lse[h, some] = (m + np.log(l))[:, 0]
    return o, lse, a
