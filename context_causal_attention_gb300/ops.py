"""Python binding of the libcpattn C ABI (same names as include/cpattn.h).

Argument marshalling only: shapes and pointers are read from torch tensors,
outputs are allocated with torch when not given, and the call is enqueued on
the current torch CUDA stream, or on `stream` (a torch.cuda.Stream) where one is
given: outputs and scratch then come out of that stream's memory, and the caller
orders the streams.  All arithmetic happens in the CUDA library.
"""
import ctypes
import math

import torch

from . import _lib
from ._lib import (CP_BF16, CP_CONTIGUOUS, CP_F32, CP_GLOBAL_ORDER, CP_HEAD_TO_SEQ, CP_RANK_ORDER,
                   CP_RING_FUSED_MERGE, CP_RING_PREFETCH, CP_RING_TF32, CP_ROPE_BASE, CP_ROPE_BY_PARTS, CP_ROPE_HALF,
                   CP_ROPE_INTERLEAVED, CP_ROPE_LINEAR, CP_ROPE_PLAIN, CP_SEQ_TO_HEAD, CP_ZIGZAG, CpError, RopeStruct)

__all__ = [
    "cp_zigzag_shard", "cp_zigzag_unshard", "cp_zigzag_positions", "cp_ulysses_relayout", "cp_attn_partial",
    "cp_attn_workspace_size",
    "cp_lse_merge", "cp_ring_workspace_size", "cp_ring_attention_fwd", "cp_ring_attention_fwd_noalloc",
    "cp_allgather_attention_fwd", "cp_ulysses_attention_fwd",
    "cp_device_status", "cp_version", "cp_rope_freqs", "cp_rope_phases", "cp_rope_fwd", "cp_rope_bwd",
    "cp_qk_norm_rope_fwd", "cp_qk_norm_rope_bwd_workspace_size", "cp_qk_norm_rope_bwd", "cp_cache_append",
    "cp_prefix_attn_workspace_size", "cp_prefix_attn_fwd", "cp_cache_plan", "cp_cache_append_at", "cp_cache_keep",
    "cp_tree_plan", "cp_tree_attn_workspace_size", "cp_tree_attn_fwd", "CpCaches",
    "CP_BF16", "CP_F32", "CP_ZIGZAG", "CP_CONTIGUOUS", "CP_SEQ_TO_HEAD", "CP_HEAD_TO_SEQ", "CP_RANK_ORDER",
    "CP_GLOBAL_ORDER", "CP_RING_PREFETCH", "CP_RING_FUSED_MERGE", "CP_RING_TF32", "CP_ROPE_HALF",
    "CP_ROPE_INTERLEAVED", "CP_ROPE_PLAIN", "CP_ROPE_LINEAR", "CP_ROPE_BASE", "CP_ROPE_BY_PARTS", "CpRope", "CpError",
]

_DT = {torch.bfloat16: CP_BF16, torch.float32: CP_F32}


def _dtype_code(t):
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError("unsupported dtype %s (bf16 or fp32)" % t.dtype)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t, host_ok=False):
    """Raw pointer of a contiguous tensor.  Device tensors only, unless host_ok
    (the library then checks that host memory is pinned and mapped), so a CPU
    tensor never reaches a kernel by mistake."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    if not (t.is_cuda or host_ok):
        raise ValueError("tensor must be a CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def cp_version():
    return _lib.lib().cp_version().decode()


def _scratch(nbytes, device, stream):
    """A call's scratch on `stream`, out of that stream's memory: it goes back there when the call
    returns, so nothing but later work of the same stream is given it."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _new(shape, dtype, device, stream):
    """An output of a call on `stream`, out of that stream's memory: nothing that is still at work
    on another stream used the place before, and an output that is dropped early goes to later work
    of that stream only.  The current stream, which will read it, is waited for then too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if t.is_cuda:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def cp_zigzag_shard(x, C, layout=CP_ZIGZAG, out=None, stream=None):
    """x [B,S,N,D] -> rank-major shards [C,B,S/C,N,D] (bit-exact permutation).

    x may be a pinned host tensor: the kernel then reads it across the host
    link (copy and shard in one pass) into `out` on the current CUDA device."""
    B, S, N, D = x.shape
    if out is None:
        dev = x.device if x.is_cuda else torch.device("cuda", torch.cuda.current_device())
        out = _new((C, B, S // C, N, D), x.dtype, dev, stream)
    st = _lib.lib().cp_zigzag_shard(_ptr(x, host_ok=True), _ptr(out), B, S, N, D, C, _dtype_code(x), layout,
                                    _stream(stream))
    _lib.check("cp_zigzag_shard", st)
    return out


def cp_zigzag_unshard(x_sh, layout=CP_ZIGZAG, out=None, stream=None):
    """Rank-major shards [C,B,s,N,D] -> x [B,C*s,N,D] in global order.

    `out` may be a pinned host tensor: the kernel then writes it across the
    host link (unshard and device-to-host copy in one pass)."""
    C, B, s, N, D = x_sh.shape
    if out is None:
        out = _new((B, C * s, N, D), x_sh.dtype, x_sh.device, stream)
    st = _lib.lib().cp_zigzag_unshard(_ptr(x_sh), _ptr(out, host_ok=True), B, C * s, N, D, C, _dtype_code(x_sh),
                                      layout, _stream(stream))
    _lib.check("cp_zigzag_unshard", st)
    return out


def cp_zigzag_positions(S, C, layout=CP_ZIGZAG, device="cuda", out=None, stream=None):
    """int32 [C, S/C] global positions of every local token."""
    dev = torch.device(device)
    if out is None:
        out = _new((C, S // C), torch.int32, dev, stream)
    on_dev = 1 if out.is_cuda else 0
    st = _lib.lib().cp_zigzag_positions(_ptr(out, host_ok=True), S, C, layout, on_dev,
                                        _stream(stream) if on_dev else None)
    _lib.check("cp_zigzag_positions", st)
    return out


def cp_ulysses_relayout(x, C, direction=CP_SEQ_TO_HEAD, order=CP_RANK_ORDER, out=None, stream=None):
    """[C,B,S/C,N,D] <-> [C,B,S,N/C,D] (Ulysses all-to-all as a local permutation)."""
    if direction == CP_SEQ_TO_HEAD:
        Cx, B, s, N, D = x.shape
        S = C * s
        shape = (C, B, S, N // C, D)
    else:
        Cx, B, S, nh, D = x.shape
        N = nh * C
        shape = (C, B, S // C, N, D)
    if Cx != C:
        raise ValueError("leading dimension must be C")
    if out is None:
        out = _new(shape, x.dtype, x.device, stream)
    st = _lib.lib().cp_ulysses_relayout(_ptr(x), _ptr(out), B, S, N, D, C, _dtype_code(x), direction, order,
                                        _stream(stream))
    _lib.check("cp_ulysses_relayout", st)
    return out


def cp_attn_workspace_size(B, Sq, Sk, N, Nkv, D):
    n = ctypes.c_size_t(0)
    _lib.check("cp_attn_workspace_size", _lib.lib().cp_attn_workspace_size(B, Sq, Sk, N, Nkv, D, ctypes.byref(n)))
    return n.value


def cp_attn_partial(q, k, v, q_pos, k_pos, scale=None, o=None, lse=None, workspace=None, stream=None):
    """Partial causal attention -> (o fp32 [B,Sq,N,D], lse fp32 [B,N,Sq]).  Long
    sequences whose work plan does not fit on chip go through cp_attn_partial_ws
    with a workspace (allocated here unless given)."""
    B, Sq, N, D = q.shape
    Sk, Nkv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if o is None:
        o = _new((B, Sq, N, D), torch.float32, q.device, stream)
    if lse is None:
        lse = _new((B, N, Sq), torch.float32, q.device, stream)
    L = _lib.lib()
    need = cp_attn_workspace_size(B, Sq, Sk, N, Nkv, D)
    if need == 0 and workspace is None:
        st = L.cp_attn_partial(_ptr(q), _ptr(k), _ptr(v), _ptr(q_pos), _ptr(k_pos), B, Sq, Sk, N, Nkv, D, float(scale),
                               _ptr(o), _ptr(lse), _stream(stream))
        _lib.check("cp_attn_partial", st)
        return o, lse
    if workspace is None:
        workspace = _scratch(max(256, need), q.device, stream)
    st = L.cp_attn_partial_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(q_pos), _ptr(k_pos), B, Sq, Sk, N, Nkv, D, float(scale),
                              _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream(stream))
    _lib.check("cp_attn_partial_ws", st)
    return o, lse


def cp_attn_partial_f32(q, k, v, q_pos, k_pos, scale=None, o=None, lse=None, workspace=None, stream=None):
    """cp_attn_partial for fp32 q, k, v with the tensor cores in tf32 -> (o fp32, lse fp32)."""
    B, Sq, N, D = q.shape
    Sk, Nkv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dev = q.device
    if o is None:
        o = _new((B, Sq, N, D), torch.float32, dev, stream)
    if lse is None:
        lse = _new((B, N, Sq), torch.float32, dev, stream)
    L = _lib.lib()
    n = ctypes.c_size_t(0)
    _lib.check("cp_attn_f32_workspace_size", L.cp_attn_f32_workspace_size(B, Sq, Sk, N, Nkv, D, ctypes.byref(n)))
    if workspace is None:
        workspace = _scratch(max(256, n.value), dev, stream)
    st = L.cp_attn_partial_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(q_pos), _ptr(k_pos), B, Sq, Sk, N, Nkv, D, float(scale),
                               _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream))
    _lib.check("cp_attn_partial_f32", st)
    return o, lse


def cp_lse_merge(o_acc, lse_acc, o_tile, lse_tile, stream=None):
    """In-place merge of (o_tile, lse_tile) into (o_acc, lse_acc)."""
    B, Sq, N, D = o_acc.shape
    st = _lib.lib().cp_lse_merge(_ptr(o_acc), _ptr(lse_acc), _ptr(o_tile), _ptr(lse_tile), B, Sq, N, D,
                                 _stream(stream))
    _lib.check("cp_lse_merge", st)
    return o_acc, lse_acc


def _ring_flags(prefetch, fused_merge, tf32=False):
    return ((CP_RING_PREFETCH if prefetch else 0) | (CP_RING_FUSED_MERGE if fused_merge else 0) |
            (CP_RING_TF32 if tf32 else 0))


def cp_ring_workspace_size(B, S, N, Nkv, D, C, prefetch=0, o_dtype=CP_F32, fused_merge=False, tf32=False):
    n = ctypes.c_size_t(0)
    st = _lib.lib().cp_ring_workspace_size(B, S, N, Nkv, D, C, _ring_flags(prefetch, fused_merge, tf32), o_dtype,
                                           ctypes.byref(n))
    _lib.check("cp_ring_workspace_size", st)
    return n.value


def cp_ring_attention_fwd(q_sh, k_sh, v_sh, pos, scale=None, layout=CP_ZIGZAG, prefetch=0, o_dtype=CP_F32,
                          workspace=None, o=None, lse=None, events=None, stream=None, fused_merge=False, tf32=False):
    """Ring attention forward over C resident virtual ranks.

    Returns (o_sh [C,B,s,N,D] of o_dtype, lse_sh fp32 [C,B,N,s]).  `events`, if
    given, is a list of >= 4*C recorded torch.cuda.Event objects (see the C
    header for their meaning).  tf32: fp32 shards, tensor cores in tf32."""
    C, B, s, N, D = q_sh.shape
    Nkv = k_sh.shape[3]
    S = C * s
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dev = q_sh.device
    if o is None:
        o = _new((C, B, s, N, D), torch.float32 if o_dtype == CP_F32 else torch.bfloat16, dev, stream)
    if lse is None:
        lse = _new((C, B, N, s), torch.float32, dev, stream)
    need = cp_ring_workspace_size(B, S, N, Nkv, D, C, prefetch, o_dtype, fused_merge, tf32)
    if workspace is None:
        workspace = _scratch(max(need, 256), dev, stream)
    L = _lib.lib()
    args = [_ptr(q_sh), _ptr(k_sh), _ptr(v_sh), _ptr(pos), B, S, N, Nkv, D, C, float(scale), layout,
            _ring_flags(prefetch, fused_merge, tf32),
            _ptr(o), o_dtype, _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(stream)]
    if events is None:
        st = L.cp_ring_attention_fwd(*args)
        _lib.check("cp_ring_attention_fwd", st)
    else:
        arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
        st = L.cp_ring_attention_fwd_traced(*args, arr, len(events))
        _lib.check("cp_ring_attention_fwd_traced", st)
    return o, lse


def cp_allgather_attention_fwd(q_sh, k_sh, v_sh, pos, scale=None, layout=CP_ZIGZAG, workspace=None, o=None,
                               lse=None, stream=None):
    """All-gather CP forward over C resident virtual ranks -> (o_sh fp32, lse_sh fp32)."""
    C, B, s, N, D = q_sh.shape
    Nkv = k_sh.shape[3]
    S = C * s
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dev = q_sh.device
    if o is None:
        o = _new((C, B, s, N, D), torch.float32, dev, stream)
    if lse is None:
        lse = _new((C, B, N, s), torch.float32, dev, stream)
    L = _lib.lib()
    n = ctypes.c_size_t(0)
    _lib.check("cp_allgather_workspace_size", L.cp_allgather_workspace_size(B, S, N, Nkv, D, C, ctypes.byref(n)))
    if workspace is None:
        workspace = _scratch(max(256, n.value), dev, stream)
    st = L.cp_allgather_attention_fwd(_ptr(q_sh), _ptr(k_sh), _ptr(v_sh), _ptr(pos), B, S, N, Nkv, D, C,
                                      float(scale), layout, _ptr(o), _ptr(lse), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream))
    _lib.check("cp_allgather_attention_fwd", st)
    return o, lse


def cp_ulysses_attention_fwd(q_sh, k_sh, v_sh, scale=None, layout=CP_ZIGZAG, workspace=None, o=None, lse=None,
                             stream=None):
    """Ulysses (all-to-all) CP forward -> (o_sh fp32 [C,B,s,N,D], lse_h fp32 [C,B,N/C,S])."""
    C, B, s, N, D = q_sh.shape
    Nkv = k_sh.shape[3]
    S = C * s
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dev = q_sh.device
    if o is None:
        o = _new((C, B, s, N, D), torch.float32, dev, stream)
    if lse is None:
        lse = _new((C, B, N // C, S), torch.float32, dev, stream)
    L = _lib.lib()
    n = ctypes.c_size_t(0)
    _lib.check("cp_ulysses_workspace_size", L.cp_ulysses_workspace_size(B, S, N, Nkv, D, C, ctypes.byref(n)))
    if workspace is None:
        workspace = _scratch(max(256, n.value), dev, stream)
    st = L.cp_ulysses_attention_fwd(_ptr(q_sh), _ptr(k_sh), _ptr(v_sh), B, S, N, Nkv, D, C, float(scale), layout,
                                    _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    _lib.check("cp_ulysses_attention_fwd", st)
    return o, lse


def cp_mesh_workspace_size(B, S, N, Nkv, D, A, R, prefetch=0, fused_merge=False):
    n = ctypes.c_size_t(0)
    st = _lib.lib().cp_mesh_workspace_size(B, S, N, Nkv, D, A, R, _ring_flags(prefetch, fused_merge), ctypes.byref(n))
    _lib.check("cp_mesh_workspace_size", st)
    return n.value


def cp_mesh_attention_fwd(q_sh, k_sh, v_sh, pos, A, R, scale=None, layout=CP_ZIGZAG, prefetch=0, fused_merge=False,
                          workspace=None, o=None, lse=None, stream=None):
    """A2A x P2P mesh CP forward over C = A*R resident virtual ranks.

    Returns (o_sh fp32 [C,B,s,N,D], lse_h fp32 [R,A,B,N/A,S/R])."""
    C, B, s, N, D = q_sh.shape
    Nkv = k_sh.shape[3]
    if A * R != C:
        raise ValueError("cp_mesh_attention_fwd: A*R must equal the number of shards")
    S = C * s
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dev = q_sh.device
    if o is None:
        o = _new((C, B, s, N, D), torch.float32, dev, stream)
    if lse is None:
        lse = _new((R, A, B, N // A, S // R), torch.float32, dev, stream)
    need = cp_mesh_workspace_size(B, S, N, Nkv, D, A, R, prefetch, fused_merge)
    if workspace is None:
        workspace = _scratch(max(256, need), dev, stream)
    st = _lib.lib().cp_mesh_attention_fwd(_ptr(q_sh), _ptr(k_sh), _ptr(v_sh), _ptr(pos), B, S, N, Nkv, D, A, R,
                                          float(scale), layout, _ring_flags(prefetch, fused_merge), _ptr(o),
                                          _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                          _stream(stream))
    _lib.check("cp_mesh_attention_fwd", st)
    return o, lse


def cp_attn_bwd_partial(q, k, v, o, dout, lse, q_pos, k_pos, scale=None, dq=None, dk=None, dv=None, accumulate=False,
                        workspace=None, stream=None):
    """Tile backward -> (dq fp32 [B,Sq,N,D], dk, dv fp32 [B,Sk,Nkv,D]) from the
    final output o (fp32) and lse; q, k, v, dout bf16."""
    B, Sq, N, D = q.shape
    Sk, Nkv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dev = q.device
    dq = _new((B, Sq, N, D), torch.float32, dev, stream) if dq is None else dq
    dk = _new((B, Sk, Nkv, D), torch.float32, dev, stream) if dk is None else dk
    dv = _new((B, Sk, Nkv, D), torch.float32, dev, stream) if dv is None else dv
    L = _lib.lib()
    n = ctypes.c_size_t(0)
    _lib.check("cp_attn_bwd_workspace_size", L.cp_attn_bwd_workspace_size(B, Sq, Sk, N, ctypes.byref(n)))
    if workspace is None:
        workspace = _scratch(max(256, n.value), dev, stream)
    st = L.cp_attn_bwd_partial(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(q_pos), _ptr(k_pos), B,
                               Sq, Sk, N, Nkv, D, float(scale), _ptr(dq), _ptr(dk), _ptr(dv), 1 if accumulate else 0,
                               _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _lib.check("cp_attn_bwd_partial", st)
    return dq, dk, dv


def cp_ring_bwd_workspace_size(B, S, N, C):
    n = ctypes.c_size_t(0)
    _lib.check("cp_ring_bwd_workspace_size", _lib.lib().cp_ring_bwd_workspace_size(B, S, N, C, ctypes.byref(n)))
    return n.value


def cp_ring_attention_bwd(q_sh, k_sh, v_sh, o_sh, lse_sh, do_sh, pos, scale=None, layout=CP_ZIGZAG, workspace=None,
                          dq=None, dk=None, dv=None, stream=None):
    """Ring backward over C resident virtual ranks -> (dq_sh, dk_sh, dv_sh) fp32, rank-major."""
    C, B, s, N, D = q_sh.shape
    Nkv = k_sh.shape[3]
    S = C * s
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dev = q_sh.device
    dq = _new((C, B, s, N, D), torch.float32, dev, stream) if dq is None else dq
    dk = _new((C, B, s, Nkv, D), torch.float32, dev, stream) if dk is None else dk
    dv = _new((C, B, s, Nkv, D), torch.float32, dev, stream) if dv is None else dv
    if workspace is None:
        workspace = _scratch(max(256, cp_ring_bwd_workspace_size(B, S, N, C)), dev, stream)
    st = _lib.lib().cp_ring_attention_bwd(_ptr(q_sh), _ptr(k_sh), _ptr(v_sh), _ptr(o_sh), _ptr(lse_sh), _ptr(do_sh),
                                          _ptr(pos), B, S, N, Nkv, D, C, float(scale), layout, _ptr(dq), _ptr(dk),
                                          _ptr(dv), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                          _stream(stream))
    _lib.check("cp_ring_attention_bwd", st)
    return dq, dk, dv


def cp_ring_attention_fwd_noalloc(q_sh, k_sh, v_sh, pos, o, lse, scale=None, layout=CP_ZIGZAG, o_dtype=CP_F32,
                                  stream=None):
    """Ring forward that allocates nothing: for callers that may not call
    cudaMalloc (or cannot pass a workspace).  Its scratch is a fixed-size array
    inside the library (CP_NOALLOC_SCRATCH_BYTES); outputs o and lse must be
    given.  Calls on one device share that array: do not overlap them."""
    C, B, s, N, D = q_sh.shape
    Nkv = k_sh.shape[3]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    st = _lib.lib().cp_ring_attention_fwd_noalloc(_ptr(q_sh), _ptr(k_sh), _ptr(v_sh), _ptr(pos), B, C * s, N, Nkv,
                                                  D, C, float(scale), layout, _ptr(o), o_dtype, _ptr(lse),
                                                  _stream(stream))
    _lib.check("cp_ring_attention_fwd_noalloc", st)
    return o, lse


class CpRope:
    """A rotation (cp_rope of the C header): frequencies on the device, rotated
    part, order of the pairs, amplitude.  Made by cp_rope_freqs or
    cp_rope_phases and kept by the caller; another rotation is another object."""

    def __init__(self, freqs, rot_dim, order, amplitude):
        if freqs.dtype != torch.int64 or not freqs.is_contiguous() or 2 * freqs.numel() < rot_dim:
            raise ValueError("freqs must be contiguous int64 [rot_dim / 2]")
        self._freqs, self._rest = freqs, (rot_dim, order, amplitude)
        self._struct = RopeStruct(freqs.data_ptr(), rot_dim, order, amplitude)
        self._ref, self._at = ctypes.byref(self._struct), ctypes.addressof(self._struct)

    # read only: calls use the struct above
    freqs = property(lambda self: self._freqs)
    rot_dim = property(lambda self: self._rest[0])
    order = property(lambda self: self._rest[1])
    amplitude = property(lambda self: self._rest[2])


def cp_rope_freqs(rot_dim, base=10000.0, scaling=CP_ROPE_PLAIN, factor=1.0, original_len=0, order=CP_ROPE_HALF,
                  device="cuda"):
    """Frequencies base^(-2i/rot_dim) under one of the header's scalings -> CpRope on `device`."""
    f = torch.empty(max(rot_dim // 2, 1), dtype=torch.int64)
    amp = ctypes.c_float(0.0)
    _lib.check("cp_rope_freqs", _lib.lib().cp_rope_freqs(rot_dim, base, scaling, factor, original_len, f.data_ptr(),
                                                         ctypes.byref(amp)))
    return CpRope(f.to(device), rot_dim, order, amp.value)


def cp_rope_phases(inv_freq, amplitude=1.0, order=CP_ROPE_HALF, device="cuda"):
    """Any other frequencies, in radians per position -> CpRope on `device`."""
    w = torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu").contiguous()
    f = torch.empty(w.numel(), dtype=torch.int64)
    _lib.check("cp_rope_phases", _lib.lib().cp_rope_phases(w.data_ptr(), w.numel(), f.data_ptr()))
    return CpRope(f.to(device), 2 * w.numel(), order, amplitude)


def _here(*ts):
    """Every given tensor lies on the current CUDA device, which is returned."""
    dev = torch.cuda.current_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensor must be on the current CUDA device")
    return dev


def _raw_stream(stream, dev):
    """Handle of `stream`, or of the device's current stream (without making a Stream object: these
    calls are short)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _head_rows(t):
    """(elements between tokens, tokens' leading shape, heads, D) of [..., heads, D] whose
    head rows are dense and whose tokens lie at one distance from one another."""
    shape = t.shape
    n = len(shape)
    if n < 3:
        raise ValueError("expected [..., heads, D] with at least one leading dimension")
    H, D = shape[-2], shape[-1]
    if t.is_contiguous():
        return H * D, shape[:-2], H, D
    st = t.stride()
    if (D > 1 and st[-1] != 1) or (H > 1 and st[-2] != D):
        raise ValueError("the head rows of a token must be dense")
    step, count = 0, 1
    for i in range(n - 3, -1, -1):
        if shape[i] > 1:
            if count == 1:
                step = st[i]
            # (an expanded dimension repeats its tokens: no distance at all)
            if st[i] != step * count or step == 0:
                raise ValueError("tokens must lie at one distance from one another")
            count *= shape[i]
    return (step if count > 1 else H * D), shape[:-2], H, D


def _tokens(lead):
    """(C, B, s) of leading dimensions [C, B, s], [B, s] or [s]."""
    if len(lead) > 3:
        raise ValueError("expected [C, B, s, heads, D], [B, s, heads, D] or [s, heads, D]")
    return (1, 1, 1)[:3 - len(lead)] + tuple(lead)


def _qk(q, k):
    """Common description of q and k (k may be None): (C, B, s, N, Nkv, D, q stride, k stride)."""
    qs, lead, N, D = _head_rows(q)
    ks, Nkv = 0, 0
    if k is not None:
        ks, lead_k, Nkv, Dk = _head_rows(k)
        if lead_k != lead or Dk != D or k.dtype != q.dtype:
            raise ValueError("q and k must have the same tokens, head size and dtype")
    C, B, s = _tokens(lead)
    return C, B, s, N, Nkv, D, qs, ks


def _check_pos(pos, C, s):
    if pos is not None and (pos.dtype != torch.int32 or pos.numel() != C * s or not pos.is_contiguous()):
        raise ValueError("pos must be contiguous int32 [C, s]")


def _row_out(out, x, stream):
    """An output of x's rows: a new dense one, x itself (in place), or a dense one that was given."""
    if x is None:
        return None
    if out is None:
        return _new(x.shape, x.dtype, x.device, stream)
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("an output must have its input's shape and dtype")
    if out.data_ptr() == x.data_ptr():
        if out.stride() != x.stride():
            raise ValueError("an output in place must have its input's strides")
    elif not out.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return out


def _addr(t):
    return None if t is None else t.data_ptr()


def _rope_call(name, q, k, pos, rope, q_out, k_out, stream):
    C, B, s, N, Nkv, D, qs, ks = _qk(q, k)
    _check_pos(pos, C, s)
    q_out, k_out = _row_out(q_out, q, stream), _row_out(k_out, k, stream)
    dev = _here(q, k, pos, None if rope is None else rope.freqs, q_out, k_out)
    st = getattr(_lib.lib(), name)(_addr(q), _addr(k), _addr(pos), C, B, s, N, Nkv, D, qs, ks, _dtype_code(q),
                                   None if rope is None else rope._ref, _addr(q_out), _addr(k_out), _raw_stream(stream, dev))
    _lib.check(name, st)
    return q_out, k_out


def cp_rope_fwd(q, k, pos, rope, q_out=None, k_out=None, stream=None):
    """Rotate q [C,B,s,N,D] and k [C,B,s,Nkv,D] (or [B,s,..], [s,..]; k may be None) by
    their tokens' positions pos [C,s] -> (q_out, k_out).  Rows may be strided
    (slices of a fused projection); outputs dense, or the inputs themselves."""
    return _rope_call("cp_rope_fwd", q, k, pos, rope, q_out, k_out, stream)


def cp_rope_bwd(dq_out, dk_out, pos, rope, dq=None, dk=None, stream=None):
    """Gradients of cp_rope_fwd's inputs from those of its outputs -> (dq, dk)."""
    return _rope_call("cp_rope_bwd", dq_out, dk_out, pos, rope, dq, dk, stream)


def _check_weights(wq, wk, D):
    for w in (wq, wk):
        if w is not None and (w.numel() != D or not w.is_contiguous()):
            raise ValueError("norm weights must be contiguous [D]")
    if wq is not None and wk is not None and wq.dtype != wk.dtype:
        raise ValueError("wq and wk must have the same dtype")
    w = wq if wq is not None else wk
    return CP_F32 if w is None else _dtype_code(w)


def cp_qk_norm_rope_fwd(q, k, wq, wk, pos, rope, eps=1e-6, q_out=None, k_out=None, stream=None):
    """Root-mean-square norm of every head row of q and k with weights wq, wk
    [D], then the rotation of cp_rope_fwd (rope None: norm alone) -> (q_out, k_out)."""
    C, B, s, N, Nkv, D, qs, ks = _qk(q, k)
    if rope is not None:
        _check_pos(pos, C, s)
    wd = _check_weights(wq, wk, D)
    q_out, k_out = _row_out(q_out, q, stream), _row_out(k_out, k, stream)
    dev = _here(q, k, wq, wk, pos, None if rope is None else rope.freqs, q_out, k_out)
    st = _lib.lib().cp_qk_norm_rope_fwd(_addr(q), _addr(k), _addr(wq), _addr(wk), _addr(pos), C, B, s, N, Nkv, D, qs,
                                        ks, _dtype_code(q), wd, eps, None if rope is None else rope._ref,
                                        _addr(q_out), _addr(k_out), _raw_stream(stream, dev))
    _lib.check("cp_qk_norm_rope_fwd", st)
    return q_out, k_out


def cp_qk_norm_rope_bwd_workspace_size(C, B, s, N, Nkv, D):
    n = ctypes.c_size_t(0)
    _lib.check("cp_qk_norm_rope_bwd_workspace_size",
               _lib.lib().cp_qk_norm_rope_bwd_workspace_size(C, B, s, N, Nkv, D, ctypes.byref(n)))
    return n.value


def cp_qk_norm_rope_bwd(dq_out, dk_out, q, k, wq, wk, pos, rope, eps=1e-6, dq=None, dk=None, dwq=None, dwk=None,
                        workspace=None, stream=None):
    """Gradients of cp_qk_norm_rope_fwd -> (dq, dk, dwq fp32 [D], dwk fp32 [D])
    from the dense gradients of its outputs and its inputs."""
    C, B, s, N, Nkv, D, qs, ks = _qk(q, k)
    if rope is not None:
        _check_pos(pos, C, s)
    wd = _check_weights(wq, wk, D)
    for g, x in ((dq_out, q), (dk_out, k)):
        if (g is None) != (x is None) or (g is not None and (g.shape != x.shape or g.dtype != x.dtype or
                                                             not g.is_contiguous())):
            raise ValueError("the gradients must be dense, of the inputs' shapes and dtype")
    dq = dq_out if dq is dq_out else _row_out(dq, q, stream)
    dk = dk_out if dk is dk_out else _row_out(dk, k, stream)
    if dwq is None:
        dwq = _new(D, torch.float32, q.device, stream)
    if dwk is None and k is not None:
        dwk = _new(D, torch.float32, q.device, stream)
    for w in (dwq, dwk):
        if w is not None and (w.dtype != torch.float32 or w.numel() != D or not w.is_contiguous()):
            raise ValueError("weight gradients must be contiguous fp32 [D]")
    if workspace is None:
        workspace = _scratch(max(256, cp_qk_norm_rope_bwd_workspace_size(C, B, s, N, Nkv, D)), q.device, stream)
    dev = _here(dq_out, dk_out, q, k, wq, wk, pos, None if rope is None else rope.freqs, dq, dk, dwq, dwk, workspace)
    st = _lib.lib().cp_qk_norm_rope_bwd(_addr(dq_out), _addr(dk_out), _addr(q), _addr(k), _addr(wq), _addr(wk),
                                        _addr(pos), C, B, s, N, Nkv, D, qs, ks, _dtype_code(q), wd, eps,
                                        None if rope is None else rope._ref, _addr(dq), _addr(dk), _addr(dwq),
                                        _addr(dwk), _addr(workspace), workspace.numel() * workspace.element_size(),
                                        _raw_stream(stream, dev))
    _lib.check("cp_qk_norm_rope_bwd", st)
    return dq, dk, dwq, dwk


def _check_cache(k_cache, v_cache, table, cu_new, kv_len):
    """(n_pages, page_size, Nkv, D, B, max_pages) of a paged cache and its lists."""
    shape, tab = k_cache.shape, table.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("the caches must be [n_pages, page_size, Nkv, D], both alike")
    if k_cache.dtype is not torch.bfloat16 or v_cache.dtype is not torch.bfloat16:
        raise TypeError("the caches must be bf16")
    if len(tab) != 2 or kv_len.shape != (tab[0],) or cu_new.shape != (tab[0] + 1,):
        raise ValueError("table [B, max_pages], cu_new [B + 1] and kv_len [B] must agree")
    if not (table.dtype is cu_new.dtype is kv_len.dtype is torch.int32):
        raise TypeError("table, cu_new and kv_len must be int32")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous() and table.is_contiguous() and
            cu_new.is_contiguous() and kv_len.is_contiguous()):
        raise ValueError("tensor must be contiguous")
    return (*shape, *tab)


def cp_cache_append(k, v, k_cache, v_cache, table, cu_new, kv_len, rope=None, q=None, q_out=None, wq=None, wk=None,
                    eps=1e-6, pos_base=0, stream=None):
    """Append the new tokens' k, v [R,Nkv,D] to the pages of their sequences,
    k normed (wk) and rotated (rope) on the way; q [R,N,D], if given, likewise into
    q_out bf16 [R,N,D].  kv_len counts each sequence's tokens after the call.
    Returns q_out (None without q)."""
    n_pages, page, Nkv, D, B, max_pages = _check_cache(k_cache, v_cache, table, cu_new, kv_len)
    shape, dtype = k.shape, k.dtype
    if len(shape) != 3 or v.shape != shape or shape[1] != Nkv or shape[2] != D or v.dtype is not dtype:
        raise ValueError("k and v must be [R, Nkv, D] of the cache's heads, of one dtype")
    ks, vs = _head_rows(k)[0], _head_rows(v)[0]
    R, qs, N = shape[0], 0, 0
    if q is not None:
        qs, lead, N, Dq = _head_rows(q)
        if lead != shape[:1] or Dq != D or q.dtype is not dtype:
            raise ValueError("q must be [R, N, D] of k's tokens and dtype")
        if q_out is None:
            q_out = _new((R, N, D), torch.bfloat16, q.device, stream)
        elif q_out.shape != q.shape or q_out.dtype != torch.bfloat16 or not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous bf16 [R, N, D]")
    elif q_out is not None:
        raise ValueError("q_out without q")
    wd = _check_weights(wq, wk, D)
    dev = _here(q, k, v, k_cache, v_cache, table, cu_new, kv_len, wq, wk, None if rope is None else rope.freqs, q_out)
    st = _lib.lib().cp_cache_append(_addr(q), _addr(k), _addr(v), qs, ks, vs, _dtype_code(k), R, N, Nkv, D, _addr(wq),
                                    _addr(wk), wd, eps, None if rope is None else rope._ref, pos_base, _addr(k_cache),
                                    _addr(v_cache), n_pages, page, _addr(table), B, max_pages, _addr(cu_new),
                                    _addr(kv_len), _addr(q_out), _raw_stream(stream, dev))
    _lib.check("cp_cache_append", st)
    return q_out


_I32 = torch.int32


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def cp_cache_plan(kv_had, kv_keep, n_new, table, free_pages, n_free, page_size, R, pos_base=0, kv_len=None, cu_new=None,
                  slots=None, pos=None, n_free_out=None, stream=None):
    """Pages and slots of a step from the sequences' lengths (see the C header): page numbers go between
    table [B,max_pages] and the stack free_pages [n_pages].  Returns (kv_len [B], cu_new [B+1], slots [R],
    pos [R], n_free_out [2]), all int32."""
    if kv_len is None:
        kv_len = _new(table.shape[0], _I32, table.device, stream)
    if cu_new is None:
        cu_new = _new(table.shape[0] + 1, _I32, table.device, stream)
    if slots is None:
        slots = _new(R, _I32, table.device, stream)
    if pos is None:
        pos = _new(R, _I32, table.device, stream)
    if n_free_out is None:
        n_free_out = _new(2, _I32, table.device, stream)
    st = _lib.bind().cache_plan(table, free_pages, kv_had, kv_keep, n_new, n_free, page_size, R, pos_base, kv_len, cu_new,
                                slots, pos, n_free_out, _handle(stream))
    if st:
        _lib.check("cp_cache_plan", st)
    return kv_len, cu_new, slots, pos, n_free_out


def cp_cache_append_at(k, v, k_cache, v_cache, slots, pos, rope=None, q=None, q_out=None, wq=None, wk=None, eps=1e-6,
                       stream=None):
    """cp_cache_append with the rows' slots and positions, int32 [R] each (slot -1: the row is skipped).
    Returns q_out (None without q)."""
    if q is not None and q_out is None:
        q_out = _new(q.shape, torch.bfloat16, q.device, stream)
    at, freqs = (0, None) if rope is None else (rope._at, rope._freqs)
    st = _lib.bind().cache_append_at(k, v, k_cache, v_cache, slots, pos, at, freqs, q, q_out, wq, wk, eps, _handle(stream))
    if st:
        _lib.check("cp_cache_append_at", st)
    return q_out


class CpCaches:
    """The caches of all layers (K and V of each, in any order), for cp_cache_keep: bf16
    [n_pages, page_size, Nkv, D] each, all alike.  Made once and kept by the caller."""

    def __init__(self, caches):
        caches = tuple(caches)
        if not caches or len(caches[0].shape) != 4:
            raise ValueError("expected caches [n_pages, page_size, Nkv, D]")
        for c in caches:
            if c.dtype is not torch.bfloat16:
                raise TypeError("the caches must be bf16")
            if c.shape != caches[0].shape or c.device != caches[0].device or not c.is_contiguous():
                raise ValueError("the caches must be contiguous, all alike, on one device")
        self._caches = caches
        self._ptrs = (ctypes.c_void_p * len(caches))(*[c.data_ptr() for c in caches])
        self._words = (caches[0], ctypes.addressof(self._ptrs), len(caches), *caches[0].shape)

    # read only: calls use the addresses above
    caches = property(lambda self: self._caches)


def cp_cache_keep(caches, table, cu_new, kv_len, kept, n_kept, R=None, kv_keep=None, stream=None):
    """Move the accepted tokens kept [B,max_kept] (n_kept [B] of each sequence; below zero: all stay) of the step's
    new tokens together, in every one of `caches` (a CpCaches, or a list of tensors); R: the step's rows.
    Returns kv_keep int32 [B], the tokens that stay."""
    if not isinstance(caches, CpCaches):
        caches = CpCaches(caches)
    if kv_keep is None:
        kv_keep = _new(table.shape[0], _I32, table.device, stream)
    st = _lib.bind().cache_keep(*caches._words, table, cu_new, kv_len, (1 << 30) - 1 if R is None else R, kept, n_kept,
                                kv_keep, _handle(stream))
    if st:
        _lib.check("cp_cache_keep", st)
    return kv_keep


def cp_tree_plan(parent, cu_new, kv_len, words, pos_base=0, mask=None, pos=None, stream=None):
    """Ancestors and positions of drafted trees from each row's parent [R] among its sequence's new tokens (-1: it
    follows the cached ones) -> (mask int32 [R,words], pos int32 [R]); see the C header."""
    if mask is None:
        mask = _new((parent.shape[0], words), _I32, parent.device, stream)
    if pos is None:
        pos = _new(parent.shape[0], _I32, parent.device, stream)
    st = _lib.bind().tree_plan(parent, kv_len, cu_new, words, pos_base, mask, pos, _handle(stream))
    if st:
        _lib.check("cp_tree_plan", st)
    return mask, pos


def cp_prefix_attn_workspace_size(R, B, max_new, prefix_len, N, Nkv, D, page_size, max_pages):
    n = ctypes.c_size_t(0)
    _lib.check("cp_prefix_attn_workspace_size",
               _lib.lib().cp_prefix_attn_workspace_size(R, B, max_new, prefix_len, N, Nkv, D, page_size, max_pages,
                                                        ctypes.byref(n)))
    return n.value


def cp_tree_attn_workspace_size(R, B, max_new, words, prefix_len, N, Nkv, D, page_size, max_pages):
    n = ctypes.c_size_t(0)
    _lib.check("cp_tree_attn_workspace_size",
               _lib.lib().cp_tree_attn_workspace_size(R, B, max_new, words, prefix_len, N, Nkv, D, page_size, max_pages,
                                                      ctypes.byref(n)))
    return n.value


def _prefix_call(name, more, q, k_cache, v_cache, prefix_pages, prefix_len, table, cu_new, kv_len, max_new, scale,
                 o_dtype, o, lse, workspace, stream, mask=None):
    """A call of the shared-prefix attention, or with `mask` of the tree attention, through ctypes."""
    n_pages, page, Nkv, D, B, max_pages = _check_cache(k_cache, v_cache, table, cu_new, kv_len)
    if q.dim() != 3 or q.shape[2] != D or q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [R, N, D]")
    R, N = q.shape[0], q.shape[1]
    if mask is not None and (mask.dim() != 2 or mask.dtype != torch.int32 or mask.shape[0] != R or
                             not mask.is_contiguous()):
        raise ValueError("mask must be contiguous int32 [R, words]")
    masked = () if mask is None else (_addr(mask), mask.shape[1])
    # (a list that is missing is the library's to refuse)
    if prefix_len and prefix_pages is not None and (prefix_pages.dtype != torch.int32 or
                                                    not prefix_pages.is_contiguous() or
                                                    prefix_pages.numel() * page < prefix_len):
        raise ValueError("prefix_pages must be contiguous int32 and cover prefix_len tokens")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if o is None:
        o = _new((R, N, D), torch.float32 if o_dtype == CP_F32 else torch.bfloat16, q.device, stream)
    elif o.shape != q.shape or not o.is_contiguous():
        raise ValueError("o must be contiguous [R, N, D]")
    if lse is None:
        lse = _new((N, R), torch.float32, q.device, stream)
    elif lse.shape != (N, R) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [N, R]")
    if workspace is None:
        workspace = _scratch(max(256, cp_prefix_attn_workspace_size(R, B, max_new, prefix_len, N, Nkv, D, page,
                                                                    max_pages)), q.device, stream)
    dev = _here(q, k_cache, v_cache, prefix_pages, table, cu_new, kv_len, mask, o, lse, workspace)
    st = getattr(_lib.lib(), name)(_addr(q), _addr(k_cache), _addr(v_cache), n_pages, page, _addr(prefix_pages),
                                   prefix_len, _addr(table), B, max_pages, _addr(cu_new), _addr(kv_len), *masked,
                                   max_new, R, N, Nkv, D, scale, _addr(o), _dtype_code(o), _addr(lse), _addr(workspace),
                                   workspace.numel() * workspace.element_size(), *more, _raw_stream(stream, dev))
    _lib.check(name, st)
    return o, lse


def cp_prefix_attn_fwd(q, k_cache, v_cache, prefix_pages, prefix_len, table, cu_new, kv_len, max_new, scale=None,
                       o_dtype=CP_BF16, o=None, lse=None, workspace=None, stream=None):
    """Attention of the new tokens q bf16 [R,N,D] over the shared prefix and their own sequences'
    pages -> (o [R,N,D], lse fp32 [N,R]); see the C header.  max_new: the
    largest number of new tokens of a sequence (chooses the tiles only)."""
    return _prefix_call("cp_prefix_attn_fwd", (), q, k_cache, v_cache, prefix_pages, prefix_len, table, cu_new, kv_len,
                        max_new, scale, o_dtype, o, lse, workspace, stream)


def cp_tree_attn_fwd(q, k_cache, v_cache, mask, prefix_pages, prefix_len, table, cu_new, kv_len, max_new, scale=None,
                     o_dtype=CP_BF16, o=None, lse=None, workspace=None, stream=None):
    """cp_prefix_attn_fwd for drafted trees: of its sequence's new tokens a row sees those whose bits its row of
    mask int32 [R,words] has (cp_tree_plan) -> (o [R,N,D], lse fp32 [N,R])."""
    R, N, D = q.shape
    if o is None:
        o = _new((R, N, D), torch.float32 if o_dtype == CP_F32 else torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _new((N, R), torch.float32, q.device, stream)
    if workspace is None:
        if mask is None or mask.dim() != 2 or k_cache.dim() != 4 or table.dim() != 2:
            raise ValueError("expected mask [R, words], caches [n_pages, page_size, Nkv, D] and table [B, max_pages]")
        B, max_pages = table.shape
        workspace = _scratch(max(256, cp_tree_attn_workspace_size(R, B, max_new, mask.shape[1], prefix_len, N,
                                                                  k_cache.shape[2], D, k_cache.shape[1], max_pages)),
                             q.device, stream)
    st = _lib.bind().tree_attn_fwd(q, k_cache, v_cache, mask, prefix_pages, prefix_len, table, cu_new, kv_len, max_new,
                                   D ** -0.5 if scale is None else scale, o, lse, workspace, _handle(stream))
    if st:
        _lib.check("cp_tree_attn_fwd", st)
    return o, lse


def cp_selftest_stalled_prefix_attn(timeout_ns, q, k_cache, v_cache, prefix_pages, prefix_len, table, cu_new, kv_len,
                                    max_new, workspace=None, stream=None):
    """The self-test of the shared-prefix attention's bounded waits: a call whose loads are held on a word
    that nothing sets (see the C header); read the outcome with cp_device_status."""
    _prefix_call("cp_selftest_stalled_prefix_attn", (int(timeout_ns),), q, k_cache, v_cache, prefix_pages, prefix_len,
                 table, cu_new, kv_len, max_new, None, CP_BF16, None, None, workspace, stream)


def cp_selftest_stalled_tree_attn(timeout_ns, q, k_cache, v_cache, mask, prefix_pages, prefix_len, table, cu_new, kv_len,
                                  max_new, workspace=None, stream=None):
    """The same of the tree attention, with the kernels that cp_tree_attn_fwd takes for these arguments."""
    if mask is None:
        raise ValueError("mask must be contiguous int32 [R, words]")
    _prefix_call("cp_selftest_stalled_tree_attn", (int(timeout_ns),), q, k_cache, v_cache, prefix_pages, prefix_len,
                 table, cu_new, kv_len, max_new, None, CP_BF16, None, None, workspace, stream, mask)


def cp_selftest_stalled_producer(q, k, v, pos, o, lse, timeout_ns, stream=None):
    """Failure-detection self-test: the attention kernel with its producer held
    on a flag nothing sets; its bounded waits give up after timeout_ns and the
    device status becomes CP_ERR_DEVICE_TIMEOUT (read it with cp_device_status)."""
    st = _lib.lib().cp_selftest_stalled_producer(_ptr(q), _ptr(k), _ptr(v), _ptr(pos), _ptr(o), _ptr(lse),
                                                 int(timeout_ns), _stream(stream))
    _lib.check("cp_selftest_stalled_producer", st)


CP_SELFTEST_SCRATCH_BYTES = 512 << 10


def cp_selftest_stalled_kernel(kernel, timeout_ns, scratch=None, device="cuda", stream=None):
    """The same self-test for kernel 0 (bf16 forward), 1 (tf32 forward) or 2
    (backward: its dK/dV and dQ launches), on a tiny problem laid out in
    `scratch` (allocated here unless given)."""
    if scratch is None:
        scratch = _scratch(CP_SELFTEST_SCRATCH_BYTES, device, stream)
    st = _lib.lib().cp_selftest_stalled_kernel(int(kernel), _ptr(scratch), scratch.numel() * scratch.element_size(),
                                               int(timeout_ns), _stream(stream))
    _lib.check("cp_selftest_stalled_kernel", st)


def cp_device_status(clear=True, stream=None):
    """Synchronise the stream and return the library's device status code."""
    code = ctypes.c_int(0)
    st = _lib.lib().cp_device_status(ctypes.byref(code), 1 if clear else 0, _stream(stream))
    _lib.check("cp_device_status", st)
    return code.value
