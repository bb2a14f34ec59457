"""Operators on the tokens of voxelized frames: argument marshalling only.

A batch of frames (:func:`voxelize_batch`) is a ragged sequence of tokens, one
row per voxel, frame b the rows ``offsets[b]:offsets[b + 1]``; ``offsets`` is a
host sequence of ints, as ``frame_offsets`` of the voxelizer is.  The work is
done by libpv.so (``include/pv.h``, "Operators on voxel tokens"); this file
checks dtypes, devices and shapes and allocates outputs.  There is no CPU
fallback.  Nothing here records autograd history: a backward pass is a call of
its own, to be used from a ``torch.autograd.Function``.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence

from ._binding import (MAX_FRAMES, AttentionParams, Heads, PVError, RopeParams, ScanParams, _torch, load)


def _dtypes():
    torch = _torch()
    return {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


_DTYPES = None


def _dtype(t, name: str, wide: bool = True) -> int:
    global _DTYPES
    if _DTYPES is None:
        _DTYPES = _dtypes()
    code = _DTYPES.get(t.dtype)
    if code is None or (code == 0 and not wide):
        raise TypeError(f"{name} must be {'float32, ' if wide else ''}bfloat16 or float16, got {t.dtype}")
    return code


def _heads(t, name: str, like=None, heads: Optional[int] = None) -> Heads:
    """[rows, heads, head_dim] as the library reads it: any strides that are
    multiples of 16 bytes, the last dimension dense."""
    if t.dim() != 3:
        raise ValueError(f"{name} must have shape [rows, heads, head_dim]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None:
        if t.dtype != like.dtype or t.device != like.device:
            raise TypeError(f"{name} must have the dtype and device of the other tensors")
        if t.shape[2] != like.shape[2] or (heads is None and t.shape != like.shape):
            raise ValueError(f"{name} has the wrong shape {tuple(t.shape)}")
    s = t.stride()
    if t.numel():
        align = 16 // t.element_size()
        if (s[2] != 1 and t.shape[2] > 1) or s[0] % align or s[1] % align or s[0] < 0 or t.data_ptr() % 16:
            raise ValueError(f"{name}: head_dim must be dense, its rows and heads on 16-byte boundaries")
    return Heads(t.data_ptr(), s[0], s[1])


def _floats(t, shape, device, name: str) -> int:
    torch = _torch()
    if t.dtype != torch.float32 or t.device != device:
        raise TypeError(f"{name} must be a float32 tensor on {device}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}")
    return t.data_ptr()


def _positions(t, rows: int, device, name: str):
    """int32 [rows, axes], 1 to 3 axes, rows strided as they come (a slice of
    the voxelizer's coordinates)."""
    torch = _torch()
    if t.dtype != torch.int32 or t.device != device:
        raise TypeError(f"{name} must be an int32 tensor on {device}")
    if t.dim() != 2 or t.shape[0] != rows or not 1 <= t.shape[1] <= 3:
        raise ValueError(f"{name} must have shape [{rows}, 1..3]")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the axes of a row must be dense")
    return t.data_ptr(), (t.stride(0) if rows > 1 else max(t.stride(0), t.shape[1])), int(t.shape[1])


def _offsets(seq: Sequence[int], rows: int, name: str):
    n = len(seq) - 1
    if not 1 <= n <= MAX_FRAMES:
        raise ValueError(f"{name} must hold 1 to {MAX_FRAMES} frames' offsets and the end")
    off = (ctypes.c_int64 * (n + 1))(*seq)
    if off[0] != 0 or off[n] != rows:
        raise ValueError(f"{name} must run from 0 to the {rows} rows")
    return off, n


def _stream(stream, device):
    if stream is None:
        stream = _torch().cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(status: int, where: str) -> None:
    if status != 0:
        raise PVError(status, where)


def rope_frequencies(head_dim: int, axes: int = 1, theta: float = 10000.0, device=None):
    """The usual frequencies for :func:`qk_norm_rope`, float32 [head_dim / 2]:
    pair p turns with axis p mod axes, each axis from 1 down to about 1/theta."""
    torch = _torch()
    if head_dim % 2 or not 1 <= axes <= 3:
        raise ValueError("head_dim must be even, axes 1 to 3")
    half = head_dim // 2
    return torch.tensor([theta ** (-(axes * (p // axes)) / half) for p in range(half)], dtype=torch.float32,
                        device=device)


def _rope_params(q, k, q_weight, k_weight, positions, inv_freq, eps):
    rows, hq, D = q.shape
    p = RopeParams()
    p.rows, p.q_heads, p.k_heads, p.head_dim = rows, hq, k.shape[1], D
    p.dtype = _dtype(q, "q")
    if k.shape[0] != rows:
        raise ValueError("k must have the rows of q")
    p.q_weight = _floats(q_weight, (D,), q.device, "q_weight")
    p.k_weight = _floats(k_weight, (D,), q.device, "k_weight")
    p.positions, p.position_stride, p.axes = _positions(positions, rows, q.device, "positions")
    p.inv_freq = _floats(inv_freq, (D // 2,), q.device, "inv_freq")
    p.eps = eps
    return p


def qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps: float = 1e-6, out=None, stream=None):
    """Queries [rows, H, D] and keys [rows, Hk, D] normalised per head and
    rotated by position, in one pass.

    ``x / sqrt(mean(x^2) + eps) * weight`` over each head, then the pairs
    (p, p + D/2) turned by ``positions[row, p % axes] * inv_freq[p]``.
    float32, bfloat16 or float16; D a multiple of 16 up to 256; weights and
    inv_freq float32; positions int32 [rows, axes], 1 to 3 axes (voxel
    coordinates as they stand, e.g. ``coords[:, 1:]``).  ``out`` = (q, k)
    buffers, which may be the inputs.  Returns (q, k).
    """
    torch = _torch()
    hq, hk = _heads(q, "q"), _heads(k, "k", q, k.shape[1] if k.dim() == 3 else None)
    p = _rope_params(q, k, q_weight, k_weight, positions, inv_freq, eps)
    oq, ok = out if out is not None else (torch.empty(q.shape, dtype=q.dtype, device=q.device),
                                          torch.empty(k.shape, dtype=q.dtype, device=q.device))
    _check(load().pv_qk_norm_rope(p, hq, hk, _heads(oq, "out q", q), _heads(ok, "out k", k),
                                  _stream(stream, q.device)), "pv_qk_norm_rope")
    return oq, ok


def qk_norm_rope_backward(dout_q, dout_k, q, k, q_weight, k_weight, positions, inv_freq, eps: float = 1e-6,
                          stream=None):
    """Gradients of :func:`qk_norm_rope` from those of its outputs and its
    inputs: (dq, dk, dq_weight, dk_weight), the last two float32."""
    torch = _torch()
    hq, hk = _heads(q, "q"), _heads(k, "k", q, k.shape[1] if k.dim() == 3 else None)
    p = _rope_params(q, k, q_weight, k_weight, positions, inv_freq, eps)
    dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    dk = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    dw = torch.empty((2, q.shape[2]), dtype=torch.float32, device=q.device)
    _check(load().pv_qk_norm_rope_backward(
        p, _heads(dout_q, "dout_q", q), _heads(dout_k, "dout_k", k), hq, hk, _heads(dq, "dq"), _heads(dk, "dk"),
        dw.data_ptr(), dw.data_ptr() + 4 * q.shape[2], _stream(stream, q.device)), "pv_qk_norm_rope_backward")
    return dq, dk, dw[0], dw[1]


def _attention_params(q, k, v, q_offsets, k_offsets, scale, cap, slopes, q_positions, k_positions, causal, prefix):
    p = AttentionParams()
    p.dtype = _dtype(q, "q", wide=False)
    if v.shape != k.shape:
        raise ValueError("k and v must have one shape")
    p.q_offsets, p.frames = _offsets(q_offsets, q.shape[0], "q_offsets")
    p.k_offsets, n = _offsets(k_offsets, k.shape[0], "k_offsets")
    if n != p.frames:
        raise ValueError("q_offsets and k_offsets must hold the same frames")
    p.q_heads, p.k_heads, p.head_dim = q.shape[1], k.shape[1], q.shape[2]
    if k.shape[1] < 1 or q.shape[1] % k.shape[1]:
        raise ValueError("the heads of q must be a multiple of those of k")
    p.scale = q.shape[2] ** -0.5 if scale is None else scale
    p.cap = cap
    if slopes is not None:
        if q_positions is None or k_positions is None:
            raise ValueError("slopes need q_positions and k_positions")
        p.slopes = _floats(slopes, (q.shape[1],), q.device, "slopes")
        p.q_positions, p.q_position_stride, p.axes = _positions(q_positions, q.shape[0], q.device, "q_positions")
        p.k_positions, p.k_position_stride, axes = _positions(k_positions, k.shape[0], q.device, "k_positions")
        if axes != p.axes:
            raise ValueError("q_positions and k_positions must have the same axes")
    p.causal = bool(causal)
    if prefix is not None:
        if not causal:
            raise ValueError("prefix is for causal attention")
        if len(prefix) != p.frames:
            raise ValueError("prefix must hold one length per frame")
        p.prefix = (ctypes.c_int64 * p.frames)(*prefix)
    return p


def attention(q, k, v, q_offsets, k_offsets, scale: Optional[float] = None, cap: float = 0.0, slopes=None,
              q_positions=None, k_positions=None, causal: bool = False, prefix=None, return_lse: bool = False,
              out=None, stream=None):
    """Attention of each frame's queries over the same frame's keys.

    q [queries, H, D], k and v [keys, Hk, D], bfloat16 or float16, D a multiple
    of 8 up to 128, H a multiple of Hk; ``q_offsets`` and ``k_offsets`` are the
    frames' host row offsets.  Scores ``scale * q.k`` (scale: 1/sqrt(D)) are
    capped to ``cap * tanh(s / cap)`` if cap > 0, then lowered by
    ``slopes[h] * |position difference|`` (sum over the axes) if slopes are
    given; with ``causal``, key j of nk is visible to query i of nq if
    ``j <= i + nk - nq`` or ``j < prefix[frame]``.  A query that sees no key
    gives 0.  Returns out [queries, H, D], with ``return_lse`` also the float32
    [H, queries] logarithms of the softmax sums for :func:`attention_backward`.
    """
    torch = _torch()
    hq, hk, hv = _heads(q, "q"), _heads(k, "k", q, 1), _heads(v, "v", k)
    p = _attention_params(q, k, v, q_offsets, k_offsets, scale, cap, slopes, q_positions, k_positions, causal, prefix)
    o = out if out is not None else torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device) if return_lse else None
    _check(load().pv_attention(p, hq, hk, hv, _heads(o, "out", q), lse.data_ptr() if return_lse else None,
                               _stream(stream, q.device)), "pv_attention")
    return (o, lse) if return_lse else o


def attention_backward(dout, q, k, v, out, lse, q_offsets, k_offsets, scale: Optional[float] = None, cap: float = 0.0,
                       slopes=None, q_positions=None, k_positions=None, causal: bool = False, prefix=None,
                       stream=None):
    """Gradients (dq, dk, dv) of :func:`attention` from that of its output,
    its inputs, ``out`` and ``lse``; the other arguments as there."""
    torch = _torch()
    hq, hk, hv = _heads(q, "q"), _heads(k, "k", q, 1), _heads(v, "v", k)
    p = _attention_params(q, k, v, q_offsets, k_offsets, scale, cap, slopes, q_positions, k_positions, causal, prefix)
    dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    dk = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    dv = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    _check(load().pv_attention_backward(
        p, _heads(dout, "dout", q), hq, hk, hv, _heads(out, "out", q),
        _floats(lse, (q.shape[1], q.shape[0]), q.device, "lse"), _heads(dq, "dq"), _heads(dk, "dk"), _heads(dv, "dv"),
        _stream(stream, q.device)), "pv_attention_backward")
    return dq, dk, dv


def _rows(t, name: str, like=None):
    """[rows, channels], rows strided as they come, channels dense."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor of shape [rows, channels]")
    if like is not None:
        if t.dtype != like.dtype or t.device != like.device:
            raise TypeError(f"{name} must have the dtype and device of x")
        if t.shape != like.shape:
            raise ValueError(f"{name} must have the shape of x")
    if t.shape[1] < 1 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: the channels of a row must be dense")
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else t.shape[1])


def _scan_params(x, gate, offsets, reverse):
    p = ScanParams()
    p.x, p.x_stride = _rows(x, "x")
    p.gate, p.gate_stride = _rows(gate, "gate", x)
    p.dtype = _dtype(x, "x")
    p.offsets, p.frames = _offsets(offsets, x.shape[0], "offsets")
    p.channels = x.shape[1]
    p.reverse = bool(reverse)
    return p


def gated_scan(x, gate, offsets, h0=None, reverse: bool = False, return_states: bool = False, out=None, stream=None):
    """Gated linear recurrence along each frame, every channel by itself:
    ``h[t] = (1 - z) h[t - 1] + z x[t]``, ``z = sigmoid(gate[t])``, from
    ``h0[frame]`` (zeros if None), from a frame's last row to its first if
    ``reverse``.

    x and gate [rows, channels] in float32, bfloat16 or float16 (the state is
    held in 32 bits), h0 float32 [frames, channels].  Returns (h, last): h like
    x, last float32 [frames, channels], the state after each frame's last step;
    with ``return_states`` also the states that :func:`gated_scan_backward`
    starts from.
    """
    torch = _torch()
    p = _scan_params(x, gate, offsets, reverse)
    C = x.shape[1]
    h = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    last = torch.empty((p.frames, C), dtype=torch.float32, device=x.device)
    lib = load()
    states = None
    if return_states:
        n = lib.pv_gated_scan_states(p)
        if n < 0:
            raise PVError(int(n), "pv_gated_scan_states")
        states = torch.empty((n, C), dtype=torch.float32, device=x.device)
    _check(lib.pv_gated_scan(p, None if h0 is None else _floats(h0, (p.frames, C), x.device, "h0"),
                             *_rows(h, "out", x), last.data_ptr(), states.data_ptr() if return_states else None,
                             _stream(stream, x.device)), "pv_gated_scan")
    return (h, last, states) if return_states else (h, last)


def gated_scan_backward(dh, dlast, x, gate, states, offsets, reverse: bool = False, stream=None):
    """Gradients (dx, dgate, dh0) of :func:`gated_scan` from those of h and of
    the last states (``dlast`` None: zeros), its inputs and its ``states``."""
    torch = _torch()
    p = _scan_params(x, gate, offsets, reverse)
    C = x.shape[1]
    n = load().pv_gated_scan_states(p)
    if n < 0:
        raise PVError(int(n), "pv_gated_scan_states")
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dgate = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dh0 = torch.empty((p.frames, C), dtype=torch.float32, device=x.device)
    _check(load().pv_gated_scan_backward(
        p, *_rows(dh, "dh", x), None if dlast is None else _floats(dlast, (p.frames, C), x.device, "dlast"),
        _floats(states, (n, C), x.device, "states"), *_rows(dx, "dx"), *_rows(dgate, "dgate"), dh0.data_ptr(),
        _stream(stream, x.device)), "pv_gated_scan_backward")
    return dx, dgate, dh0
