"""Operators on the tokens of voxelized frames: argument marshalling only.

A batch of frames (:func:`voxelize_batch`) is a ragged sequence of tokens, one
row per voxel, frame b the rows ``offsets[b]:offsets[b + 1]``; ``offsets`` is a
host sequence of ints (not the voxelizer's ``frame_offsets``, which count points: the
tokens of each frame are counted in the coordinates' first column).  The work is
done by libpv.so (``include/pv.h``, "Operators on voxel tokens"); this file
checks dtypes, devices and shapes and allocates outputs.  There is no CPU
fallback.  Nothing here records autograd history: a backward pass is a call of
its own, to be used from a ``torch.autograd.Function``.
"""

from __future__ import annotations

import array
from typing import Optional, Sequence

from ._binding import (MAX_FRAMES, AttentionParams, Heads, PVError, RopeParams, ScanParams, _torch, load)

_codes = None


def _dtype(t, name: str, wide: bool = True) -> int:
    global _codes
    if _codes is None:
        torch = _torch()
        _codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    code = _codes.get(t.dtype)
    if code is None or (code == 0 and not wide):
        raise TypeError(f"{name} must be {'float32, ' if wide else ''}bfloat16 or float16, got {t.dtype}")
    return code


def _strides(t, shape):
    """Those of rows and heads (0 where there is one only: torch gives it any) and of head_dim."""
    row, head, one = t.stride()
    return row if shape[0] > 1 else 0, head if shape[1] > 1 else 0, one


def _heads(t, name: str, like=None, heads: Optional[int] = None, apart: bool = False) -> Heads:
    """[rows, heads, head_dim] as the library reads it: any strides that are
    multiples of 16 bytes, the last dimension dense.  `like`: the tensor whose
    dtype, device and head_dim (and, with no `heads`, shape) it must have.
    `apart`: a tensor expanded over its rows (as the gradient of a sum over them
    is) is copied, for calls whose rows have to lie apart."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must have shape [rows, heads, head_dim]")
    if like is None:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
    else:
        if t.dtype is not like.dtype or t.get_device() != like.get_device():
            raise TypeError(f"{name} must have the dtype and device of the other tensors")
        if shape[2] != like.shape[2] or (heads is None and shape != like.shape):
            raise ValueError(f"{name} has the wrong shape {tuple(shape)}")
    row, head, one = _strides(t, shape)
    copy = apart and row == 0 and shape[0] > 1
    if copy:
        t = t.contiguous()
        row, head, one = _strides(t, shape)
    at = t.data_ptr()
    size = t.element_size()
    if (at | row * size | head * size) & 15 or one != 1 or row < 0:
        if t.numel() and not (one != 1 and shape[2] == 1 and not (at | row * size | head * size) & 15):
            raise ValueError(f"{name}: head_dim must be dense, its rows and heads on 16-byte boundaries")
    h = Heads(at, row, head)
    if copy:
        h.kept = t  # until the call that reads it has been enqueued
    return h


def _gradient(t):
    """A gradient with a dense last dimension: that of a plain sum is one element
    expanded over everything, and is written out."""
    return t.contiguous() if t.dim() and t.numel() and t.stride(-1) == 0 else t


def _dense(like):
    torch = _torch()
    if like.is_contiguous():
        return torch.empty_like(like)  # the quickest of torch's ways
    return torch.empty(like.shape, dtype=like.dtype, device=like.device)


def _new(like):
    """A dense tensor like this one, and how the library reads it."""
    t = _dense(like)
    row, head, _ = _strides(t, t.shape)
    return t, Heads(t.data_ptr(), row, head)


def _floats(t, shape, dev: int, name: str) -> int:
    if t.dtype is not _torch().float32 or t.get_device() != dev:
        raise TypeError(f"{name} must be a float32 tensor on the device of the others")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {shape}")
    return t.data_ptr()


def _positions(t, rows: int, dev: int, name: str):
    """int32 [rows, axes], 1 to 3 axes, rows strided as they come (a slice of
    the voxelizer's coordinates)."""
    if t.dtype is not _torch().int32 or t.get_device() != dev:
        raise TypeError(f"{name} must be an int32 tensor on the device of the others")
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or not 1 <= shape[1] <= 3:
        raise ValueError(f"{name} must have shape [{rows}, 1..3]")
    stride, one = t.stride()
    if shape[1] > 1 and one != 1:
        raise ValueError(f"{name}: the axes of a row must be dense")
    return t.data_ptr(), (stride if rows > 1 else max(stride, shape[1])), shape[1]


def _offsets(seq: Sequence[int], rows: int, name: str):
    n = len(seq) - 1
    if not 1 <= n <= MAX_FRAMES:
        raise ValueError(f"{name} must hold 1 to {MAX_FRAMES} frames' offsets and the end")
    off = array.array("q", seq)
    if off[0] != 0 or off[n] != rows:
        raise ValueError(f"{name} must run from 0 to the {rows} rows")
    return off, n


def _stream(t) -> int:
    return _torch()._C._cuda_getCurrentRawStream(t.get_device())


def _on(stream, t):
    """`stream` (a torch stream or a handle) made the current one, so that outputs come
    from its memory: what another stream still uses is not handed to it."""
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(handle, device=t.device)
    return torch.cuda.stream(stream)


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
    if k.shape[0] != rows:
        raise ValueError("k must have the rows of q")
    dev = q.get_device()
    pos, stride, axes = _positions(positions, rows, dev, "positions")
    return RopeParams(rows, hq, k.shape[1], D, _dtype(q, "q"), _floats(q_weight, (D,), dev, "q_weight"),
                      _floats(k_weight, (D,), dev, "k_weight"), pos, stride, axes,
                      _floats(inv_freq, (D // 2,), dev, "inv_freq"), eps)


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
    if stream is not None:
        with _on(stream, q):
            return qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps, out)
    hq, hk = _heads(q, "q"), _heads(k, "k", q, 1)
    p = _rope_params(q, k, q_weight, k_weight, positions, inv_freq, eps)
    if out is None:
        (oq, hoq), (ok, hok) = _new(q), _new(k)
    else:
        oq, ok = out
        hoq, hok = _heads(oq, "out q", q), _heads(ok, "out k", k)
    _check(load().pv_qk_norm_rope(p, hq, hk, hoq, hok, _stream(q)), "pv_qk_norm_rope")
    return oq, ok


def qk_norm_rope_backward(dout_q, dout_k, q, k, q_weight, k_weight, positions, inv_freq, eps: float = 1e-6,
                          stream=None):
    """Gradients of :func:`qk_norm_rope` from those of its outputs and its
    inputs: (dq, dk, dq_weight, dk_weight), the last two float32."""
    if stream is not None:
        with _on(stream, q):
            return qk_norm_rope_backward(dout_q, dout_k, q, k, q_weight, k_weight, positions, inv_freq, eps)
    torch = _torch()
    dout_q, dout_k = _gradient(dout_q), _gradient(dout_k)
    hq, hk = _heads(q, "q"), _heads(k, "k", q, 1)
    p = _rope_params(q, k, q_weight, k_weight, positions, inv_freq, eps)
    (dq, hdq), (dk, hdk) = _new(q), _new(k)
    D = q.shape[2]
    dw = (torch.empty if k.shape[1] else torch.zeros)((2, D), dtype=torch.float32, device=q.device)
    at = dw.data_ptr()
    _check(load().pv_qk_norm_rope_backward(p, _heads(dout_q, "dout_q", q), _heads(dout_k, "dout_k", k), hq, hk, hdq, hdk,
                                           at, at + 4 * D, _stream(q)), "pv_qk_norm_rope_backward")
    return dq, dk, dw[0], dw[1]


def _attention_params(q, k, v, q_offsets, k_offsets, scale, cap, slopes, q_positions, k_positions, causal, prefix):
    """The call's parameters, and the host arrays that they point to."""
    if v.shape != k.shape:
        raise ValueError("k and v must have one shape")
    rows, H, D = q.shape
    keys, Hk, _ = k.shape
    qo, frames = _offsets(q_offsets, rows, "q_offsets")
    ko, n = _offsets(k_offsets, keys, "k_offsets")
    if n != frames:
        raise ValueError("q_offsets and k_offsets must hold the same frames")
    if Hk < 1 or H % Hk:
        raise ValueError("the heads of q must be a multiple of those of k")
    p = AttentionParams(frames, qo.buffer_info()[0], ko.buffer_info()[0], H, Hk, D, _dtype(q, "q", wide=False),
                        D ** -0.5 if scale is None else scale, cap)
    if slopes is not None:
        if q_positions is None or k_positions is None:
            raise ValueError("slopes need q_positions and k_positions")
        dev = q.get_device()
        p.slopes = _floats(slopes, (H,), dev, "slopes")
        p.q_positions, p.q_position_stride, p.axes = _positions(q_positions, rows, dev, "q_positions")
        p.k_positions, p.k_position_stride, axes = _positions(k_positions, keys, dev, "k_positions")
        if axes != p.axes:
            raise ValueError("q_positions and k_positions must have the same axes")
    pre = None
    if causal:
        p.causal = 1
    if prefix is not None:
        if not causal:
            raise ValueError("prefix is for causal attention")
        if len(prefix) != frames:
            raise ValueError("prefix must hold one length per frame")
        pre = array.array("q", prefix)
        p.prefix = pre.buffer_info()[0]
    return p, (qo, ko, pre)


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
    Sums are held in 32 bits; the probabilities are rounded to q's type for the
    product with v, as the tensor cores take them.  Tensors expanded over their
    rows are copied.
    """
    if stream is not None:
        with _on(stream, q):
            return attention(q, k, v, q_offsets, k_offsets, scale, cap, slopes, q_positions, k_positions, causal, prefix,
                             return_lse, out)
    hq, hk, hv = _heads(q, "q", apart=True), _heads(k, "k", q, 1, apart=True), _heads(v, "v", k, apart=True)
    p, _alive = _attention_params(q, k, v, q_offsets, k_offsets, scale, cap, slopes, q_positions, k_positions, causal,
                                  prefix)
    o, ho = _new(q) if out is None else (out, _heads(out, "out", q))
    if not return_lse:
        _check(load().pv_attention(p, hq, hk, hv, ho, None, _stream(q)), "pv_attention")
        return o
    torch = _torch()
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    _check(load().pv_attention(p, hq, hk, hv, ho, lse.data_ptr(), _stream(q)), "pv_attention")
    return o, lse


def attention_backward(dout, q, k, v, out, lse, q_offsets, k_offsets, scale: Optional[float] = None, cap: float = 0.0,
                       slopes=None, q_positions=None, k_positions=None, causal: bool = False, prefix=None,
                       stream=None):
    """Gradients (dq, dk, dv) of :func:`attention` from that of its output,
    its inputs, ``out`` and ``lse``; the other arguments as there.  Probabilities
    and the scores' gradients are rounded to q's type for the products (in
    float16 scaled so that they neither overflow nor run out of exponent)."""
    if stream is not None:
        with _on(stream, q):
            return attention_backward(dout, q, k, v, out, lse, q_offsets, k_offsets, scale, cap, slopes, q_positions,
                                      k_positions, causal, prefix)
    hq, hk, hv = _heads(q, "q", apart=True), _heads(k, "k", q, 1, apart=True), _heads(v, "v", k, apart=True)
    p, _alive = _attention_params(q, k, v, q_offsets, k_offsets, scale, cap, slopes, q_positions, k_positions, causal,
                                  prefix)
    (dq, hdq), (dk, hdk), (dv, hdv) = _new(q), _new(k), _new(k)
    _check(load().pv_attention_backward(
        p, _heads(dout, "dout", q, apart=True), hq, hk, hv, _heads(out, "out", q),
        _floats(lse, (q.shape[1], q.shape[0]), q.get_device(), "lse"), hdq, hdk, hdv, _stream(q)),
        "pv_attention_backward")
    return dq, dk, dv


def _rows(t, name: str, like=None):
    """[rows, channels], rows strided as they come, channels dense."""
    shape = t.shape
    if len(shape) != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor of shape [rows, channels]")
    if like is not None:
        if t.dtype is not like.dtype or t.get_device() != like.get_device():
            raise TypeError(f"{name} must have the dtype and device of x")
        if shape != like.shape:
            raise ValueError(f"{name} must have the shape of x")
    row, one = t.stride()
    if shape[1] < 1 or (shape[1] > 1 and one != 1):
        raise ValueError(f"{name}: the channels of a row must be dense")
    return t.data_ptr(), (row if shape[0] > 1 else shape[1])


def _scan_params(x, gate, offsets, reverse):
    """The call's parameters, and the host array that they point to."""
    xp, xs = _rows(x, "x")
    gp, gs = _rows(gate, "gate", x)
    code = _dtype(x, "x")
    off, frames = _offsets(offsets, x.shape[0], "offsets")
    return ScanParams(frames, off.buffer_info()[0], x.shape[1], code, 1 if reverse else 0, xp, xs, gp, gs), off


def _states(lib, p) -> int:
    n = lib.pv_gated_scan_states(p)
    if n < 0:
        raise PVError(int(n), "pv_gated_scan_states")
    return n


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
    if stream is not None:
        with _on(stream, x):
            return gated_scan(x, gate, offsets, h0, reverse, return_states, out)
    torch = _torch()
    p, _alive = _scan_params(x, gate, offsets, reverse)
    C = x.shape[1]
    state = (p.frames, C)
    lib = load()
    if out is None:
        out = _dense(x)
        h, hs = out.data_ptr(), C
    else:
        h, hs = _rows(out, "out", x)
    last = torch.empty(state, dtype=torch.float32, device=x.device)
    states = torch.empty((_states(lib, p), C), dtype=torch.float32, device=x.device) if return_states else None
    _check(lib.pv_gated_scan(p, None if h0 is None else _floats(h0, state, x.get_device(), "h0"), h, hs, last.data_ptr(),
                             states.data_ptr() if return_states else None, _stream(x)), "pv_gated_scan")
    return (out, last, states) if return_states else (out, last)


def gated_scan_backward(dh, dlast, x, gate, states, offsets, reverse: bool = False, stream=None):
    """Gradients (dx, dgate, dh0) of :func:`gated_scan` from those of h and of
    the last states (``dlast`` None: zeros), its inputs and its ``states``."""
    if stream is not None:
        with _on(stream, x):
            return gated_scan_backward(dh, dlast, x, gate, states, offsets, reverse)
    p, _alive = _scan_params(x, gate, offsets, reverse)
    C, dev = x.shape[1], x.get_device()
    state = (p.frames, C)
    lib = load()
    dh = _gradient(dh)
    dhp, dhs = _rows(dh, "dh", x)
    dx, dgate = _dense(x), _dense(x)
    torch = _torch()
    dh0 = torch.empty(state, dtype=torch.float32, device=x.device)
    _check(lib.pv_gated_scan_backward(
        p, dhp, dhs, None if dlast is None else _floats(dlast, state, dev, "dlast"),
        _floats(states, (_states(lib, p), C), dev, "states"), dx.data_ptr(), C, dgate.data_ptr(), C, dh0.data_ptr(),
        _stream(x)), "pv_gated_scan_backward")
    return dx, dgate, dh0
