"""The token operators without a GPU: their argument checks in the library and in
the binding, and the sizes that the library works out on the host.  Nothing is launched."""

from __future__ import annotations

import array
import ctypes

import numpy as np
import pytest

import lidar_point_cloud_gb300 as pv
from lidar_point_cloud_gb300 import _binding, _build

INVALID = -1


@pytest.fixture(scope="module")
def lib():
    if _build.is_stale():
        _build.build()
    return pv.load()


HOST = np.zeros(4096, dtype=np.float32)  # host memory where device memory is needed
PTR = HOST.ctypes.data - HOST.ctypes.data % 16 + 16
HEADS = _binding.Heads(PTR, 64, 16)


def offsets(*values):
    return array.array("q", values)


def rope(**change):
    p = dict(rows=4, q_heads=2, k_heads=1, head_dim=32, dtype=1, q_weight=PTR, k_weight=PTR, positions=PTR,
             position_stride=3, axes=3, inv_freq=PTR, eps=1e-6)
    p.update(change)
    return _binding.RopeParams(**p)


@pytest.mark.parametrize("change", [
    {}, {"dtype": 7}, {"rows": -1}, {"rows": 1 << 31}, {"q_heads": 0}, {"k_heads": -1}, {"head_dim": 24}, {"head_dim": 8},
    {"head_dim": 272}, {"axes": 0}, {"axes": 4}, {"position_stride": 2}, {"eps": -1.0}, {"eps": float("nan")},
    {"q_weight": None}, {"k_weight": None}, {"positions": None}, {"inv_freq": None}])
def test_rotation_refuses(lib, change):
    p = rope(**change)
    assert lib.pv_qk_norm_rope(p, HEADS, HEADS, HEADS, HEADS, None) == INVALID
    assert lib.pv_qk_norm_rope_backward(p, HEADS, HEADS, HEADS, HEADS, HEADS, HEADS, PTR, PTR, None) == INVALID


def attention(q=(0, 4), k=(0, 4), **change):
    qo, ko = offsets(*q), offsets(*k)
    p = dict(frames=len(q) - 1, q_offsets=qo.buffer_info()[0], k_offsets=ko.buffer_info()[0], q_heads=2, k_heads=1,
             head_dim=32, dtype=1, scale=0.2, cap=0.0)
    p.update(change)
    return _binding.AttentionParams(**p), (qo, ko)


@pytest.mark.parametrize("change", [
    {}, {"dtype": 0}, {"dtype": 9}, {"q_heads": 3, "k_heads": 2}, {"q_heads": 0}, {"k_heads": 0}, {"head_dim": 12},
    {"head_dim": 136}, {"head_dim": 0}, {"scale": 0.0}, {"scale": float("inf")}, {"cap": -1.0}, {"cap": float("nan")},
    {"q": (1, 4)}, {"q": (0, 4, 3), "k": (0, 2, 4)}, {"k": (0, 1 << 31)}, {"q_offsets": None}, {"k_offsets": None}, {"frames": 0},
    {"frames": 257}, {"slopes": PTR, "axes": 0}, {"slopes": PTR, "axes": 2, "q_position_stride": 1, "k_position_stride": 2}])
def test_attention_refuses(lib, change):
    p, alive = attention(**change)
    assert lib.pv_attention(p, HEADS, HEADS, HEADS, HEADS, None, None) == INVALID
    assert lib.pv_attention_backward(p, HEADS, HEADS, HEADS, HEADS, HEADS, PTR, HEADS, HEADS, HEADS, None) == INVALID
    del alive


def test_null_blocks_are_refused(lib):
    p, alive = attention()
    assert lib.pv_attention(None, HEADS, HEADS, HEADS, HEADS, None, None) == INVALID
    assert lib.pv_attention(p, None, HEADS, HEADS, HEADS, None, None) == INVALID
    assert lib.pv_attention(p, HEADS, HEADS, HEADS, None, None, None) == INVALID
    assert lib.pv_qk_norm_rope(None, HEADS, HEADS, HEADS, HEADS, None) == INVALID
    assert lib.pv_gated_scan(None, None, PTR, 8, None, None, None) == INVALID
    assert lib.pv_gated_scan_states(None) == INVALID
    del alive


def scan(off=(0, 100), **change):
    o = offsets(*off)
    p = dict(frames=len(off) - 1, offsets=o.buffer_info()[0], channels=64, dtype=1, reverse=0, x=PTR, x_stride=64, gate=PTR,
             gate_stride=64)
    p.update(change)
    return _binding.ScanParams(**p), o


@pytest.mark.parametrize("change", [
    {}, {"dtype": 5}, {"channels": 0}, {"channels": (1 << 20) + 1}, {"off": (0, 5, 4)}, {"off": (2, 5)}, {"off": (0, 1 << 31)},
    {"offsets": None}, {"frames": 0}, {"x_stride": 63}, {"gate_stride": 8}, {"x": None}, {"gate": None}])
def test_recurrence_refuses(lib, change):
    p, alive = scan(**change)
    assert lib.pv_gated_scan(p, None, PTR, 64, None, None, None) == INVALID
    assert lib.pv_gated_scan_backward(p, PTR, 64, None, PTR, PTR, 64, PTR, 64, None, None) == INVALID
    del alive


def test_states_cover_every_frame(lib):
    # A state before each stretch of a frame's steps: none for an empty frame, at least
    # one for any other, and no more than one a step.
    for off, channels, dtype in (((0, 1), 64, 1), ((0, 0), 64, 1), ((0, 1000), 64, 1), ((0, 1000), 1, 0), ((0, 7, 7, 500), 33, 2),
                                 ((0, 100_000), 512, 1)):
        p, alive = scan(off, channels=channels, dtype=dtype)
        n = lib.pv_gated_scan_states(p)
        some = sum(b > a for a, b in zip(off, off[1:]))
        assert some <= n <= off[-1]
        one, keep = scan((0, off[-1]), channels=channels, dtype=dtype)
        assert n >= lib.pv_gated_scan_states(one)
        del alive, keep


def test_binding_refuses_host_tensors(lib):
    torch = pytest.importorskip("torch")
    q = torch.zeros((4, 2, 32), dtype=torch.bfloat16)
    w = torch.ones((32,))
    with pytest.raises(ValueError):
        pv.qk_norm_rope(q, q, w, w, torch.zeros((4, 1), dtype=torch.int32), torch.ones((16,)))
    with pytest.raises(ValueError):
        pv.attention(q, q, q, [0, 4], [0, 4])
    with pytest.raises(ValueError):
        pv.gated_scan(q[:, 0], q[:, 0], [0, 4])


def test_frequencies():
    pytest.importorskip("torch")
    f = pv.rope_frequencies(64)
    assert f.shape == (32,) and f[0] == 1.0 and f[31] == pytest.approx(10000.0 ** (-31 / 32))
    g = pv.rope_frequencies(48, axes=3)
    assert [float(x) for x in g[:3]] == [1.0, 1.0, 1.0] and g[3] == pytest.approx(10000.0 ** (-3 / 24))
    with pytest.raises(ValueError):
        pv.rope_frequencies(63)


def test_structures_match_the_header():
    # Field by field as pv.h lays them out on a 64-bit machine.
    sizes = {_binding.Heads: 24, _binding.RopeParams: 80, _binding.AttentionParams: 104, _binding.ScanParams: 64}
    for block, size in sizes.items():
        assert ctypes.sizeof(block) == size, block
