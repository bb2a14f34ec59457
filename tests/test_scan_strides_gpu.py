"""The gated recurrence whose rows begin on odd elements."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")
import _tokens as ref  # noqa: E402
from test_scan_gpu import close, make  # noqa: E402

pytestmark = pytest.mark.gpu


def check(x, gate, dh, off, h0, dlast, reverse=False, forward_x=None):
    """Both passes against 64 bits; `forward_x`: the same x, laid out otherwise, for the forward call."""
    dtype = x.dtype
    h, last, states = pv.gated_scan(x if forward_x is None else forward_x, gate, off, h0, reverse=reverse, return_states=True)
    dx, dgate, dh0 = pv.gated_scan_backward(dh, dlast, x, gate, states, off, reverse=reverse)
    want = ref.scan(x, gate, off, h0, reverse, dh, dlast)
    close(h, want["h"], dtype, "h", 4.0)
    close(last, want["last"], torch.float32, "last", 4.0)
    close(dx, want["dx"], dtype, "dx", 16.0)
    close(dgate, want["dgate"], dtype, "dgate", 64.0)
    close(dh0, want["dh0"], torch.float32, "dh0", 64.0)


def wider(t, at, extra):
    """The same values, rows `extra` elements further apart, beginning `at` elements in."""
    w = torch.zeros((t.shape[0], t.shape[1] + extra), dtype=t.dtype, device=t.device)
    w[:, at:at + t.shape[1]] = t
    return w[:, at:at + t.shape[1]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,C", [([130, 260], 48), ([1], 2), ([300, 0, 7], 2), ([700], 64), ([500, 40], 130), ([90], 6)])
@pytest.mark.parametrize("at,extra", [(1, 2), (0, 1), (3, 4)])
def test_rows_that_begin_on_odd_elements(lens, C, at, extra, dtype):
    # An odd offset with an even row stride, and an odd row stride: no two channels share a word.
    x, gate, dh, off, h0, dlast = make(lens, C, dtype)
    odd = [wider(t, at, extra) for t in (x, gate, dh)]
    check(*odd, off, h0, dlast)
    # One tensor of either kind, and states that another layout's forward call left.
    check(x, gate, odd[2], off, h0, dlast, reverse=True)
    check(odd[0], gate, dh, off, h0, dlast, forward_x=x)
    check(x, gate, dh, off, h0, dlast, forward_x=odd[0])
