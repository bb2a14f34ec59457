"""The recurrence and the rotation on tensors expanded from one row or one element, as the gradients
of sums are."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")
import test_rope_gpu as rope  # noqa: E402
from test_scan_gpu import DTYPES, make  # noqa: E402
from test_scan_strides_gpu import check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [24, 7])
def test_recurrence(C, dtype):
    # The gradients of h.sum(0) and of h.sum(), and inputs that are one row seen as many.
    x, gate, dh, off, h0, dlast = make([60, 23], C, dtype)
    check(x, gate, dh[:1].expand(83, -1), off, h0, dlast)
    check(x, gate, dh[:1, :1].expand(83, C), off, h0, dlast)
    check(x[:1].expand(83, -1), gate[:1].expand(83, -1), dh, off, h0, dlast)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rotation(dtype):
    q, k, dq, dk, wq, wk, pos, freq = rope.make(83, 4, 2, 32, 2, dtype)
    for a, b in ((dq[:1].expand(83, -1, -1), dk[:1].expand(83, -1, -1)),
                 (dq[:1, :1, :1].expand(83, 4, 32), dk[:1, :1, :1].expand(83, 2, 32))):
        got = pv.qk_norm_rope_backward(a, b, q, k, wq, wk, pos, freq)
        want = pv.qk_norm_rope_backward(a.contiguous(), b.contiguous(), q, k, wq, wk, pos, freq)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
