"""The gated recurrence where its values are not finite."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")
import _tokens as ref  # noqa: E402
from test_scan_gpu import DTYPES, close, make  # noqa: E402

pytestmark = pytest.mark.gpu


def same_kind(got, want, name):
    got, want = got.double().cpu(), want.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), name
    assert torch.equal(got.isposinf(), want.isposinf()) and torch.equal(got.isneginf(), want.isneginf()), name
    some = torch.isfinite(want)
    return got[some], want[some]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("mean", [-2.0, 4.0])
@pytest.mark.parametrize("length", [20, 300, 5000])
def test_infinities_stay(length, mean, reverse, dtype):
    # (1 - z) h + z x with 0 < z < 1: an infinite state stays infinite, and meets its opposite as
    # no number, however many steps on.  (Mostly open gates: the product of a tile's 1 - z is 0 in 32 bits.)
    inf = float("inf")
    x, gate, dh, off, h0, dlast = make([length, 7, 40], 34, dtype, mean=mean)
    gate.clamp_(-8.0, 8.0)
    x[5, 0], x[7, 1], x[off[1] - 1, 2], x[9, 3] = inf, -inf, inf, inf
    x[12, 3] = -inf
    h0[0, 4], h0[1, 5], h0[2, 6] = inf, -inf, inf
    dh[length - 3, 7], dh[2, 8], dlast[0, 9], dlast[2, 10] = inf, -inf, inf, -inf
    h, last, states = pv.gated_scan(x, gate, off, h0, reverse=reverse, return_states=True)
    grads = pv.gated_scan_backward(dh, dlast, x, gate, states, off, reverse=reverse)
    want = ref.scan(x, gate, off, h0, reverse, dh, dlast)
    for got, n, big in ((h, "h", 4.0), (last, "last", 4.0), *zip(grads, ("dx", "dgate", "dh0"), (16.0, 64.0, 64.0))):
        a, b = same_kind(got, want[n], n)
        close(a, b, torch.float32 if n in ("last", "dh0") else dtype, n, big)


def test_a_closed_gate_keeps_an_infinite_state_and_an_open_one_ends_it():
    # A gate of -inf: z = 0.  A gate of +inf: z = 1, and 0 times infinity is no number.
    x, gate, _, off, h0, _ = make([600], 8, torch.float32)
    gate[:] = -float("inf")
    h0[:] = float("inf")
    h, last = pv.gated_scan(x, gate, off, h0)
    assert h.isposinf().all() and last.isposinf().all()
    gate[300] = float("inf")
    h, last = pv.gated_scan(x, gate, off, h0)
    assert h[:300].isposinf().all() and torch.isnan(h[300:]).all() and torch.isnan(last).all()
