"""Attention's errors as a share of each result's norm.

Bounds on single elements are worst cases, some tens of times a usual error.  Over a whole tensor
independent roundings add up as squares: an output carries its own rounding, of at most `unit`,
and that of the probabilities (in the storage type), so that its norm is off by less than
2 unit; a gradient also that of the scores' gradients and of the sum subtracted there: 3 unit."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")
import _tokens as ref  # noqa: E402
from test_attention_gpu import DTYPES, make, own  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hk,D", [(4, 4, 32), (8, 2, 64), (4, 1, 128)])
@pytest.mark.parametrize("axes,how", [(0, {}), (0, {"causal": True, "prefix": [50, 0]}), (2, {}), (0, {"cap": 5.0}),
                                      (3, {"cap": 20.0, "causal": True}), (0, {"cap": 500.0})])
def test_relative_norms(axes, how, H, Hk, D, dtype):
    t = make([400, 150], [600, 150], H, Hk, D, dtype, axes=axes, loud=2.0, seed=3)
    how = {**t["how"], **how}
    want, _ = ref.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], dout=t["dout"], **how)
    o, lse = pv.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], return_lse=True, **own(how))
    grads = pv.attention_backward(t["dout"], t["q"], t["k"], t["v"], o, lse, t["qo"], t["ko"], **own(how))
    for got, n, units in zip((o, *grads), ("out", "dq", "dk", "dv"), (2, 3, 3, 3)):
        off = float((got.double() - want[n]).norm() / want[n].norm())
        assert off < units * ref.UNIT[dtype], (n, off / ref.UNIT[dtype])
