"""The rotation of queries alone: keys of no heads."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")
from test_rope_gpu import make  # noqa: E402

pytestmark = pytest.mark.gpu


def test_the_weight_that_nothing_used_gets_no_gradient(monkeypatch):
    q, k, dq, dk, wq, wk, pos, freq = make(50, 4, 2, 64, 2, torch.bfloat16)
    want = pv.qk_norm_rope_backward(dq, dk, q, k, wq, wk, pos, freq)
    # What is allocated holds something.
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **how: empty(*a, **how).fill_(float("nan")))
    oq, ok = pv.qk_norm_rope(q, k[:, :0], wq, wk, pos, freq)
    gq, gk, gwq, gwk = pv.qk_norm_rope_backward(dq, dk[:, :0], q, k[:, :0], wq, wk, pos, freq)
    assert torch.equal(oq, pv.qk_norm_rope(q, k, wq, wk, pos, freq)[0]) and ok.shape == gk.shape == (50, 0, 64)
    assert torch.equal(gq, want[0]) and torch.equal(gwq, want[2]) and not gwk.any()
