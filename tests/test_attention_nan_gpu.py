"""Attention with queries that are not numbers."""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")
from test_attention_gpu import make  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("keys", [40, 20000])
def test_a_query_that_is_not_a_number(keys):
    # Its softmax sum is not one either, and the other queries' are as before.  (20,000 keys
    # are cut over blocks and joined.)
    t = make([3], [keys], 2, 1, 64, torch.bfloat16)
    o, lse = pv.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], return_lse=True)
    t["q"][1, 0] = math.nan
    o2, lse2 = pv.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], return_lse=True)
    assert torch.isnan(o2[1, 0]).all() and torch.isnan(lse2[0, 1])
    keep = torch.ones((3, 2), dtype=torch.bool, device="cuda")
    keep[1, 0] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse.T[keep], lse2.T[keep])
