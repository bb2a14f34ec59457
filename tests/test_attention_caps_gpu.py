"""Attention with caps of any size."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytest.importorskip("lidar_point_cloud_gb300")
from test_attention_gpu import DTYPES, check, make  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cap", [1e-38, 0.01, 64.0, 65.0, 300.0, 1e4, 1e5, 1e6, 1e30, 3.3e38])
def test_caps_of_any_size(cap, dtype):
    check(make([150, 33], [260, 129], 4, 2, 64, dtype, loud=4.0), cap=cap)
    check(make([200], [200], 4, 1, 128, dtype, axes=2, loud=4.0), cap=cap, causal=True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_large_cap_among_scores_of_all_sizes(dtype):
    # Keys from 0.1 to 20 times unit size: scores from fractions to hundreds in one row.
    t = make([140], [900], 2, 1, 64, dtype)
    t["k"] *= torch.linspace(0.1, 20.0, 900, device="cuda")[:, None, None].to(dtype)
    check(t, lse_slack=2.0 ** -15, cap=1000.0)
    check(t, lse_slack=2.0 ** -15, cap=2e5)
