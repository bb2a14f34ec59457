"""What the norm and the cross entropy give past the range of 32 bits, as the header says."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import lidar_point_cloud_gb300 as pv  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("C", [64, 37, 1024])
def test_rows_whose_squares_pass_32_bits_are_zeros(C, dtype):
    g = torch.Generator(device="cuda").manual_seed(C)
    x = torch.randn((5, C), generator=g, device="cuda").to(dtype)
    w = torch.ones((C,), device="cuda")
    clean = x.clone()
    x[1] = 1e25
    x[3, 0] = torch.finfo(dtype).min
    y, _ = pv.rms_norm(x, w)
    values, scales, _ = pv.rms_norm_8bit(x, w)
    for i in (1, 3):
        assert (y[i] == 0).all() and (values[i].float() == 0).all() and (scales[i] > 0).all()
    keep = [0, 2, 4]
    assert torch.equal(y[keep], pv.rms_norm(clean, w)[0][keep])
    assert torch.equal(scales[keep], pv.rms_norm_8bit(clean, w)[1][keep])


@pytest.mark.parametrize("T", [6, 300])
def test_rows_with_an_infinite_logit_are_no_numbers(T):
    # (6 rows and 300 are different kernels.)
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, 64), generator=g, device="cuda").bfloat16().abs()
    w = torch.randn((700, 64), generator=g, device="cuda").bfloat16()
    target = torch.randint(0, 500, (T,), generator=g, device="cuda")
    down = w.clone()
    down[600] = -torch.inf  # a class that no row takes
    loss, lse = pv.cross_entropy(x, down, target)
    rest = torch.cat([w[:600], w[601:]])
    want = torch.logsumexp(x.double() @ rest.double().T, -1)
    # (A logit is off by less than 2^-20 of its terms' magnitudes, some 64 at the most, and lse by a few units of 2^-23.)
    assert ((lse.double() - want).abs() <= 2.0 ** -18 * (want.abs() + 64)).all() and torch.isfinite(loss).all()
    w[600] = torch.inf
    loss, lse = pv.cross_entropy(x, w, target)
    assert torch.isnan(lse).all() and torch.isnan(loss).all()
