"""The norm in 8 bits is the norm in 32 bits divided by its scale, bit by bit."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import lidar_point_cloud_gb300 as pv  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,C,group", [(20001, 1024, 128), (20001, 1024, 0), (9001, 512, 32), (4001, 250, 64), (1001, 4096, 0)])
def test_values_and_scales_are_quotients(T, C, group, dtype):
    g = torch.Generator(device="cuda").manual_seed(C + group)
    x = torch.randn((T, C), generator=g, device="cuda").to(dtype)
    w = 1.0 + 0.2 * torch.randn((C,), generator=g, device="cuda")
    values, scales, _ = pv.rms_norm_8bit(x, w, group=group)
    # The norm of the same rows in 32 bits: the same sums, so the very numbers that are held.
    y = pv.rms_norm(x.float(), w)[0].cpu()
    width = group or C
    y = torch.nn.functional.pad(y, (0, -C % width)).view(T, -1, width)
    want = y.abs().amax(-1) / 448.0
    assert torch.equal(scales.cpu(), want)
    held = (y / want[..., None]).to(torch.float8_e4m3fn).view(T, -1)[:, :C]
    wrong = (held.contiguous().view(torch.uint8) != values.cpu().view(torch.uint8)).sum().item()
    assert wrong == 0, wrong
