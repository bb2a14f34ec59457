"""The cross entropy past what one piece of the classes holds, past the channels of one block, and with rows
whose weights lie far apart."""

from __future__ import annotations

import os
import re

import pytest

torch = pytest.importorskip("torch")

import lidar_point_cloud_gb300 as pv  # noqa: E402
from lidar_point_cloud_gb300 import _build  # noqa: E402
from test_loss_gpu import SMALL, TYPES, both, check, inputs, near  # noqa: E402

pytestmark = pytest.mark.gpu


def piece_bytes():
    with open(os.path.join(_build.CSRC, "pv_loss.cu")) as f:
        n, shift = re.search(r"kPieceBytes = int64_t\((\d+)\) << (\d+);", f.read()).groups()
    return int(n) << int(shift)


@pytest.mark.parametrize("dtype", TYPES)
def test_several_pieces_of_the_classes(dtype):
    # Three pieces or more, the last one shorter and no multiple of a tile's 256 classes.
    T, V, D = 20001, 45001, 72
    assert 2 * T * V > 2 * piece_bytes()
    x, w, target, dloss, dlse = inputs(T, V, D, dtype, seed=21)
    loss, lse, dx, dw = both(x, w, target, dloss, dlse)
    u = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * u
    wide = w.double()
    some, c1 = target >= 0, dlse.double()
    c2 = torch.where(some, dloss.double(), 0.0)
    c1 = c1 + c2
    most = max(c1.abs().max().item(), c2.abs().max().item())
    dw_want, dw_slack = torch.zeros_like(wide), torch.zeros_like(wide)
    # (The bounds are those of test_loss_gpu.check, block by block of the rows.)
    for r in torch.arange(T, device="cuda").split(2048):
        a, at = x[r].double(), target[r].clamp_min(0)[:, None]
        z = a @ wide.T
        noise = (SMALL * (a.abs() @ wide.abs().T)).amax(-1)
        want = torch.logsumexp(z, -1)
        near(lse[r], want, noise + 2.0 ** -21 * (want.abs() + 1))
        hit = z.gather(1, at)[:, 0]
        near(loss[r], torch.where(some[r], want - hit, 0.0), 2 * noise + 2.0 ** -21 * (want.abs() + hit.abs() + 1))
        G = c1[r, None] * (z - want[:, None]).exp()
        e = G.abs() * (2 * noise + 2.0 ** -20 * (1 + want.abs()))[:, None]
        G.scatter_add_(1, at, -c2[r, None])
        e += u * G.abs() + SMALL * G.abs() + (2.0 ** -39 * most if dtype == torch.float16 else 0.0)
        e.scatter_add_(1, at, 2.0 ** -22 * c2[r, None])
        dx_want = G @ wide
        near(dx[r], dx_want, e @ wide.abs() + SMALL * (G.abs() @ wide.abs()) + u * dx_want.abs() + tiny)
        dw_want += G.T @ a
        dw_slack += e.T @ a.abs() + SMALL * (G.abs().T @ a.abs())
    near(dw, dw_want, dw_slack + u * dw_want.abs() + tiny)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V,D", [(8, 700, 968), (8, 700, 1024), (32, 700, 1024), (33, 700, 1024), (8, 700, 1032), (32, 300, 2048),
                                   (300, 600, 2056), (40, 300, 16384)])
def test_many_channels(T, V, D, dtype):
    # Whole numbers (times a power of two): the sums of up to 16,384 products are exact in 32 bits, in any order.
    _, _, target, dloss, dlse = inputs(T, V, 8, dtype, seed=22)
    g = torch.Generator(device="cuda").manual_seed(D)
    x = torch.randint(-1, 2, (T, D), generator=g, device="cuda").to(dtype)
    w = (torch.randint(-2, 3, (V, D), generator=g, device="cuda") * 2.0 ** -round(torch.tensor(D ** 0.5).log2().item())).to(dtype)
    check(x, w, target, dloss, dlse, both(x, w, target, dloss, dlse))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [20, 300])
def test_rows_of_weights_far_apart(T, dtype):
    # Weights down to 2^-20 of the largest: what float16 cannot hold of a small row's probabilities is below 2^-39 of
    # the largest weight, as the bounds have it.
    x, w, target, dloss, dlse = inputs(T, 3000, 64, dtype, seed=23)
    by = 2.0 ** -(torch.arange(T, device="cuda") % 21)
    check(x, w, target, dloss * by, dlse * by, both(x, w, target, dloss * by, dlse * by))
    loss, lse = pv.cross_entropy(x, w, target)
    # Rows of one weight are as exact by themselves as among others: a small row's largest gradients, its target's, are held.
    dx, _ = pv.cross_entropy_backward(dloss * by, x, w, target, lse)
    z = x.double() @ w.double().T
    p = torch.softmax(z, -1)
    some = target >= 0
    p.scatter_add_(1, target.clamp_min(0)[:, None], -torch.ones((T, 1), dtype=torch.float64, device="cuda"))
    want = p[some] @ w.double()
    small = torch.finfo(dtype).smallest_normal
    got = dx[some].double() / (dloss * by)[some].double()[:, None]
    # (Below float16's normal numbers dx itself has fixed steps.)
    keep = (want.abs() * (dloss * by)[some].double()[:, None]).amax(-1) >= 2.0 ** 8 * small
    assert keep.any() and ((got - want)[keep].norm(dim=-1) <= 2.0 ** -6 * want[keep].norm(dim=-1)).all()
