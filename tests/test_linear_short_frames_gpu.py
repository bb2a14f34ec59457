"""Linear attention: what a short frame gives does not depend on the frames beside it."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import lidar_point_cloud_gb300 as pv  # noqa: E402
from test_linear_gpu import U, inputs, reference  # noqa: E402

pytestmark = pytest.mark.gpu

# Frames of 1, 128, 2, 0, 127, 40 and 1 tokens; between them those of several chunks of 128.
LENGTHS = [1, 129, 128, 2, 700, 0, 127, 40, 5000, 1]


def offsets(lengths):
    return [sum(lengths[:i]) for i in range(len(lengths) + 1)]


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("D", [40, 64, 128])
def test_short_frames_beside_long_ones_lose_nothing_but_the_outputs_rounding(D, reverse):
    # From no state: scores of a frame of one chunk are rounded twice, to what is left of them (2^-8 of 2^-8), and
    # sums are in 32 bits.
    off, H = offsets(LENGTHS), 8
    q, k, v, do, _, _, d = inputs(off, H, D, seed=3)
    out, _ = pv.linear_attention(q, k, v, d, off, reverse=reverse)
    dq, dk, dv, _ = pv.linear_attention_backward(do, None, q, k, v, d, off, reverse=reverse)
    values, mags = reference(q, k, v, d, off, D ** -0.5, None, reverse, do, None)
    for name, got in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        for f, n in enumerate(LENGTHS):
            if not 0 < n <= 128:
                continue
            rows = slice(off[f], off[f + 1])
            want = values[name][rows]
            slack = 1.01 * U * want.abs() + (2.0 ** -16 + 2.0 ** -20) * mags[name][rows] + 1e-37
            worst = ((got[rows].double() - want).abs() - slack).max().item()
            assert worst <= 0, (name, n, worst)


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("D", [32, 128])
def test_short_frames_have_the_bits_that_they_have_alone(D, given):
    off, H = offsets(LENGTHS), 3
    q, k, v, do, s0, dl, d = inputs(off, H, D, seed=4)
    s0, dl = (s0, dl) if given else (None, None)
    got = [*pv.linear_attention(q, k, v, d, off, state=s0), *pv.linear_attention_backward(do, dl, q, k, v, d, off, state=s0)]
    for f, n in enumerate(LENGTHS):
        if n > 128:
            continue
        rows = slice(off[f], off[f + 1])
        own = [t[rows].clone() for t in (q, k, v, do)]
        s, g = (None, None) if not given else (s0[f: f + 1].clone(), dl[f: f + 1].clone())
        alone = [*pv.linear_attention(*own[:3], d, [0, n], state=s),
                 *pv.linear_attention_backward(own[3], g, *own[:3], d, [0, n], state=s)]
        for x, (a, b) in enumerate(zip(got, alone)):
            assert torch.equal(a[f: f + 1] if a.dim() == 4 else a[rows], b), (n, x)
