"""Gradients of attention from loud, quiet and overflowed gradients of its output."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")
import _tokens as ref  # noqa: E402
from test_attention_gpu import DTYPES, check, make  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("loud", [2.0 ** -10, 16.0, 64.0, 1024.0])
def test_gradients_of_any_size(loud, dtype):
    # (Unit-variance keys and values: the largest gradients stay inside float16.)
    for how in ({}, {"cap": 10.0}, {"causal": True}):
        t = make([150, 33], [260, 129], 4, 2, 64, dtype, axes=2 if not how else 0, loud=2.0)
        t["dout"] = (t["dout"].float() * loud).to(dtype)
        check(t, **how)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_gradient_that_fits_though_its_score_gradient_is_large(dtype, D):
    # One query, two keys, k = v = +-1, dout 64: the scores' gradients are +-32 D, dq is 64 D / sqrt(D).
    one = torch.ones((1, 1, D), dtype=dtype, device="cuda")
    q, k, do = 0 * one, torch.cat([one, -one]), 64 * one
    o, lse = pv.attention(q, k, k, [0, 1], [0, 2], return_lse=True)
    dq, dk, dv = pv.attention_backward(do, q, k, k, o, lse, [0, 1], [0, 2])
    want = 64.0 * D ** 0.5
    assert torch.equal(o, 0 * one) and not dk.any()
    assert (dv == 32.0).all()
    assert ((dq.double() - want).abs() <= 2 * ref.UNIT[dtype] * want).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_frames_of_very_different_gradients(dtype):
    # A frame's gradients are as good as if it were alone, whatever the other frames hold.
    t = make([70, 90], [80, 60], 2, 1, 64, dtype)
    t["dout"][70:] = (t["dout"][70:].float() * 512.0).to(dtype)
    _, _, grads = check(t)
    one = {n: t[n][:m].contiguous() for n, m in (("q", 70), ("dout", 70), ("k", 80), ("v", 80))}
    o, lse = pv.attention(one["q"], one["k"], one["v"], [0, 70], [0, 80], return_lse=True)
    alone = pv.attention_backward(one["dout"], one["q"], one["k"], one["v"], o, lse, [0, 70], [0, 80])
    want, slack = ref.attention(one["q"], one["k"], one["v"], [0, 70], [0, 80], 64 ** -0.5, dout=one["dout"])
    for n, both, a in zip(("dq", "dk", "dv"), grads, alone):
        ref.within(a, want[n], slack[n], n)
        ref.within(both[:len(a)], want[n], slack[n], n)


@pytest.mark.parametrize("dtype", DTYPES)
def test_other_frames_may_hold_anything(dtype):
    t = make([100, 60, 77], [90, 200, 50], 2, 2, 64, dtype)
    o, lse, grads = check(t)
    u = {n: (x.clone() if isinstance(x, torch.Tensor) else x) for n, x in t.items()}
    for n, lo, hi in (("q", 100, 160), ("dout", 100, 160), ("k", 90, 290), ("v", 90, 290)):
        u[n][lo:hi] = float("nan")
        u[n][lo + 1:hi:2] = float("inf")
    o2, lse2 = pv.attention(u["q"], u["k"], u["v"], u["qo"], u["ko"], return_lse=True)
    g2 = pv.attention_backward(u["dout"], u["q"], u["k"], u["v"], o2, lse2, u["qo"], u["ko"])
    for a, b, lo, hi in ((o, o2, 100, 160), (grads[0], g2[0], 100, 160), (grads[1], g2[1], 90, 290), (grads[2], g2[2], 90, 290)):
        assert torch.equal(a[:lo], b[:lo]) and torch.equal(a[hi:], b[hi:])


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_gradient_row_that_overflowed_leaves_the_other_queries_alone(dtype):
    # What a loss scale that is too high makes: the row's own dq is not finite, the others' are as before.
    t = make([60], [90], 2, 1, 64, dtype)
    _, _, (dq, _, _) = check(t)
    t["dout"][17] = float("inf")
    o, lse = pv.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], return_lse=True)
    dq2, dk2, dv2 = pv.attention_backward(t["dout"], t["q"], t["k"], t["v"], o, lse, t["qo"], t["ko"])
    keep = torch.arange(60, device="cuda") != 17
    assert torch.equal(dq[keep], dq2[keep]) and not torch.isfinite(dq2[17]).any()
    assert not torch.isfinite(dk2).any() and not torch.isfinite(dv2).any()


@pytest.mark.parametrize("cap", [0.0, 10.0])
def test_rows_of_very_different_gradients(cap):
    # A few loud rows beside quiet ones, 2^24 apart: the quiet rows' dq is as good as theirs alone would be.
    # Two roundings to float16 of 2^-12 and sums that average them out: 2^-9 of a row's norm leaves room.
    t = make([60], [90], 2, 1, 64, torch.float16, loud=2.0)
    loud = torch.zeros(60, dtype=torch.bool, device="cuda")
    loud[[3, 17, 40]] = True
    t["dout"] = (t["dout"].float() * torch.where(loud, 2.0 ** 13, 2.0 ** -11)[:, None, None]).half()
    _, _, (dq, _, _) = check(t, cap=cap)
    want = ref.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], cap=cap, dout=t["dout"], **t["how"])[0]["dq"]
    off = ((dq.double() - want).norm(dim=-1) - 2.0 ** -25 * 8).clamp_min(0)  # (64 roundings of numbers near 2^-14)
    assert (off / want.norm(dim=-1)).max() < 2.0 ** -9


def test_probabilities_of_millions_of_keys():
    # Queries that see every key alike: dv of every key is the mean of dout's rows, times queries
    # over keys.  A probability of 2^-23 and the result are each rounded by 2^-12 at most.
    n, rows, D = 8_400_001, 4096, 8
    k, q = torch.zeros((n, 1, D), dtype=torch.float16, device="cuda"), torch.zeros((rows, 1, D), dtype=torch.float16, device="cuda")
    v = torch.randn((n, 1, D), device="cuda").half()
    do = torch.full((rows, 1, D), 512.0, dtype=torch.float16, device="cuda")
    o, lse = pv.attention(q, k, v, [0, rows], [0, n], return_lse=True)
    _, _, dv = pv.attention_backward(do, q, k, v, o, lse, [0, rows], [0, n])
    want = 512.0 * rows / n
    # (32 bits add 2^-22 times lse, 16, to a probability.)
    assert float((dv.double() / want - 1.0).abs().max()) < 2 * 2.0 ** -12 + 16 * 2.0 ** -21
