"""Per-head normalisation and rotation of queries and keys against 64 bits."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")
import _tokens as ref  # noqa: E402

pytestmark = pytest.mark.gpu

EPS = 1e-6
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def make(rows, H, Hk, D, axes, dtype, seed=0, far=496):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return (2.0 * torch.randn(s, generator=g, device="cuda")).to(dtype)

    q, k, dq, dk = normal(rows, H, D), normal(rows, Hk, D), normal(rows, H, D), normal(rows, Hk, D)
    wq, wk = (1.0 + 0.2 * torch.randn((D,), generator=g, device="cuda") for _ in range(2))
    pos = torch.randint(-far, far, (rows, axes), generator=g, device="cuda", dtype=torch.int32)
    return q, k, dq, dk, wq, wk, pos, pv.rope_frequencies(D, axes, device="cuda")


def close(got, want, mag, dtype, name):
    # One rounding to the storage type; some ten 32-bit operations on terms of size `mag`.
    ref.within(got, want, 2 * ref.UNIT[dtype] * want.abs() + 2.0 ** -19 * mag + (2.0 ** -24 if dtype is torch.float16 else 0.0), name)


def close_weight(got, want, mag, rows, name):
    # A 32-bit sum over rows and heads of terms that are good to 2^-19.
    ref.within(got, want, (2.0 ** -19 + 2.0 ** -24 * (rows ** 0.5 + 64)) * mag + 1e-30, name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H,Hk,D,axes", [(1, 8, 2, 64, 1), (1, 1, 1, 16, 3), (2, 3, 1, 48, 2), (33, 4, 4, 32, 3),
                                              (257, 16, 4, 128, 2), (1001, 5, 5, 96, 1), (129, 2, 1, 256, 3),
                                              (5003, 8, 8, 64, 2)])
def test_forward_and_backward(rows, H, Hk, D, axes, dtype):
    q, k, dq, dk, wq, wk, pos, freq = make(rows, H, Hk, D, axes, dtype)
    oq, ok = pv.qk_norm_rope(q, k, wq, wk, pos, freq, EPS)
    gq, gk, gwq, gwk = pv.qk_norm_rope_backward(dq, dk, q, k, wq, wk, pos, freq, EPS)
    for x, w, dy, y, gx, gw, n in ((q, wq, dq, oq, gq, gwq, "q"), (k, wk, dk, ok, gk, gwk, "k")):
        want, mag = ref.rope(x, w, pos, freq, EPS)
        close(y, want, mag, dtype, n)
        dx, mx, dw, mw = ref.rope_backward(dy, x, w, pos, freq, EPS)
        close(gx, dx, mx, dtype, "d" + n)
        close_weight(gw, dw, mw, rows * x.shape[1], "dw" + n)


def test_long_positions():
    q, k, dq, dk, wq, wk, pos, freq = make(300, 2, 2, 64, 1, torch.float32, far=1 << 20)
    oq, _ = pv.qk_norm_rope(q, k, wq, wk, pos, freq, EPS)
    close(oq, *ref.rope(q, wq, pos, freq, EPS), torch.float32, "q")


def test_slices_of_a_projection_and_of_coordinates():
    # Queries and keys inside one [rows, (H + 2 Hk) D] projection, positions the
    # (z, y, x) of the voxelizer's (batch, z, y, x).
    rows, H, Hk, D = 211, 6, 2, 64
    _, _, _, _, wq, wk, _, freq = make(1, H, Hk, D, 3, torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn((rows, (H + 2 * Hk), D), generator=g, device="cuda").to(torch.bfloat16)
    coords = torch.randint(0, 400, (rows, 4), generator=g, device="cuda", dtype=torch.int32)
    q, k = qkv[:, :H], qkv[:, H:H + Hk]
    kept = qkv.clone()
    oq, ok = pv.qk_norm_rope(q, k, wq, wk, coords[:, 1:], freq, EPS)
    assert torch.equal(qkv, kept)
    for x, w, y in ((q, wq, oq), (k, wk, ok)):
        close(y, *ref.rope(x, w, coords[:, 1:], freq, EPS), torch.bfloat16, "slice")
    # The same in place: only the queries and keys change.
    pv.qk_norm_rope(q, k, wq, wk, coords[:, 1:], freq, EPS, out=(q, k))
    assert torch.equal(q, oq) and torch.equal(k, ok) and torch.equal(qkv[:, H + Hk:], kept[:, H + Hk:])


def test_heads_first_layout_and_no_rows():
    q, k, dq, dk, wq, wk, pos, freq = make(77, 4, 2, 32, 2, torch.float16)
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert not qt.is_contiguous()
    a, b = pv.qk_norm_rope(q, k, wq, wk, pos, freq, EPS), pv.qk_norm_rope(qt, k, wq, wk, pos, freq, EPS)
    assert torch.equal(a[0], b[0])
    oq, ok = pv.qk_norm_rope(q[:0], k[:0], wq, wk, pos[:0], freq, EPS)
    assert oq.shape == (0, 4, 32) and ok.shape == (0, 2, 32)
    *_, gwq, gwk = pv.qk_norm_rope_backward(dq[:0], dk[:0], q[:0], k[:0], wq, wk, pos[:0], freq, EPS)
    assert not gwq.any() and not gwk.any()


def test_same_bits_every_time_and_on_another_stream():
    args = make(40001, 8, 8, 64, 2, torch.bfloat16)
    q, k, dq, dk, wq, wk, pos, freq = args
    first = pv.qk_norm_rope_backward(dq, dk, q, k, wq, wk, pos, freq, EPS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = pv.qk_norm_rope_backward(dq, dk, q, k, wq, wk, pos, freq, EPS)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))


def test_gradient_against_differences():
    q, k, dq, dk, wq, wk, pos, freq = make(9, 2, 1, 32, 2, torch.float32, seed=5)
    gq, gk, gwq, gwk = pv.qk_norm_rope_backward(dq, dk, q, k, wq, wk, pos, freq, EPS)

    def loss(q, k, wq, wk):
        return ((ref.rope(q, wq, pos, freq, EPS)[0] * dq.double()).sum()
                + (ref.rope(k, wk, pos, freq, EPS)[0] * dk.double()).sum())

    at = [t.double() for t in (q, k, wq, wk)]
    g = torch.Generator(device="cuda").manual_seed(6)
    for n, grad in enumerate((gq, gk, gwq, gwk)):
        way = torch.randn(at[n].shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-5
        up, down = list(at), list(at)
        up[n], down[n] = at[n] + step * way, at[n] - step * way
        slope = (loss(*up) - loss(*down)) / (2 * step)
        # Central differences: step^2 of the third derivative (here below 1e-8 of the
        # gradient's size) and 1e-16 / step of the loss; the gradient itself is in 32 bits.
        size = (grad.double().abs() * way.abs()).sum()
        assert abs((grad.double() * way).sum() - slope) <= 1e-5 * size


def test_refusals():
    q, k, dq, dk, wq, wk, pos, freq = make(10, 4, 2, 32, 2, torch.bfloat16)
    ok = (q, k, wq, wk, pos, freq)

    def call(error, **change):
        names = ("q", "k", "wq", "wk", "pos", "freq")
        with pytest.raises(error):
            pv.qk_norm_rope(*[change.get(n, v) for n, v in zip(names, ok)], EPS)

    call(TypeError, q=q.double(), k=k.double())
    call(TypeError, k=k.float())
    call(TypeError, wq=wq.bfloat16())
    call(TypeError, pos=pos.long())
    call(ValueError, q=q[:, :, 0])
    call(ValueError, k=k[:9])
    call(ValueError, pos=pos[:9])
    call(ValueError, pos=torch.zeros((10, 4), dtype=torch.int32, device="cuda"))
    call(ValueError, freq=freq[:8])
    call(ValueError, q=q.cpu(), k=k.cpu())
    call(ValueError, q=torch.zeros((10, 4, 40), dtype=torch.bfloat16, device="cuda")[:, :, 1:33])
    with pytest.raises(pv.PVError) as e:  # head_dim 24 is no multiple of 16
        t = torch.zeros((10, 1, 24), dtype=torch.bfloat16, device="cuda")
        w = torch.ones((24,), device="cuda")
        pv.qk_norm_rope(t, t, w, w, pos, torch.ones((12,), device="cuda"), EPS)
    assert e.value.status == -1
    with pytest.raises(pv.PVError):
        pv.qk_norm_rope(q, k, wq, wk, pos, freq, -1.0)
