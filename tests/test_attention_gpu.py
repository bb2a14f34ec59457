"""Attention inside frames, forward and backward, against 64 bits."""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")
import _tokens as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]


def offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return off


def make(lq, lk, H, Hk, D, dtype, axes=0, seed=0, loud=1.0):
    qo, ko = offsets(lq), offsets(lk)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g, device="cuda")

    t = {"q": (loud * normal(qo[-1], H, D)).to(dtype), "k": normal(ko[-1], Hk, D).to(dtype),
         "v": normal(ko[-1], Hk, D).to(dtype), "dout": normal(qo[-1], H, D).to(dtype), "qo": qo, "ko": ko}
    t["how"] = {"scale": D ** -0.5}
    if axes:
        t["how"].update(slopes=torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda"),
                        qpos=torch.randint(-60, 60, (qo[-1], axes), generator=g, device="cuda", dtype=torch.int32),
                        kpos=torch.randint(-60, 60, (ko[-1], axes), generator=g, device="cuda", dtype=torch.int32))
    return t


def own(how):
    how = dict(how)
    if "qpos" in how:
        how["q_positions"], how["k_positions"] = how.pop("qpos"), how.pop("kpos")
    return how


def check(t, lse_slack=2.0 ** -16, **more):
    how = {**t["how"], **more}
    want, slack = ref.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], dout=t["dout"], **how)
    o, lse = pv.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], return_lse=True, **own(how))
    ref.within(o, want["out"], slack["out"], "out")
    assert torch.equal(lse.isinf(), want["lse"].isinf()) and not lse.isnan().any()
    live = ~want["lse"].isinf()
    ref.within(lse[live], want["lse"][live], lse_slack * (1.0 + want["lse"][live].abs()), "lse")
    assert torch.equal(o, pv.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], **own(how)))
    grads = pv.attention_backward(t["dout"], t["q"], t["k"], t["v"], o, lse, t["qo"], t["ko"], **own(how))
    for got, n in zip(grads, ("dq", "dk", "dv")):
        ref.within(got, want[n], slack[n], n)
    return o, lse, grads


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lq,lk,H,Hk,D", [
    ([1], [1], 1, 1, 8), ([1], [300], 8, 2, 64), ([300], [1], 2, 1, 64), ([127, 128, 129], [129, 127, 128], 2, 2, 32),
    ([64, 65], [200, 63], 4, 1, 128), ([5, 0, 70, 3], [9, 4, 0, 130], 3, 3, 40), ([257], [511], 4, 2, 72),
    ([2, 2, 2], [1000, 130, 1], 16, 2, 128), ([385], [385], 5, 1, 64), ([700], [700], 6, 2, 24)])
def test_plain(lq, lk, H, Hk, D, dtype):
    check(make(lq, lk, H, Hk, D, dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lq,lk,prefix", [([130], [130], None), ([300, 40], [300, 40], [100, 0]), ([100], [400], None),
                                          ([400], [100], None), ([1, 1], [500, 3], [2, 2]), ([260], [260], [10 ** 9]),
                                          ([200, 50], [10, 0], [3, 5]), ([513], [513], [129])])
def test_causal_and_prefix(lq, lk, prefix, dtype):
    t = make(lq, lk, 4, 2, 64, dtype)
    check(t, causal=True, prefix=prefix)


def test_rows_that_see_nothing():
    t = make([300, 5], [40, 0], 2, 2, 64, torch.bfloat16)
    o, lse, (dq, dk, dv) = check(t, causal=True)
    assert not o[:260].any() and not o[300:].any() and not dq[:260].any() and not dq[300:].any()
    assert (lse[:, :260] == -math.inf).all() and (lse[:, 300:] == -math.inf).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("axes", [1, 2, 3])
def test_distance(axes, dtype):
    check(make([150, 33], [260, 129], 4, 2, 64, dtype, axes=axes))
    check(make([200], [200], 8, 8, 32, dtype, axes=axes), causal=True, prefix=[20])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [32, 128])
def test_cap(D, dtype):
    check(make([150, 33], [260, 129], 4, 2, D, dtype, loud=8.0), cap=10.0)
    check(make([200], [200], 4, 1, D, dtype, axes=2, loud=20.0), cap=30.0, causal=True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scores_that_are_far_apart(dtype):
    # Scores of hundreds: one key takes a row; maxima that rise along the row.
    t = make([140], [900], 2, 1, 64, dtype, loud=1.0)
    t["k"] *= torch.linspace(0.1, 20.0, 900, device="cuda")[:, None, None].to(dtype)
    t["q"] *= 6.0
    check(t, lse_slack=2.0 ** -15)


def test_other_frames_may_hold_anything():
    t = make([100, 60, 77], [90, 200, 50], 2, 2, 64, torch.bfloat16)
    o, lse, grads = check(t)
    u = {n: (x.clone() if isinstance(x, torch.Tensor) else x) for n, x in t.items()}
    for n, lo, hi in (("q", 100, 160), ("dout", 100, 160), ("k", 90, 290), ("v", 90, 290)):
        u[n][lo:hi] = float("nan")
        u[n][lo + 1:hi:2] = float("inf")
    o2, lse2 = pv.attention(u["q"], u["k"], u["v"], u["qo"], u["ko"], return_lse=True)
    g2 = pv.attention_backward(u["dout"], u["q"], u["k"], u["v"], o2, lse2, u["qo"], u["ko"])
    for a, b, rows in ((o, o2, (100, 160)), (grads[0], g2[0], (100, 160)), (grads[1], g2[1], (90, 290)), (grads[2], g2[2], (90, 290))):
        assert torch.equal(a[:rows[0]], b[:rows[0]]) and torch.equal(a[rows[1]:], b[rows[1]:])


def test_slices_of_a_projection():
    lens, H, Hk, D = [70, 130], 4, 2, 64
    off = offsets(lens)
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((off[-1], H + 2 * Hk, D), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    a = pv.attention(q, k, v, off, off)
    b = pv.attention(q.contiguous(), k.contiguous(), v.contiguous(), off, off)
    assert torch.equal(a, b)
    heads_first = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    assert torch.equal(a, pv.attention(*heads_first, off, off))
    one = k[:, :1].expand(-1, Hk, -1)  # one key head seen as several
    assert torch.equal(pv.attention(q, one, v, off, off), pv.attention(q, one.contiguous(), v, off, off))


def test_a_cache_past_32_bit_offsets():
    # 70,000 keys, 32,768 elements apart: the last lie past 2^31 elements and 2^32 bytes.
    H, Hk, D, n = 8, 1, 64, 70000
    cache = torch.empty((n, 2, 16384), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (cache[:, i, :D].unflatten(1, (Hk, D)) for i in range(2))
    k.copy_(torch.randn((n, Hk, D), generator=g, device="cuda"))
    v.copy_(torch.randn((n, Hk, D), generator=g, device="cuda"))
    q = (3.0 * torch.randn((2, H, D), generator=g, device="cuda")).to(torch.bfloat16)
    want, slack = ref.attention(q, k, v, [0, 2], [0, n], D ** -0.5)
    ref.within(pv.attention(q, k, v, [0, 2], [0, n]), want["out"], slack["out"], "out")


def test_same_bits_every_time_and_on_another_stream():
    t = make([900, 20], [1500, 700], 4, 2, 64, torch.bfloat16, axes=2)

    def go():
        o, lse = pv.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], return_lse=True, **own(t["how"]))
        return (o, lse, *pv.attention_backward(t["dout"], t["q"], t["k"], t["v"], o, lse, t["qo"], t["ko"], **own(t["how"])))

    first = go()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = go()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))


def test_one_query_on_two_streams():
    runs = [make([1, 1], [5000, 3000], 8, 2, 128, torch.bfloat16, seed=s) for s in (1, 2)]
    want = [pv.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"]) for t in runs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in runs], []
    for _ in range(4):
        for s, t in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(pv.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[n % 2]) for n, g in enumerate(got))


def test_gradient_against_differences():
    t = make([20, 6], [17, 30], 2, 1, 16, torch.float16, axes=2, seed=4)
    how = {**t["how"], "cap": 4.0}
    o, lse = pv.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], return_lse=True, **own(how))
    grads = pv.attention_backward(t["dout"], t["q"], t["k"], t["v"], o, lse, t["qo"], t["ko"], **own(how))

    at = [t[n].double() for n in "qkv"]
    g = torch.Generator(device="cuda").manual_seed(5)

    def loss(q, k, v):
        return (ref.attention(q, k, v, t["qo"], t["ko"], **how)[0]["out"] * t["dout"].double()).sum()

    for n, grad in enumerate(grads):
        way = torch.randn(at[n].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = list(at), list(at)
        up[n], down[n] = at[n] + 1e-5 * way, at[n] - 1e-5 * way
        slope = (loss(*up) - loss(*down)) / 2e-5
        # A float16 gradient: 2^-11 an element on top of the products' roundings, which
        # average out along a random direction; eight such units of the sum of magnitudes.
        assert abs((grad.double() * way).sum() - slope) <= 8 * 2.0 ** -11 * (grad.double().abs() * way.abs()).sum()


def test_refusals():
    t = make([10, 20], [30, 40], 4, 2, 64, torch.bfloat16, axes=2)
    q, k, v, qo, ko = (t[n] for n in ("q", "k", "v", "qo", "ko"))
    pos = t["how"]["kpos"]

    def refuse(error, *args, **how):
        with pytest.raises(error) as e:
            pv.attention(*args, **how)
        return e.value

    refuse(TypeError, q.float(), k.float(), v.float(), qo, ko)
    refuse(TypeError, q, k.half(), v.half(), qo, ko)
    refuse(ValueError, q, k, v[:, :1], qo, ko)
    refuse(ValueError, q[:, :3], k, v, qo, ko)
    refuse(ValueError, q, k, v, [0, 10, 31], ko)
    refuse(ValueError, q, k, v, qo, [0, 70])
    refuse(ValueError, q.cpu(), k.cpu(), v.cpu(), qo, ko)
    refuse(ValueError, q, k, v, qo, ko, slopes=t["how"]["slopes"])
    refuse(ValueError, q, k, v, qo, ko, slopes=t["how"]["slopes"], q_positions=t["how"]["qpos"], k_positions=pos[:, :1])
    refuse(ValueError, q, k, v, qo, ko, prefix=[1, 1])
    refuse(ValueError, q, k, v, qo, ko, causal=True, prefix=[1])
    wide = torch.zeros((30, 4, 136), dtype=torch.bfloat16, device="cuda")
    assert refuse(pv.PVError, wide, wide, wide, [0, 30], [0, 30]).status == -1  # head_dim over 128
    assert refuse(pv.PVError, q, k, v, qo, ko, scale=-1.0).status == -1
    assert refuse(pv.PVError, q, k, v, qo, ko, cap=float("nan")).status == -1
    assert refuse(pv.PVError, q, k, v, qo, ko, causal=True, prefix=[1, -1]).status == -1
    assert refuse(pv.PVError, q, k, v, [0, 31, 30], ko).status == -1
    o, lse = pv.attention(q, k, v, qo, ko, return_lse=True)
    with pytest.raises(ValueError):
        pv.attention_backward(t["dout"], q, k, v, o, lse[:2], qo, ko)
