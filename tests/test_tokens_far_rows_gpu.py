"""The token operators on rows whose offsets pass 2^31 elements (a few GB a tensor)."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")

pytestmark = pytest.mark.gpu

ROWS = 17_000_001  # of 128 elements: 2.18e9


@pytest.fixture(scope="module")
def rows():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(0)
    x, y = (torch.empty((ROWS, 128), dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    yield x, y
    del x, y
    torch.cuda.empty_cache()


def test_attention_over_one_long_cache(rows):
    k, v = (t.view(ROWS, 1, 128) for t in rows)
    q, do = (torch.randn((2, 2, 128), device="cuda").bfloat16() for _ in range(2))
    qo, ko = [0, 1, 2], [0, 5, ROWS]
    o, lse = pv.attention(q, k, v, qo, ko, return_lse=True)
    scale = 128 ** -0.5
    total = torch.zeros((2, 1), dtype=torch.float64, device="cuda")
    acc = torch.zeros((2, 128), dtype=torch.float64, device="cuda")
    for a in range(5, ROWS, 1_000_000):  # scores are a few units: their exponentials need no maximum
        b = min(ROWS, a + 1_000_000)
        w = torch.exp(q[1].double() @ k[a:b, 0].double().T * scale)
        total += w.sum(1, keepdim=True)
        acc += w @ v[a:b, 0].double()
    want = acc / total
    # Two roundings to the storage type, of 2^-9 each, of the probabilities and of the result.
    assert float((o[1].double() - want).norm() / want.norm()) < 2.0 ** -8
    assert float((lse[:, 1].double() - total.log()[:, 0]).abs().max()) < 2.0 ** -18
    dq, dk, dv = pv.attention_backward(do, q, k, v, o, lse, qo, ko)
    a = ROWS - 1000
    p = torch.exp(q[1].double() @ k[a:, 0].double().T * scale) / total
    ds = p * (do[1].double() @ v[a:, 0].double().T - (do[1].double() * want).sum(1, keepdim=True))
    for got, ref in ((dv, p.T @ do[1].double()), (dk, ds.T @ q[1].double() * scale)):
        assert float((got[a:, 0].double() - ref).norm() / ref.norm()) < 2.0 ** -8


def test_rotation_of_the_last_rows(rows):
    k = rows[0].view(ROWS, 2, 64)
    w, freq = torch.ones(64, device="cuda"), pv.rope_frequencies(64, 1, device="cuda")
    pos = torch.arange(ROWS, dtype=torch.int32, device="cuda")[:, None]
    a = ROWS - 1000
    far = pv.qk_norm_rope(k, k[:, :1], w, w, pos, freq)
    near = pv.qk_norm_rope(k[a:].clone(), k[a:, :1].clone(), w, w, pos[a:].clone(), freq)
    assert all(torch.equal(f[a:], n) for f, n in zip(far, near))


def test_recurrence_along_one_long_frame(rows):
    x, gate = rows
    h, last, states = pv.gated_scan(x, gate, [0, ROWS], return_states=True)
    dx, dgate, _ = pv.gated_scan_backward(x, None, x, gate, states, [0, ROWS])
    # The gates are half open: 300 steps before the compared ones forget what was there.
    a, b = ROWS - 1300, ROWS - 1000
    X, Z = x[a:].double().cpu(), torch.sigmoid(gate[a:].double().cpu())
    s, want, before = torch.zeros(128, dtype=torch.float64), [], []
    for t in range(ROWS - a):
        before.append(s)
        s = (1 - Z[t]) * s + Z[t] * X[t]
        want.append(s)
    want, before, e = torch.stack(want), torch.stack(before), torch.zeros(128, dtype=torch.float64)
    grad_x, grad_g = torch.empty_like(want), torch.empty_like(want)
    for t in reversed(range(ROWS - a)):
        e = X[t] + e
        grad_x[t], grad_g[t] = e * Z[t], e * (X[t] - before[t]) * Z[t] * (1 - Z[t])
        e = e * (1 - Z[t])
    for got, ref in ((h, want), (dx, grad_x), (dgate, grad_g)):
        got, ref = got[b:].double().cpu(), ref[b - a:]
        assert float(((got - ref).abs() - 2.0 ** -8 * ref.abs()).max()) < 2.0 ** -14
    assert float((last[0].double().cpu() - want[-1]).abs().max()) < 2.0 ** -14
