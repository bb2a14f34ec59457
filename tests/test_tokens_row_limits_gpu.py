"""The token operators on row counts whose index arithmetic comes to 2^31."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")
import _tokens as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB of device memory")
    yield
    torch.cuda.empty_cache()


def test_attention_of_more_than_two_to_the_31_queries_and_heads():
    # 2^28 queries and some of eight heads that share a key head: rows of a block count both.
    n = (1 << 28) + 1000
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.empty((n, 8, 8), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    k, v = (torch.randn((5, 1, 8), generator=g, device="cuda").bfloat16() for _ in range(2))
    out = torch.full_like(q, float("nan"))
    pv.attention(q, k, v, [0, 3, n], [0, 2, 5], out=out)
    for a, b in ((0, 3), (3, 1003), ((1 << 27) - 500, (1 << 27) + 500), (n - 3000, n)):
        keys = slice(0, 2) if b == 3 else slice(2, 5)
        rows, nk = b - a, 2 if b == 3 else 3
        want, slack = ref.attention(q[a:b], k[keys], v[keys], [0, rows], [0, nk], 8 ** -0.5)
        ref.within(out[a:b], want["out"], slack["out"], f"rows {a} to {b}")
    assert not any(part.isnan().any() for part in out.split(1 << 25))


def test_rotation_of_almost_two_to_the_31_rows():
    rows, D = (1 << 31) - 300, 16
    one, dy = (torch.randn((1, 1, D), device="cuda").half() for _ in range(2))
    w, freq = torch.ones(D, device="cuda"), pv.rope_frequencies(D, device="cuda")
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")[:, None] % 1000
    # (No keys, and one query seen as many: the outputs are what is large.)
    q, d = one.expand(rows, 1, D), dy.expand(rows, 1, D)
    parts = [slice(0, 1000), slice(rows - 1000, rows)]

    def small(p):
        return pv.qk_norm_rope(q[p], q[p, :0], w, w, pos[p], freq)[0]

    def small_back(p):
        return pv.qk_norm_rope_backward(d[p], d[p, :0], q[p], q[p, :0], w, w, pos[p], freq)[0]

    out, _ = pv.qk_norm_rope(q, q[:, :0], w, w, pos, freq)
    assert all(torch.equal(out[p], small(p)) for p in parts)
    del out
    torch.cuda.empty_cache()
    dq, *_ = pv.qk_norm_rope_backward(d, d[:, :0], q, q[:, :0], w, w, pos, freq)
    assert all(torch.equal(dq[p], small_back(p)) for p in parts)
