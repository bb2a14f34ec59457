"""Attention on tensors expanded over their rows, as the gradient of a sum over rows is, or over their
heads, and on single rows and heads."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")
from lidar_point_cloud_gb300 import _binding, _tokens  # noqa: E402
from test_attention_gpu import make  # noqa: E402

pytestmark = pytest.mark.gpu


def run(t):
    o, lse = pv.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], return_lse=True)
    return (o, lse, *pv.attention_backward(t["dout"], t["q"], t["k"], t["v"], o, lse, t["qo"], t["ko"]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lq,lk", [([1], [1]), ([300, 5], [260, 40]), ([2], [700])])
@pytest.mark.parametrize("names", [("q",), ("k",), ("v",), ("dout",), ("q", "k", "v", "dout")])
def test_rows_expanded_from_one(names, lq, lk, dtype):
    t = make(lq, lk, 4, 2, 64, dtype)
    for n in names:
        t[n] = t[n][:1].expand(len(t[n]), -1, -1)
        assert len(t[n]) == 1 or t[n].stride(0) == 0
    dense = {n: (x.contiguous() if isinstance(x, torch.Tensor) else x) for n, x in t.items()}
    assert all(torch.equal(a, b) for a, b in zip(run(t), run(dense)))


def test_gradients_that_autograd_expands():
    # out.sum(0) hands back strides (0, D, 1), out.sum() (0, 0, 0).
    t = make([70, 130], [90, 60], 4, 2, 64, torch.bfloat16)
    for sum_of in (lambda o: o.sum(0) * t["dout"][0], lambda o: o.sum()):
        o = torch.zeros_like(t["q"]).requires_grad_()
        g, = torch.autograd.grad(sum_of(o).sum(), o)
        got = run({**t, "dout": g})
        assert all(torch.equal(a, b) for a, b in zip(got, run({**t, "dout": g.contiguous()})))


def test_the_library_refuses_what_its_tiles_cannot_read():
    t = make([20], [30], 2, 2, 64, torch.bfloat16)
    lib, h = pv.load(), {n: _tokens._heads(t[n], n) for n in ("q", "k", "v", "dout")}
    p, alive = _tokens._attention_params(t["q"], t["k"], t["v"], t["qo"], t["ko"], None, 0.0, None, None, None, False, None)
    o, lse = torch.zeros_like(t["q"]), torch.zeros((2, 20), device="cuda")
    grads = [torch.zeros_like(t[n]) for n in ("q", "k", "v")]
    ho, hg = _tokens._heads(o, "out"), [_tokens._heads(g, "gradient") for g in grads]

    def flat(x, heads=False):
        return _binding.Heads(x.data, x.row_stride if heads else 0, 0 if heads else x.head_stride)

    for n in ("q", "k", "v"):
        x = {**h, n: flat(h[n])}
        assert lib.pv_attention(p, x["q"], x["k"], x["v"], ho, None, None) == -1
    for bad in (flat(ho), flat(ho, heads=True)):
        assert lib.pv_attention(p, h["q"], h["k"], h["v"], bad, None, None) == -1
    for n in ("q", "k", "v", "dout"):
        x = {**h, n: flat(h[n])}
        assert lib.pv_attention_backward(p, x["dout"], x["q"], x["k"], x["v"], ho, lse.data_ptr(), *hg, None) == -1
    for n in range(3):
        for heads in (False, True):
            x = [flat(g, heads) if i == n else g for i, g in enumerate(hg)]
            assert lib.pv_attention_backward(p, h["dout"], h["q"], h["k"], h["v"], ho, lse.data_ptr(), *x, None) == -1
    torch.cuda.synchronize()
    assert not o.any() and not any(g.any() for g in grads)
    # The same through the entry points that take an output.
    with pytest.raises(pv.PVError):
        pv.attention(t["q"], t["k"], t["v"], t["qo"], t["ko"], out=o[:1].expand(20, -1, -1))
    w, pos = torch.ones(64, device="cuda"), torch.zeros((20, 1), dtype=torch.int32, device="cuda")
    with pytest.raises(pv.PVError):
        pv.qk_norm_rope(t["q"], t["q"], w, w, pos, pv.rope_frequencies(64, device="cuda"),
                        out=(o, o[:, :1].expand(-1, 2, -1)))
    del alive


def test_strides_of_a_single_row_or_head_do_not_matter():
    t = make([33], [50], 1, 1, 64, torch.bfloat16)
    want = run(t)
    odd = {n: (x.as_strided(x.shape, (64, 1, 1)) if isinstance(x, torch.Tensor) else x) for n, x in t.items()}
    assert all(torch.equal(a, b) for a, b in zip(run(odd), want))
    one = make([1], [1], 4, 2, 64, torch.bfloat16)
    want = run(one)
    for n in ("q", "k", "v", "dout"):
        one[n] = one[n].as_strided(one[n].shape, (3, 64, 1))
    assert all(torch.equal(a, b) for a, b in zip(run(one), want))


def test_heads_expanded_from_one():
    # The gradient of out.sum(1), and queries that all heads share.
    t = make([130, 70], [90, 60], 4, 2, 64, torch.float16)
    for names in (("dout",), ("q",), ("q", "k", "v", "dout")):
        u = dict(t)
        for n in names:
            u[n] = t[n][:, :1].expand(-1, t[n].shape[1], -1)
        dense = {n: (x.contiguous() if isinstance(x, torch.Tensor) else x) for n, x in u.items()}
        for a, b in zip(run(u), run(dense)):
            assert (a.float() - b.float()).abs().max() <= 2.0 ** -9 * b[b.isfinite()].float().abs().max()
