"""The gated linear recurrence along frames against 64 bits."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")
import _tokens as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return off


def make(lens, C, dtype, seed=0, mean=-2.0):
    off = offsets(lens)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s, std=1.0, mean=0.0):
        return torch.randn(s, generator=g, device="cuda") * std + mean

    x, gate, dh = (normal(off[-1], C, std=s, mean=m).to(dtype) for s, m in ((1.0, 0.0), (1.5, mean), (1.0, 0.0)))
    return x, gate, dh, off, normal(len(lens), C), normal(len(lens), C)


def close(got, want, dtype, name, big):
    # Rounded once; the state is a convex mean of values of size `big`, whose 32-bit
    # errors (z good to 2^-20, one rounding a step) are forgotten as fast as the state
    # forgets: 1 / z steps, some hundreds here.
    got, want = got.cpu(), want.cpu()
    tiny = 2.0 ** -24 if dtype is torch.float16 else 0.0
    ref.within(got, want, 2 * ref.UNIT[dtype] * want.abs() + (2.0 ** -16 if dtype is not torch.float32 else 2.0 ** -17) * big + tiny, name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("lens,C", [([1], 1), ([1], 64), ([5], 7), ([16, 17], 8), ([127, 128, 129], 64), ([0, 300, 0, 1], 33),
                                    ([700], 2), ([2100, 40], 130), ([4500], 3)])
def test_forward_and_backward(lens, C, reverse, dtype):
    x, gate, dh, off, h0, dlast = make(lens, C, dtype)
    h, last, states = pv.gated_scan(x, gate, off, h0, reverse=reverse, return_states=True)
    dx, dgate, dh0 = pv.gated_scan_backward(dh, dlast, x, gate, states, off, reverse=reverse)
    want = ref.scan(x, gate, off, h0, reverse, dh, dlast)
    close(h, want["h"], dtype, "h", 4.0)
    close(last, want["last"], torch.float32, "last", 4.0)
    # A step's gradient collects those of the steps after it: up to some 1 / z terms.
    close(dx, want["dx"], dtype, "dx", 16.0)
    close(dgate, want["dgate"], dtype, "dgate", 64.0)
    close(dh0, want["dh0"], torch.float32, "dh0", 64.0)


def test_without_first_or_last_states():
    x, gate, dh, off, _, _ = make([50, 3], 24, torch.float32)
    h, last, states = pv.gated_scan(x, gate, off, return_states=True)
    dx, dgate, dh0 = pv.gated_scan_backward(dh, None, x, gate, states, off)
    want = ref.scan(x, gate, off, None, False, dh, None)
    for got, n in ((h, "h"), (last, "last"), (dx, "dx"), (dgate, "dgate"), (dh0, "dh0")):
        close(got, want[n], torch.float32, n, 64.0)


def test_token_by_token_is_the_whole_sequence():
    x, gate, _, off, h0, _ = make([40], 96, torch.float32)
    h, last = pv.gated_scan(x, gate, off, h0)
    state = h0
    for t in range(40):
        step, state = pv.gated_scan(x[t:t + 1], gate[t:t + 1], [0, 1], state)
        close(step, h[t:t + 1].double(), torch.float32, "step", 4.0)
    close(state, last.double(), torch.float32, "state", 4.0)


def test_gates_at_their_ends_and_a_state_that_is_kept():
    # A gate of -inf keeps the state to the bit, one of +inf replaces it.
    lens = [3000]
    x, gate, _, off, h0, _ = make(lens, 66, torch.float32)
    gate[:] = -float("inf")
    gate[1500] = float("inf")
    h, last = pv.gated_scan(x, gate, off, h0)
    assert torch.equal(h[:1500], h0.expand(1500, -1)) and torch.equal(h[1500:], x[1500].expand(1500, -1))
    assert torch.equal(last[0], x[1500])


def test_strided_rows_and_a_stretch_of_channels():
    x, gate, dh, off, h0, dlast = make([130, 260], 48, torch.bfloat16)
    wide = torch.zeros((390, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:50], wide[:, 64:112] = x, gate
    a = pv.gated_scan(x, gate, off, h0)
    b = pv.gated_scan(wide[:, 2:50], wide[:, 64:112], off, h0)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    odd = pv.gated_scan(wide[:, 2:50].clone()[:, 1:48], wide[:, 64:112].clone()[:, 1:48], off, h0[:, 1:48].contiguous())
    want = ref.scan(x[:, 1:48], gate[:, 1:48], off, h0[:, 1:48])
    close(odd[0], want["h"], torch.bfloat16, "odd", 4.0)


def test_same_bits_every_time():
    x, gate, dh, off, h0, dlast = make([60000, 10, 3000], 64, torch.bfloat16, mean=-4.0)
    runs = []
    for _ in range(4):
        h, last, states = pv.gated_scan(x, gate, off, h0, return_states=True)
        runs.append((h, last, *pv.gated_scan_backward(dh, dlast, x, gate, states, off)))
    for r in runs[1:]:
        assert all(torch.equal(s, t) for s, t in zip(runs[0], r))


def test_two_streams():
    a, b = make([5000], 128, torch.float32, seed=1), make([7000], 128, torch.float32, seed=2)
    want = [pv.gated_scan(t[0], t[1], t[3], t[4]) for t in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s, t in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(pv.gated_scan(t[0], t[1], t[3], t[4]))
    torch.cuda.synchronize()
    for n, g in enumerate(got):
        assert all(torch.equal(s, t) for s, t in zip(g, want[n % 2]))


def test_captured_in_a_graph():
    x, gate, _, off, h0, _ = make([3000], 64, torch.float32)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        want = pv.gated_scan(x, gate, off, h0)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = pv.gated_scan(x, gate, off, h0)
        for _ in range(3):
            got[0].zero_()
            graph.replay()
            stream.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_gradient_against_differences():
    x, gate, dh, off, h0, dlast = make([70, 5], 4, torch.float32, seed=9)
    *_, states = pv.gated_scan(x, gate, off, h0, return_states=True)
    grads = pv.gated_scan_backward(dh, dlast, x, gate, states, off)

    def loss(x, gate, h0):
        r = ref.scan(x, gate, off, h0)
        return (r["h"] * dh.double().cpu()).sum() + (r["last"] * dlast.double().cpu()).sum()

    at = [t.double().cpu() for t in (x, gate, h0)]
    g = torch.Generator().manual_seed(10)
    for n, grad in enumerate(grads):
        grad = grad.double().cpu()
        way = torch.randn(at[n].shape, generator=g, dtype=torch.float64)
        up, down = list(at), list(at)
        up[n], down[n] = at[n] + 1e-5 * way, at[n] - 1e-5 * way
        slope = (loss(*up) - loss(*down)) / 2e-5
        assert abs((grad * way).sum() - slope) <= 1e-5 * (grad.abs() * way.abs()).sum()


def test_refusals():
    x, gate, dh, off, h0, dlast = make([30, 40], 16, torch.bfloat16)
    for error, args in ((TypeError, (x.double(), gate.double(), off, h0)), (TypeError, (x, gate.float(), off, h0)),
                        (ValueError, (x, gate[:69], off, h0)), (ValueError, (x, gate, [0, 30, 71], h0)),
                        (ValueError, (x, gate, [0], h0)), (ValueError, (x, gate, off, h0[:1])),
                        (TypeError, (x, gate, off, h0.bfloat16())), (ValueError, (x.cpu(), gate.cpu(), off, h0)),
                        (ValueError, (x.T, gate.T, [0, 16], h0))):
        with pytest.raises(error):
            pv.gated_scan(*args)
    with pytest.raises(pv.PVError) as e:
        pv.gated_scan(x, gate, [0, 50, 40, 70], torch.zeros((3, 16), device="cuda"))
    assert e.value.status == -1
    with pytest.raises(ValueError):
        pv.gated_scan_backward(dh, dlast, x, gate, torch.zeros((1, 16), device="cuda"), off)
