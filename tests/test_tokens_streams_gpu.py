"""The token operators on a stream that is passed to them."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")

pytestmark = pytest.mark.gpu

OFF = [0, 300, 500]


def inputs():
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v, do = (torch.randn((500, 4, 64), generator=g, device="cuda").bfloat16() for _ in range(4))
    pos = torch.randint(0, 400, (500, 2), generator=g, device="cuda", dtype=torch.int32)
    return q, k, v, do, pos, torch.ones(64, device="cuda"), pv.rope_frequencies(64, 2, device="cuda")


def run(q, k, v, do, pos, w, freq, **on):
    qr, kr = pv.qk_norm_rope(q, k, w, w, pos, freq, **on)
    o, lse = pv.attention(qr, kr, v, OFF, OFF, return_lse=True, **on)
    grads = pv.attention_backward(do, qr, kr, v, o, lse, OFF, OFF, **on)
    back = pv.qk_norm_rope_backward(grads[0], grads[1], q, k, w, w, pos, freq, **on)
    x, gate = v.reshape(500, 256), do.reshape(500, 256)
    h, last, states = pv.gated_scan(x, gate, OFF, return_states=True, **on)
    return (qr, kr, o, lse, *grads, *back, h, last, *pv.gated_scan_backward(x, None, x, gate, states, OFF, **on))


@pytest.mark.parametrize("handle", [False, True])
def test_results_are_the_same(handle):
    t = inputs()
    want = run(*t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(*t, stream=side.cuda_stream if handle else side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_outputs_are_not_memory_that_another_stream_may_still_use():
    # Freed by this stream, whose queue may still hold its last use: free for this
    # stream's next calls only.
    x = torch.zeros((4096, 512), device="cuda")
    junk = torch.empty_like(x)
    at = junk.data_ptr()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    del junk
    h, _ = pv.gated_scan(x, x, [0, 4096], stream=side)
    side.synchronize()
    assert h.data_ptr() != at
    h, _ = pv.gated_scan(x, x, [0, 4096])
    assert h.data_ptr() == at


def test_captured_in_a_graph():
    # Warm workspaces: nothing is allocated but outputs, nothing synchronizes.
    t = inputs()
    want = run(*t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*t)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run(*t)
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
