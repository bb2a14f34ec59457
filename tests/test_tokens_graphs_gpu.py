"""Graphs of the token operators: what they hold stays theirs, whatever is called, captured or
released after them."""

from __future__ import annotations

import gc
import time

import pytest

torch = pytest.importorskip("torch")
pv = pytest.importorskip("lidar_point_cloud_gb300")

pytestmark = pytest.mark.gpu


def inputs(rows, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, do = (torch.randn((rows, 8, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn((rows, 1, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    pos = torch.randint(0, 400, (rows, 2), generator=g, device="cuda", dtype=torch.int32)
    return q, k, v, do, pos, torch.ones(64, device="cuda"), pv.rope_frequencies(64, 2, device="cuda")


def run(q, k, v, do, pos, w, freq):
    """Every operator that keeps something in a workspace: keys cut into parts, heads cut into
    parts, sums of weights, published states."""
    rows = len(q)
    off = [0, rows]
    o1 = pv.attention(q[:2], k, v, [0, 2], off)
    o, lse = pv.attention(q, k, v, off, off, return_lse=True)
    grads = pv.attention_backward(do, q, k, v, o, lse, off, off)
    back = pv.qk_norm_rope_backward(grads[0], grads[1], q, k, w, w, pos, freq)
    x, gate = q.reshape(rows, 512), do.reshape(rows, 512)
    h, last, states = pv.gated_scan(x, gate, off, return_states=True)
    return (o1, o, lse, *grads, *back, h, last, *pv.gated_scan_backward(x, None, x, gate, states, off))


def captured(t, stream):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = run(*t)
    return graph, out


def warm_stream(t):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*t)
    side.synchronize()
    return side


def replayed(graph, out, want):
    for x in out:
        x.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    return all(torch.equal(a, b) for a, b in zip(out, want))


def test_replay_after_a_larger_call_on_the_stream():
    small, large = inputs(1500, 0), inputs(9000, 1)
    want, big = run(*small), run(*large)
    side = warm_stream(small)
    graph, out = captured(small, side)
    assert replayed(graph, out, want)
    with torch.cuda.stream(side):
        got = run(*large)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, big))
    assert replayed(graph, out, want)
    with torch.cuda.stream(side):
        got = run(*large)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, big))


def test_replay_after_the_workspaces_are_released():
    t = inputs(1500, 2)
    want = run(*t)
    graph, out = captured(t, warm_stream(t))
    pv.release_workspace()
    junk = torch.full((1 << 28,), 7, dtype=torch.uint8, device="cuda")
    assert replayed(graph, out, want)
    assert all(torch.equal(a, b) for a, b in zip(run(*t), want)) and replayed(graph, out, want)
    del junk


def test_a_stream_that_was_never_used():
    # Nothing to be warmed up: a captured call brings its own workspace.
    t = inputs(700, 3)
    want = run(*t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, out = captured(t, side)
    assert replayed(graph, out, want)


def test_two_graphs_of_one_stream_beside_each_other_and_beside_calls():
    a, b = inputs(4000, 4), inputs(3100, 5)
    want = run(*a), run(*b)
    side = warm_stream(a)
    ga, oa = captured(a, side)
    gb, ob = captured(b, side)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for x in (*oa, *ob):
            x.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, (ga, gb)):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(side):
            eager = run(*a)
        torch.cuda.synchronize()
        for out, w in ((oa, want[0]), (ob, want[1]), (eager, want[0])):
            assert all(torch.equal(x, y) for x, y in zip(out, w))


def test_a_larger_call_later_in_one_capture():
    small, large = inputs(900, 6), inputs(5000, 7)
    want = (*run(*small), *run(*large), *run(*small))
    side = warm_stream(small)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = (*run(*small), *run(*large), *run(*small))
    for _ in range(3):
        assert replayed(graph, out, want)


def test_what_a_destroyed_graph_held_is_used_again():
    t = inputs(20000, 8)  # some 44 MB of parts a graph
    want = run(*t)
    side = warm_stream(t)
    free = []
    for _ in range(12):
        graph, out = captured(t, side)
        assert replayed(graph, out, want)
        graph.reset()
        del graph, out
        gc.collect()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        time.sleep(0.05)  # the space is given back by a thread of CUDA's
        free.append(torch.cuda.mem_get_info()[0])
    assert free[3] - free[-1] < 150 << 20
