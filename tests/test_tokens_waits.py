"""What a wait that runs out leaves behind, read from the kernels' sources: it cannot be brought about without
hanging a GPU's kernel on purpose.

A barrier of several arrivals (the warps that read an accumulator, or fill a tile) counts them and does not
know who has arrived.  A warp that goes on after its wait has run out, arrives without having seen anything,
and does so for tile after tile, ends phases in the place of warps that still read: these find other numbers than their
own, and take them for an answer.  So a warp arrives only for what it has seen, and what it
writes otherwise is NaN in every place.
"""

from __future__ import annotations

import os
import re

import pytest

from lidar_point_cloud_gb300 import _build

# The waits of warps of which several arrive at one barrier, and their arrivals.
WAIT = re.compile(r"ok = ok && warp_wait")
ARRIVAL = re.compile(r"warp_arrive\(&sm\.|bar_arrive_at\(")
STOP = re.compile(r"if \(!ok\) (break|\{)")


def lines(source):
    with open(os.path.join(_build.CSRC, source)) as f:
        return [x.split("//")[0] for x in f.read().splitlines()]


@pytest.mark.parametrize("source,arrivals", [("pv_loss.cu", 2), ("pv_linear.cu", 4)])
def test_a_warp_arrives_only_for_what_it_has_seen(source, arrivals):
    found, stopped = 0, False
    for n, line in enumerate(lines(source)):
        if WAIT.search(line):
            stopped = False
        if STOP.search(line) and "break" in line:
            stopped = True
        if ARRIVAL.search(line):
            found += 1
            assert stopped or re.search(r"if \(ok( && lane == 0)?\) ", line), f"{source}:{n + 1}"
    assert found == arrivals


def test_what_a_warp_of_the_cross_entropy_has_not_seen_is_nan_in_every_column():
    body = "\n".join(lines("pv_loss.cu"))
    assert not re.search(r"v\[0\] = NAN", body)
    assert "if (!ok) r.x = 1.0f, r.z = NAN;" in body  # the probabilities' exponents
    assert "by = ok ? *a.mult : NAN;" in body  # what the weights' gradient is multiplied with
    assert "ok ? make_float2(most, s) : make_float2(NAN, NAN)" in body and "v[j] = ok ? 0.0f : NAN" in body


def test_both_blocks_of_a_pair_wait_for_their_loads():
    body = "\n".join(lines("pv_loss.cu"))
    assert "bars_drain(rank == 0 ? sm.full : sm.empty, kStages, sent);" in body
