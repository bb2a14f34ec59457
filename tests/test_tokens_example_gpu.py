"""The operators together, as a network on voxel tokens uses them."""

from __future__ import annotations

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_pillar_tokens.py")


def load():
    spec = importlib.util.spec_from_file_location("train_pillar_tokens", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_lowers_the_loss_and_repeats_to_the_bit():
    example = load()
    first = example.main(["--frames", "3", "--steps", "12"])
    assert all(torch.isfinite(torch.tensor(first))) and first[-1] < 0.8 * first[0]
    # The library's operators give the same bits every time, so the first loss, and
    # the second, which has a whole backward pass in it, do too, up to the 32-bit
    # products of torch around them.
    again = example.main(["--frames", "3", "--steps", "2"])
    assert again[0] == pytest.approx(first[0], rel=1e-5) and again[1] == pytest.approx(first[1], rel=1e-3)
