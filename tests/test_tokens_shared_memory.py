"""Shared arrays that kernels of the token operators read or write in wider pieces are declared on boundaries of them."""

from __future__ import annotations

import os
import re

import pytest

from lidar_point_cloud_gb300 import _build

WIDE = {"float2": 8, "uint2": 8, "float4": 16, "uint4": 16}


@pytest.mark.parametrize("source", ["pv_linear.cu", "pv_loss.cu", "pv_norm.cu"])
def test_wide_pieces_are_aligned(source):
    with open(os.path.join(_build.CSRC, source)) as f:
        kernels = f.read().split("__global__")[1:]
    for kernel in kernels:
        for most, names in re.findall(r"^  __shared__ (?:alignas\((\d+)\) )?(?:float|int|unsigned char) ([^;]*);", kernel, re.M):
            for name in re.findall(r"(\w+)\[", names):
                for piece in re.findall(r"reinterpret_cast<(?:const )?(\w+)\*>\(&?" + name + r"\b", kernel):
                    if piece in WIDE:
                        assert int(most or 4) >= WIDE[piece], f"{source}: {name} read as {piece}"
