"""The decay that a state goes through once a chunk, compiled for the host: as good as its comment says."""

from __future__ import annotations

import os
import re
import subprocess

from lidar_point_cloud_gb300 import _build

PROGRAM = r"""
#include <cmath>
#include <cstdio>
#include <cstring>
struct float2 { float x, y; };
static float2 make_float2(float x, float y) { return {x, y}; }
static float __int_as_float(int i) { float f; memcpy(&f, &i, 4); return f; }
constexpr float kLog2e = 1.4426950408889634f;
%s
int main() {
  double worst = 0.0, single = 0.0;
  // Decays of 2^-24 up to 2 a token, over 1 token up to as many as leave e^-80 (of a chunk, a segment, a frame).
  for (int e = -24; e <= 1; ++e)
    for (int m = 0; m < 61; ++m) {
      const float d = -std::ldexp(1.0f + m / 61.0f, e);
      for (double n = 1; n < 2e7 && n * -d < 80; n = std::floor(n * 1.37) + 1) {
        const float x = static_cast<float>(n);
        const float2 w = decay_exact(d, x);
        const double want = std::exp(static_cast<double>(d) * static_cast<double>(x));
        worst = std::fmax(worst, std::fabs((static_cast<double>(w.x) + w.y) / want - 1.0));
        single = std::fmax(single, std::fabs(static_cast<double>(static_cast<float>(want)) / want - 1.0));
      }
    }
  const float2 none = decay_exact(-1e4f, 1.0f), one = decay_exact(-1e4f, 0.0f), all = decay_exact(0.0f, 1e6f);
  std::printf("%%.9e %%.9e %%d\n", worst, single,
              none.x + none.y == 0.0f && one.x + one.y == 1.0f && one.y == 0.0f && all.x + all.y == 1.0f && all.y == 0.0f);
}
"""


def test_decay_is_better_than_one_number_of_32_bits(tmp_path):
    with open(os.path.join(_build.CSRC, "pv_linear.cu")) as f:
        body = re.search(r"__device__ __forceinline__ (float2 decay_exact\(.*?^}$)", f.read(), re.M | re.S).group(1)
    source, program = tmp_path / "decay.cpp", tmp_path / "decay"
    source.write_text(PROGRAM % ("static " + body))
    # (No contraction, as the kernels are compiled: a product and a sum are two roundings, a fused one is asked for.)
    subprocess.run(["g++", "-O1", "-std=c++17", "-ffp-contract=off", str(source), "-o", str(program)], check=True)
    worst, single, ends = subprocess.run([str(program)], check=True, capture_output=True, text=True).stdout.split()
    assert ends == "1"
    # q = r^2 (1/2 + r/6 + ...) is off by three roundings, 3 2^-24 of at most 0.067 (0.054 for r < 0), and the sums that
    # end in `low` by 2^-28 each: 2^-25.6, or 2^-26 over a result of 0.7 at least, so below 2^-25.3 of the result.  One
    # number of 32 bits is off by up to 2^-24.
    assert float(single) > 2.0 ** -24.1 and float(worst) <= 2.0 ** -25.3, (float(worst), float(single))
