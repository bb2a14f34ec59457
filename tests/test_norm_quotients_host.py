"""The quotients of the norm in 8 bits, compiled for the host: on the same side of every border as a division."""

from __future__ import annotations

import os
import re
import subprocess

from lidar_point_cloud_gb300 import _build

PROGRAM = r"""
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>
static float off = 0.0f;  // of the approximate reciprocal
static uint32_t __float_as_uint(float f) { uint32_t i; memcpy(&i, &f, 4); return i; }
static float as_float(uint32_t i) { float f; memcpy(&f, &i, 4); return f; }
static float max_nan(float a, float b) { return std::isnan(a) || std::isnan(b) ? NAN : a > b ? a : b; }
using std::fmaf;
%s
int main() {
  std::mt19937 r(1);
  long long wrong = 0, scales = 0, divided = 0, tried = 0;
  for (int n = 0; n < 300000; ++n) {
    // Of any mantissa, and of mantissas of which the quotients come nearest to the middles of floats.
    uint32_t mantissa = r() & 0x7FFFFF;
    if (n & 1) mantissa = ((mantissa & 0x700000) + static_cast<int>(r() %% 4096) - 2048) & 0x7FFFFF;
    const float most = as_float((60 + r() %% 135) << 23 | mantissa);
    off = (static_cast<int>(r() %% 3) - 1) * 0x1p-23f;
    const Quotients by(most);
    scales += by.scale != most / 448.0f;
    if (!by.quick) { ++divided; continue; }
    const float s = by.scale;
    for (int k = 0; k < 40; ++k) {
      // Borders between values of e4m3: odd multiples of half steps, 2^-10 the smallest, 432 the largest.
      const int e = static_cast<int>(r() %% 15) - 6;
      const float border = k & 1 ? (r() %% 8 + 0.5f) * 0x1p-9f : std::ldexp(1.0f + (r() %% 8 + 0.5f) / 8.0f, e);
      float y = border * s;
      for (int i = 0; i < 4; ++i) y = std::nextafter(y, 0.0f);
      for (int i = 0; i < 9; ++i, y = std::nextafter(y, INFINITY)) {
        const float q = fmaf(y, by.high, y * by.low), want = y / s;
        wrong += (q < border) != (want < border) || (q > border) != (want > border);
        ++tried;
      }
    }
    const float zero = fmaf(-0.0f, by.high, -0.0f * by.low);
    wrong += !std::signbit(zero) || std::signbit(fmaf(0.0f, by.high, 0.0f * by.low));
  }
  for (float most : {0.0f, 1e-40f, 1e-30f, 1e30f, 3e38f, INFINITY, NAN}) wrong += Quotients(most).quick;
  wrong += Quotients(0.0f).scale != 0x1p-126f || !std::isinf(Quotients(INFINITY).scale) || !std::isnan(Quotients(NAN).scale);
  std::printf("%%lld %%lld %%lld %%lld\n", wrong, scales, divided, tried);
}
"""


def test_quotients_are_on_the_side_of_a_division(tmp_path):
    with open(os.path.join(_build.CSRC, "pv_norm.cu")) as f:
        found = re.search(r"^struct Quotients \{.*?^\};$", f.read(), re.M | re.S)
    assert found, "values are not taken from the quotients"
    body = found.group(0)
    body = body.replace("__device__ __forceinline__ ", "")
    body, n = re.subn(r'asm\("rcp.*?"f"\(scale\)\);', "high = 1.0f / scale; high += high * off;", body)
    assert n == 1
    source, program = tmp_path / "quotients.cpp", tmp_path / "quotients"
    source.write_text(PROGRAM % body)
    # (No contraction, as the kernels are compiled.)
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", str(source), "-o", str(program)], check=True)
    wrong, scales, divided, tried = map(int, subprocess.run([str(program)], check=True, capture_output=True, text=True).stdout.split())
    assert wrong == 0 and scales == 0, (wrong, scales, tried)
    assert divided < 30000 and tried > 10 ** 7
