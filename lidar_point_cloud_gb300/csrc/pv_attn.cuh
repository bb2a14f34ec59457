// What the attention kernels share: their arguments and the score of a pair.

#pragma once

#include "pv_seq.cuh"

namespace pvs {

struct View {
  char* data;
  long long row, head;  // strides in bytes
};

struct AttnArgs {
  View q, k, v, o, dout, dq, dk, dv;
  float* lse;            // [H, queries]
  float* delta;          // [H, queries]: sum of dout * out (backward)
  const float* slopes;
  const int32_t* qpos;
  const int32_t* kpos;
  long long qpos_stride, kpos_stride;
  float scale, cap;
  int axes, causal, H, Hk, G, D, frames, queries, keys;
  int q0[PV_MAX_FRAMES + 1];    // row offsets of the frames
  int k0[PV_MAX_FRAMES + 1];
  int tile0[PV_MAX_FRAMES + 1]; // first tile of each frame
  int prefix[PV_MAX_FRAMES];
};

// The frame that tile t belongs to: the last one whose first tile is not past t.
__device__ __forceinline__ int frame_of(const int* tile0, int frames, int t) {
  int lo = 0, hi = frames - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile0[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

}  // namespace pvs
