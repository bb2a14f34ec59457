// What the attention kernels share: their arguments and the score of a pair.

#pragma once

#include "pv_seq.cuh"

#include <cuda.h>

#include <map>
#include <utility>

namespace pvs {

struct View {
  char* data;
  long long row, head;  // strides in bytes
};

struct AttnArgs {
  View q, k, v, o, dout, dq, dk, dv;
  float* lse;            // [H, queries]
  // Backward, what dq leaves of the queries for dk and dv, rows of `sides_row` floats in
  // which each frame begins on 16 bytes (side0): [H] the exponent's offset from lse, [H]
  // delta (negated), [3] positions.
  float* sides;
  long long sides_row;
  // Backward, float16: per frame, what dk's score gradients are scaled by on top of the
  // probabilities' factor, and the largest norm of a row of v, found by norm_parts blocks a
  // frame.  Null for bfloat16.
  float2* up;      // [frames]
  float2* norms;   // [frames, norm_parts]: largest squared norms of rows of dout and v
  unsigned int* norms_done;  // [frames], zero between launches
  int norm_parts;
  const float* slopes;
  const int32_t* qpos;
  const int32_t* kpos;
  long long qpos_stride, kpos_stride;
  float scale, cap;
  int axes, causal, H, Hk, G, D, frames, queries, keys;
  int Dn;          // D rounded up to 16
  int pack_log2;   // heads of a key head that share a tile of rows (log2)
  int head_parts;  // blocks among which the query heads of a key head are cut (dk, dv)
  int chunk;       // key tiles of a block: fewer than there are if the keys are split
  float* part_o;   // split keys: [split, queries, H, D] unnormalised outputs, or null;
                   // backward with head_parts > 1: [part, dk or dv, keys, Hk, D]
  float2* part_ml; // split keys: [split, queries, H] maximum (in units of log2) and sum
  int q0[PV_MAX_FRAMES + 1];    // row offsets of the frames
  int k0[PV_MAX_FRAMES + 1];
  int prefix[PV_MAX_FRAMES];
  int side0[PV_MAX_FRAMES];
  // The blocks' list: frames by their work, most first, and the first tile of each in
  // that order.  Block b takes tile b / heads of it for head b % heads.
  unsigned char order[PV_MAX_FRAMES];
  int tile0[PV_MAX_FRAMES + 1];
  int heads;
};

struct AttnMaps {
  CUtensorMap q, k, v, dout;
};

// Tensor map of rows of heads for tiles of `rows` rows of `pack` heads of 64
// elements: dimensions (D, pack, heads / pack, rows), elements past D read as 0.
int make_map(CUtensorMap* map, const View& v, int dtype, int D, int heads, int pack, int64_t total, int rows);

// Kernel launches of pv_attn_fwd.cu and pv_attn_bwd.cu, each compiled once for
// bfloat16 and once, through its _half.cu, for float16.
#ifdef PV_ATTN_HALF
using Storage = __half;
#define PV_ATTN_NAME(name) name##_half
#else
using Storage = __nv_bfloat16;
#define PV_ATTN_NAME(name) name##_bf16
#endif
int attn_forward_bf16(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s);
int attn_forward_half(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s);
int attn_backward_up_half(const AttnArgs& a, cudaStream_t s);  // float16: `up`, first
int attn_backward_dq_bf16(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s);   // and the sides
int attn_backward_dq_half(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s);
int attn_backward_dkv_bf16(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s);  // after it
int attn_backward_dkv_half(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s);

// Lets a kernel take `bytes` of dynamic shared memory on the current device.  Asked once
// per kernel and device; a second time does no harm.
template <typename K>
int allow_smem(K kernel, int bytes) {
  static std::map<std::pair<const void*, int>, bool> done;
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PV_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  bool& ready = done[std::make_pair(reinterpret_cast<const void*>(kernel), dev)];
  if (ready) return PV_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();
    return PV_ERR_CUDA;
  }
  ready = true;
  return PV_OK;
}

template <typename K, typename... A>
int launch_pdl(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return PV_ERR_CUDA;
  }
  return PV_OK;
}

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
