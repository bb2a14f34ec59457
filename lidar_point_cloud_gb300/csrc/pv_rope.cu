// Queries and keys normalised per head and rotated by position, in one pass,
// and the backward pass (pv_qk_norm_rope, pv_qk_norm_rope_backward in pv.h).
//
// A row (token, head) is D elements.  A group of `lanes` lanes (a power of
// two) holds one: each lane 16 bytes of the first half and the same 16 bytes
// of the second half, so both elements of a rotated pair are in one lane.
// Consecutive groups take consecutive heads of a token, so a warp reads and
// writes whole contiguous lines.  The cosines and sines of a tile of tokens
// are worked out once for all heads, into shared memory.
//
// Bound by memory: each element is read once and written once (backward: two
// reads and one write).  Measured at 96,001 rows of 2 x 8 heads of 64, bf16: forward
// 70 us (5.6 TB/s), backward 152 us (3.9 TB/s; its weight sums take the registers of
// half the warps).

#include "pv_seq.cuh"

#include <algorithm>
#include <cmath>

namespace {

using namespace pvs;

constexpr int kThreads = 256;
constexpr int kTableFloats = 8192;  // cosines and sines of a tile: 32 KB of shared memory
// Blocks a multiprocessor that the tiles are cut for: forward two rounds of the six that
// it holds (one round: 81 us, two: 72 us for 96,001 rows of 2 x 8 heads of 64 in bf16),
// backward the two that it holds.
constexpr int kPerSm = 12, kPerSmBack = 2;
constexpr int kMaxBlocks = 1216;    // blocks of the backward pass: one row of weight sums each

struct View {
  char* data;
  long long row, head;  // strides in bytes
};

struct RopeArgs {
  View q, k, oq, ok;    // forward: inputs and outputs; backward: forward inputs and their gradients
  View gq, gk;          // backward: gradients of the outputs
  const float* wq;
  const float* wk;
  const int32_t* pos;
  long long pos_stride;
  const float* freq;
  int rows, hq, hk, D, axes;
  int lanes_log2;       // lanes of a group
  int tile;             // tokens of a tile
  float eps;
  float* partial;       // backward: [blocks, 2, D] weight sums
  unsigned int* done;   // backward: blocks that have written theirs
  float* dwq;
  float* dwk;
};

// (Rows come close to 2^31: the sum takes 64 bits.)
__host__ __device__ __forceinline__ int tiles_of(const RopeArgs& a) {
  return static_cast<int>((static_cast<long long>(a.rows) + a.tile - 1) / a.tile);
}

// Two pairs turned, two operations an instruction where the signs allow.
__device__ __forceinline__ void turn(float* x, float* y, float c0, float c1, float s0, float s1) {
  float a0, a1, b0, b1;
  mul2(a0, a1, x[0], x[1], s0, s1);
  mul2(b0, b1, x[0], x[1], c0, c1);
  x[0] = fmaf(-y[0], s0, b0);
  x[1] = fmaf(-y[1], s1, b1);
  fma2(y[0], y[1], y[0], y[1], c0, c1, a0, a1);
}
__device__ __forceinline__ void turn_back(float* x, float* y, float c0, float c1, float s0, float s1) {
  float a0, a1, b0, b1;
  mul2(a0, a1, y[0], y[1], s0, s1);
  mul2(b0, b1, y[0], y[1], c0, c1);
  y[0] = fmaf(-x[0], s0, b0);
  y[1] = fmaf(-x[1], s1, b1);
  fma2(x[0], x[1], x[0], x[1], c0, c1, a0, a1);
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Cosine and sine of an angle in radians.  It is brought to turns first, in two
// 32-bit parts of 1 / (2 pi) (the fused product makes the first part's rounding
// known), so that whole turns drop out exactly; then CUDA's sincospif.
__device__ __forceinline__ float2 cos_sin(float angle) {
  constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
  constexpr float kHigh = static_cast<float>(kTurn), kLow = static_cast<float>(kTurn - static_cast<double>(kHigh));
  const float t = angle * kHigh;
  const float rest = fmaf(angle, kLow, fmaf(angle, kHigh, -t));
  float2 c;
  sincospif(2.0f * ((t - rintf(t)) + rest), &c.y, &c.x);
  return c;
}

// Cosines and sines of the tile's tokens, [cosine, sine][token][pair].
__device__ __forceinline__ void fill_table(const RopeArgs& a, int t0, int tokens, float* table) {
  const int half = a.D >> 1;
  for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
    const int t = i / half, p = i - t * half;
    const float at = static_cast<float>(a.pos[static_cast<long long>(t0 + t) * a.pos_stride + p % a.axes]);
    const float2 c = cos_sin(at * a.freq[p]);
    table[i] = c.x;
    table[kTableFloats / 2 + i] = c.y;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) pv_rope_kernel(const RopeArgs a) {
  constexpr int V = Pack<T>::kN;
  __shared__ __align__(16) float table[kTableFloats];
  const int half = a.D >> 1;
  const int lanes = 1 << a.lanes_log2;
  const int sub = threadIdx.x & (lanes - 1);
  const int group = threadIdx.x >> a.lanes_log2, groups = kThreads >> a.lanes_log2;
  const bool on = sub * V < half;
  const int heads = a.hq + a.hk;
  const float inv = 1.0f / static_cast<float>(a.D);
  wait_prior_grid();
  const int t0 = blockIdx.x * a.tile;
  const int tokens = min(a.tile, a.rows - t0);
  __shared__ __align__(16) float weight[2 * 256];
  for (int i = threadIdx.x; i < a.D; i += kThreads) {
    weight[i] = a.wq[i];
    weight[256 + i] = a.hk ? a.wk[i] : 0.0f;
  }
  fill_table(a, t0, tokens, table);
  const int step_t = groups / heads, step_h = groups - step_t * heads;
  int t = group / heads, h = group - t * heads;
  // A row is loaded one round ahead of its arithmetic.
  uint4 next0 = {}, next1 = {};
  auto fetch = [&](int t, int h) {
    if (!on || t >= tokens) return;
    const View& in = h < a.hq ? a.q : a.k;
    const char* p = in.data + (t0 + t) * in.row + (h < a.hq ? h : h - a.hq) * in.head + sub * 16;
    next0 = *reinterpret_cast<const uint4*>(p);
    next1 = *reinterpret_cast<const uint4*>(p + half * sizeof(T));
  };
  fetch(t, h);
  __syncthreads();  // the table
  for (int r0 = 0; r0 < tokens * heads; r0 += groups) {
    const uint4 raw0 = next0, raw1 = next1;
    const int t_now = t, h_now = h;
    t += step_t;
    h += step_h;
    if (h >= heads) h -= heads, ++t;
    fetch(t, h);
    const bool live = on && t_now < tokens;
    float x[2 * V];
    Pack<T>::open(raw0, x);
    Pack<T>::open(raw1, x + V);
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * V; i += 2) fma2(s0, s1, x[i], x[i + 1], x[i], x[i + 1], s0, s1);
    const float ss = group_sum(on ? s0 + s1 : 0.0f, lanes);
    if (live) {
      const bool isq = h_now < a.hq;
      const float rs = rsqrtf(fmaf(ss, inv, a.eps));
      const float* w = weight + (isq ? 0 : 256) + sub * V;
      const float* cs = table + t_now * half + sub * V;
#pragma unroll
      for (int i = 0; i < 2 * V; i += 2) mul2(x[i], x[i + 1], x[i], x[i + 1], rs, rs);
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 w0 = *reinterpret_cast<const float4*>(w + i), w1 = *reinterpret_cast<const float4*>(w + half + i);
        const float4 c = *reinterpret_cast<const float4*>(cs + i);
        const float4 n = *reinterpret_cast<const float4*>(cs + kTableFloats / 2 + i);
        mul2(x[i], x[i + 1], x[i], x[i + 1], w0.x, w0.y);
        mul2(x[i + 2], x[i + 3], x[i + 2], x[i + 3], w0.z, w0.w);
        mul2(x[V + i], x[V + i + 1], x[V + i], x[V + i + 1], w1.x, w1.y);
        mul2(x[V + i + 2], x[V + i + 3], x[V + i + 2], x[V + i + 3], w1.z, w1.w);
        turn(x + i, x + V + i, c.x, c.y, n.x, n.y);
        turn(x + i + 2, x + V + i + 2, c.z, c.w, n.z, n.w);
      }
      const View& out = isq ? a.oq : a.ok;
      char* p = out.data + (t0 + t_now) * out.row + (isq ? h_now : h_now - a.hq) * out.head + sub * 16;
      Pack<T>::store(p, x);
      Pack<T>::store(p + half * sizeof(T), x + V);
    }
  }
  allow_next_grid();
}

// Backward.  With g the gradient turned back, n = x r, r = 1 / sqrt(mean(x^2) + eps):
// dx = r (g w - n mean(g w n)), dw = sum of g n over rows.  A lane keeps the
// weight sums of its own columns in registers over all of the block's tiles;
// a block's lanes are joined in shared memory, the blocks by the last one to
// finish, both in a fixed order.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) pv_rope_backward_kernel(const RopeArgs a) {
  constexpr int V = Pack<T>::kN;
  __shared__ __align__(16) float table[kTableFloats];
  __shared__ bool last;
  const int half = a.D >> 1;
  const int lanes = 1 << a.lanes_log2;
  const int sub = threadIdx.x & (lanes - 1);
  const int group = threadIdx.x >> a.lanes_log2, groups = kThreads >> a.lanes_log2;
  const bool on = sub * V < half;
  const float inv = 1.0f / static_cast<float>(a.D);
  wait_prior_grid();
  const int tiles = tiles_of(a);
  float* sums = table;
  for (int side = 0; side < 2; ++side) {
    const View& in = side ? a.k : a.q;
    const View& gr = side ? a.gk : a.gq;
    const View& out = side ? a.ok : a.oq;
    const float* wsrc = side ? a.wk : a.wq;
    const int heads = side ? a.hk : a.hq;
    if (heads == 0) continue;
    float w[2 * V], acc[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[i] = on ? wsrc[sub * V + i] : 0.0f;
      w[V + i] = on ? wsrc[half + sub * V + i] : 0.0f;
      acc[i] = acc[V + i] = 0.0f;
    }
    const int step_t = groups / heads, step_h = groups - step_t * heads;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      const int t0 = tile * a.tile;
      const int tokens = min(a.tile, a.rows - t0);
      int t = group / heads, h = group - t * heads;
      // A row is loaded one round ahead of its arithmetic.
      uint4 next[4] = {};
      auto fetch = [&](int t, int h) {
        if (!on || t >= tokens) return;
        const char* p = in.data + (t0 + t) * in.row + h * in.head + sub * 16;
        const char* pg = gr.data + (t0 + t) * gr.row + h * gr.head + sub * 16;
        next[0] = *reinterpret_cast<const uint4*>(p);
        next[1] = *reinterpret_cast<const uint4*>(p + half * sizeof(T));
        next[2] = *reinterpret_cast<const uint4*>(pg);
        next[3] = *reinterpret_cast<const uint4*>(pg + half * sizeof(T));
      };
      fetch(t, h);
      __syncthreads();  // the last tile's table is no longer read
      fill_table(a, t0, tokens, table);
      __syncthreads();
      for (int r0 = 0; r0 < tokens * heads; r0 += groups) {
        float x[2 * V], g[2 * V];
        Pack<T>::open(next[0], x);
        Pack<T>::open(next[1], x + V);
        Pack<T>::open(next[2], g);
        Pack<T>::open(next[3], g + V);
        const int t_now = t, h_now = h;
        const bool live = on && t_now < tokens;
        t += step_t;
        h += step_h;
        if (h >= heads) h -= heads, ++t;
        fetch(t, h);
        float s0 = 0.0f, s1 = 0.0f, d0 = 0.0f, d1 = 0.0f;
        if (live) {
          const float* cs = table + t_now * half + sub * V;
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            const float4 c = *reinterpret_cast<const float4*>(cs + i);
            const float4 n = *reinterpret_cast<const float4*>(cs + kTableFloats / 2 + i);
            turn_back(g + i, g + V + i, c.x, c.y, n.x, n.y);
            turn_back(g + i + 2, g + V + i + 2, c.z, c.w, n.z, n.w);
          }
#pragma unroll
          for (int i = 0; i < 2 * V; i += 2) {
            float u0, u1;
            fma2(s0, s1, x[i], x[i + 1], x[i], x[i + 1], s0, s1);
            mul2(u0, u1, g[i], g[i + 1], w[i], w[i + 1]);
            fma2(d0, d1, u0, u1, x[i], x[i + 1], d0, d1);
          }
        }
        const float ss = group_sum(s0 + s1, lanes);
        const float dot = group_sum(d0 + d1, lanes);
        if (live) {
          const float rs = rsqrtf(fmaf(ss, inv, a.eps));
          const float m = -(dot * inv * rs * rs);  // mean(g w n) over n: n = x rs
#pragma unroll
          for (int i = 0; i < 2 * V; i += 2) {
            float u0, u1;
            mul2(u0, u1, x[i], x[i + 1], rs, rs);
            fma2(acc[i], acc[i + 1], g[i], g[i + 1], u0, u1, acc[i], acc[i + 1]);
            mul2(u0, u1, x[i], x[i + 1], m, m);
            fma2(u0, u1, g[i], g[i + 1], w[i], w[i + 1], u0, u1);
            mul2(x[i], x[i + 1], u0, u1, rs, rs);
          }
          char* p = out.data + (t0 + t_now) * out.row + h_now * out.head + sub * 16;
          Pack<T>::store(p, x);
          Pack<T>::store(p + half * sizeof(T), x + V);
        }
      }
    }
    // Lanes of equal `sub` hold the same columns: joined over the warp, then
    // warp by warp.
#pragma unroll
    for (int i = 0; i < 2 * V; ++i)
      for (int o = lanes; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], o);
    __syncthreads();
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) < lanes && on) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sums[warp * a.D + sub * V + i] = acc[i];
        sums[warp * a.D + half + sub * V + i] = acc[V + i];
      }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += kThreads) {
      float v = 0.0f;
      for (int i = 0; i < kThreads / 32; ++i) v += sums[i * a.D + d];
      a.partial[(static_cast<long long>(blockIdx.x) * 2 + side) * a.D + d] = v;
    }
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.done, 1u) == gridDim.x - 1;
  __syncthreads();
  if (last) {
    __threadfence();
    // kThreads / 64 slices of the blocks for each of 64 columns, joined in order.
    const int cols = a.hk ? 2 * a.D : a.D;
    const int slice = threadIdx.x >> 6, slices = kThreads / 64;
    for (int c0 = 0; c0 < cols; c0 += 64) {
      const int c = c0 + (threadIdx.x & 63);
      float v = 0.0f;
      if (c < cols) {
#pragma unroll 8
        for (int b = slice; b < static_cast<int>(gridDim.x); b += slices)
          v += __ldcg(a.partial + static_cast<long long>(b) * 2 * a.D + c);
      }
      __syncthreads();
      sums[threadIdx.x] = v;
      __syncthreads();
      if (threadIdx.x < 64 && c < cols) {
        for (int i = 1; i < slices; ++i) v += sums[i * 64 + threadIdx.x];
        if (c < a.D)
          a.dwq[c] = v;
        else
          a.dwk[c - a.D] = v;
      }
    }
    if (threadIdx.x == 0) *a.done = 0;
  }
  allow_next_grid();
}

// ------------------------------------------------------------ host side

View view_of(const pv_heads* h, int elem) {
  View v{};
  if (h) v = View{static_cast<char*>(h->data), h->row_stride * elem, h->head_stride * elem};
  return v;
}

int check_params(const pv_rope_params* p, int* dev) {
  if (!p) return PV_ERR_INVALID;
  if (!dtype_size(p->dtype) || p->rows < 0 || p->rows >= (int64_t(1) << 31)) return PV_ERR_INVALID;
  if (p->q_heads < 1 || p->k_heads < 0 || p->q_heads > 4096 || p->k_heads > 4096) return PV_ERR_INVALID;
  if (p->head_dim < 16 || p->head_dim > 256 || p->head_dim % 16) return PV_ERR_INVALID;
  if (p->axes < 1 || p->axes > 3 || p->position_stride < p->axes) return PV_ERR_INVALID;
  if (!(p->eps >= 0.0f) || !std::isfinite(p->eps)) return PV_ERR_INVALID;
  if (!p->q_weight || !p->inv_freq || (p->k_heads && !p->k_weight) || (p->rows && !p->positions))
    return PV_ERR_INVALID;
  if (!aligned(p->q_weight, 4) || !aligned(p->k_weight, 4) || !aligned(p->inv_freq, 4) || !aligned(p->positions, 4))
    return PV_ERR_INVALID;
  *dev = device_of(p->q_weight);
  if (*dev < 0 || device_of(p->inv_freq) != *dev || (p->k_heads && device_of(p->k_weight) != *dev) ||
      (p->rows && device_of(p->positions) != *dev))
    return PV_ERR_INVALID;
  return PV_OK;
}

RopeArgs args_of(const pv_rope_params* p) {
  RopeArgs a{};
  a.wq = p->q_weight;
  a.wk = p->k_weight;
  a.pos = p->positions;
  a.pos_stride = p->position_stride;
  a.freq = p->inv_freq;
  a.rows = static_cast<int>(p->rows);
  a.hq = p->q_heads;
  a.hk = p->k_heads;
  a.D = p->head_dim;
  a.axes = p->axes;
  a.eps = p->eps;
  const int per = 16 / dtype_size(p->dtype);
  while ((per << a.lanes_log2) < a.D / 2) ++a.lanes_log2;
  return a;
}

// Tokens of a tile: as many as the table holds, fewer so that `blocks` blocks take
// equally many tiles.  (Every tile begins with its table and a round of loads that
// nothing hides: tiles of four rounds took the backward pass 166 us for 96,001 rows of
// 2 x 8 heads of 64 in bf16, tiles of ten 155 us.)
int tile_tokens(const RopeArgs& a, int blocks) {
  const long long most = kTableFloats / a.D;
  const long long turns = std::max<long long>(1, (a.rows + blocks * most - 1) / (blocks * most));
  return static_cast<int>(std::max<long long>(1, (a.rows + blocks * turns - 1) / (blocks * turns)));
}

template <typename K>
int launch(K kernel, int blocks, const RopeArgs& a, pv_stream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return PV_ERR_CUDA;
  }
  return PV_OK;
}

}  // namespace

extern "C" int pv_qk_norm_rope(const pv_rope_params* params, const pv_heads* q, const pv_heads* k,
                               const pv_heads* out_q, const pv_heads* out_k, pv_stream_t stream) try {
  int dev = 0, st = check_params(params, &dev);
  if (st != PV_OK) return st;
  const int elem = dtype_size(params->dtype);
  if ((st = check_heads(q, params->rows, params->q_heads, elem, dev)) != PV_OK ||
      (st = check_out_heads(out_q, params->rows, params->q_heads, elem, dev)) != PV_OK)
    return st;
  if (params->k_heads && ((st = check_heads(k, params->rows, params->k_heads, elem, dev)) != PV_OK ||
                          (st = check_out_heads(out_k, params->rows, params->k_heads, elem, dev)) != PV_OK))
    return st;
  if (params->rows == 0) return PV_OK;
  DeviceScope scope(dev);
  const int sms = sm_count(dev);
  if (!scope.ok() || sms < 1) return PV_ERR_CUDA;
  RopeArgs a = args_of(params);
  a.q = view_of(q, elem);
  a.k = view_of(k, elem);
  a.oq = view_of(out_q, elem);
  a.ok = view_of(out_k, elem);
  a.tile = tile_tokens(a, kPerSm * sms);
  const int blocks = tiles_of(a);
  switch (params->dtype) {
    case PV_F32: return launch(pv_rope_kernel<float>, blocks, a, stream);
    case PV_BF16: return launch(pv_rope_kernel<__nv_bfloat16>, blocks, a, stream);
    default: return launch(pv_rope_kernel<__half>, blocks, a, stream);
  }
} catch (...) {
  return caught();
}

extern "C" int pv_qk_norm_rope_backward(const pv_rope_params* params, const pv_heads* dout_q, const pv_heads* dout_k,
                                        const pv_heads* q, const pv_heads* k, const pv_heads* dq, const pv_heads* dk,
                                        float* dq_weight, float* dk_weight, pv_stream_t stream) try {
  int dev = 0, st = check_params(params, &dev);
  if (st != PV_OK) return st;
  const int elem = dtype_size(params->dtype);
  for (const pv_heads* h : {dout_q, q})
    if ((st = check_heads(h, params->rows, params->q_heads, elem, dev)) != PV_OK) return st;
  if ((st = check_out_heads(dq, params->rows, params->q_heads, elem, dev)) != PV_OK) return st;
  if (params->k_heads) {
    for (const pv_heads* h : {dout_k, k})
      if ((st = check_heads(h, params->rows, params->k_heads, elem, dev)) != PV_OK) return st;
    if ((st = check_out_heads(dk, params->rows, params->k_heads, elem, dev)) != PV_OK) return st;
  }
  if (!dq_weight || !aligned(dq_weight, 4) || device_of(dq_weight) != dev) return PV_ERR_INVALID;
  if (params->k_heads && (!dk_weight || !aligned(dk_weight, 4) || device_of(dk_weight) != dev)) return PV_ERR_INVALID;
  DeviceScope scope(dev);
  const int sms = sm_count(dev);
  if (!scope.ok() || sms < 1) return PV_ERR_CUDA;
  RopeArgs a = args_of(params);
  a.q = view_of(q, elem);
  a.k = view_of(k, elem);
  a.gq = view_of(dout_q, elem);
  a.gk = view_of(dout_k, elem);
  a.oq = view_of(dq, elem);
  a.ok = view_of(dk, elem);
  a.dwq = dq_weight;
  a.dwk = dk_weight;
  const int most = std::min(kMaxBlocks, kPerSmBack * sms);
  a.tile = tile_tokens(a, most);
  const int blocks = std::max(1, std::min(most, tiles_of(a)));
  Scratch scratch;
  if ((st = scratch.open(dev, stream, kPlain, sizeof(float) * 2 * a.D * static_cast<size_t>(blocks))) != PV_OK)
    return st;
  a.partial = static_cast<float*>(scratch.body());
  a.done = static_cast<unsigned int*>(scratch.head());
  switch (params->dtype) {
    case PV_F32: return launch(pv_rope_backward_kernel<float>, blocks, a, stream);
    case PV_BF16: return launch(pv_rope_backward_kernel<__nv_bfloat16>, blocks, a, stream);
    default: return launch(pv_rope_backward_kernel<__half>, blocks, a, stream);
  }
} catch (...) {
  return caught();
}
