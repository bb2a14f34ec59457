// Root-mean-square norm of rows with the residual's addition in front of it, its
// output in the rows' type or in 8 bits, and its backward pass (pv_rms_norm,
// pv_rms_norm_8bit, pv_rms_norm_backward in pv.h).
//
//   h = x + residual (rounded to the rows' type: it is the next layer's residual);
//   r = 1 / sqrt(mean(h^2) + eps);  n = h r;  y = n w.
//   8 bits: scale = max |y| / 448 over a group of channels, values e4m3(y / scale).
//   dx = r (g - n mean(g n)) + dh, g = dy w;  dw = sum over rows of dy n.
//
// One pass over memory each way, which bounds it: a row stays in the registers of the
// lanes that share it (8 to 512 of them, by its length), eight channels a pack.  The
// blocks are persistent, so that the weight is read once a block and its gradient is
// summed in registers, then block by block in a fixed order by a second kernel.
// In a row through the Python entries: 96,001 rows of 512 in bfloat16, forward 63 us (6.3 TB/s of its bytes), backward 64
// with the join (6.1 TB/s); 24,571 rows of 1,024 to 8 bits 34 us (5.1 TB/s).

#include "pv_seq.cuh"

#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

namespace {

using namespace pvs;

constexpr int kV = 8;  // channels of a pack
constexpr int64_t kMostChannels = 16384;

struct NormArgs {
  const char* x;
  const char* res;
  const char* dy;
  const char* dh;
  char* y;
  char* h;  // backward: dx
  const float* w;
  float* scales;   // 8 bits: [rows, groups]
  float* partial;  // backward: [blocks, C]
  float* dw;
  long long x_row, res_row, dy_row, dh_row, y_row, h_row;  // strides in bytes
  long long rows;
  int C, groups;
  int lanes_log2;        // lanes of a row
  int group_lanes_log2;  // 8 bits: lanes of a group of channels
  float eps;
};

enum Form { kPlainOut, k8Bit };

// Channels c .. c + 8 of a row; the scalar form takes rows of any alignment and length.
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const char* row, int c, int C, float* f) {
  const T* p = reinterpret_cast<const T*>(row) + c;
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kV; i += Pack<T>::kN) Pack<T>::load(p + i, f + i);
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i) f[i] = c + i < C ? Pack<T>::to(p[i]) : 0.0f;
  }
}
template <typename T, bool kVec>
__device__ __forceinline__ void store8(char* row, int c, int C, const float* f) {
  T* p = reinterpret_cast<T*>(row) + c;
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kV; i += Pack<T>::kN) Pack<T>::store(p + i, f + i);
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (c + i < C) p[i] = Pack<T>::one(f[i]);
  }
}

// The maximum, or no number if one of them is none.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// Joins kN values over the lanes of a row: within a warp by shuffles, across the warps of
// a longer row through shared memory, in the same order on every lane.  `turn` alternates between
// two places, so that one barrier a call is enough.
template <int kN, bool kMax, int kThreads>
__device__ __forceinline__ void join_row(float* v, int lanes, float (*shared)[kThreads / 32][2], int turn) {
  const int within = min(lanes, 32);
  for (int o = within >> 1; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float u = __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
      v[i] = kMax ? max_nan(v[i], u) : v[i] + u;
    }
  if (lanes <= 32) return;
  const int warp = threadIdx.x >> 5, warps = lanes >> 5, first = warp & ~(warps - 1);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < kN; ++i) shared[turn][warp][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = shared[turn][first][i];
  for (int j = 1; j < warps; ++j)
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float u = shared[turn][first + j][i];
      v[i] = kMax ? max_nan(v[i], u) : v[i] + u;
    }
}

// What y is divided by to 8 bits: scale = most / 448, rounded once (never 0, so that rows of zeros are zeros; what is not finite
// stays so), and 1 / scale in two parts, so that y low + y high gives the e4m3 values that y / scale rounded to 32 bits has.
//   scale: 1 / 448 in two parts is good to 2^-47, and no quotient by 448 comes as near to the middle of two floats (7 times
//     the distance is a whole number of 2^-25 of the value, and not 0).
//   high is below 1 / scale by less than 2^-21 of it (so that low is not negative, and zeros keep their sign); what is left, e, the sum e + e^2,
//     low and its product with y are rounded, each off by less than 2^-24 2^-21: together by less than d = 2^-43 of the quotient.
//   Rounded to 32 bits this falls on the other side of a border b 2^x of two e4m3 values (16 <= b < 32) than the quotient
//     does only if the quotient is within d of the middle of the border and the next float, (b +- 2^-20) 2^x (below b = 16 b - 2^-21).  With
//     S the scale's 24 bits as a whole number, its distance from there is |N -+ S 2^-20| / (b S), N a whole number: at least
//     64 2^-20 / 2^29 = 2^-43 where S is 64 or more from a multiple of 2^20 (S 2^-21 likewise, b S being half as large).
// One scale in 2^12 is not, and is divided by, as are those of sizes at which a product here may fall short of 2^-126.
// (24,571 x 1,024 bfloat16, groups of 128: 31.5 us with products by a rounded reciprocal, which take one value in some 10^6 to the
// wrong side, 34.4 like this, 43.6 with a division each; a scale for each row: 30.4, 30.5 and 38.5.)
struct Quotients {
  float scale, high, low;
  bool quick;
  __device__ __forceinline__ explicit Quotients(float most) {
    constexpr double k = 1.0 / 448.0;
    constexpr float kHigh = static_cast<float>(k), kLow = static_cast<float>(k - static_cast<double>(kHigh));
    constexpr uint32_t kFrom = (127u - 90) << 23, kTo = (127u + 90) << 23;  // 2^-90, 2^90
    scale = fmaf(most, kHigh, most * kLow);
    quick = __float_as_uint(most) - kFrom < kTo - kFrom && ((__float_as_uint(scale) + 128) & 0xFFFFF) > 256;
    if (!quick) scale = max_nan(most / 448.0f, 1.17549435e-38f);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(high) : "f"(scale));  // (good to 2^-23)
    high *= 1.0f - 0x1p-22f;
    const float e = fmaf(-scale, high, 1.0f);
    low = high * fmaf(e, e, e);
  }
};

// Channels c .. c + 8 as they lie in memory, opened where they are used.
template <typename T, bool kVec>
struct Row8 {
  uint4 v[kV / Pack<T>::kN];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kV / Pack<T>::kN; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const char* row, int c, int C) {
    const T* p = reinterpret_cast<const T*>(row) + c;
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < kV / Pack<T>::kN; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
      float f[kV];
      load8<T, false>(row, c, C, f);
      take(f);
    }
  }
  __device__ __forceinline__ void take(const float* f) {
#pragma unroll
    for (int i = 0; i < kV / Pack<T>::kN; ++i) Pack<T>::store(&v[i], f + i * Pack<T>::kN);
  }
  __device__ __forceinline__ void open(float* f) const {
#pragma unroll
    for (int i = 0; i < kV / Pack<T>::kN; ++i) Pack<T>::open(v[i], f + i * Pack<T>::kN);
  }
};

// Blocks of 256 threads on a multiprocessor, and whether the next row's loads are issued ahead of the work on one: as many bytes
// in flight as registers allow, by measurement.  Forward, 16 bits: 150,000 x 256 62 us with 4 blocks, 49 with 6, to
// 8 bits 56 with 5, 49 with 4 and loads ahead; 96,001 x 512 62 with 3 and 66 with loads ahead, to 8 bits 62 with 4, 56 with 3 and loads
// ahead; 17,000 x 3,000 74 with 2, 64 with loads ahead, to 8 bits 92 and 73.  32 bits: 60,000 x 512 83 with 2,
// 91 with 3 blocks.  Backward, 16 bits: 96,001 x 512 78 with 3, 64 with 2 and loads ahead; 25,000 x 2,048 95 with 1, 72 with
// loads ahead, but 4,000 x 16,384 in 512 threads, whose rows and sums of the weight's gradient do not fit into 128 registers as it
// is (356 bytes a thread spilled, 464 with 32 bits), 145 without, 200 with.  32 bits: 60,000 x 512 85 with 3, 74 with 2 blocks and 86 with loads ahead.
template <typename T, int kP, int kForm>
constexpr int kBlocks = kP == 4 ? 2 : kP == 2 ? (sizeof(T) == 4 ? 2 : 3) : kForm == kPlainOut ? 6 : 4;
template <typename T, int kP, bool kVec, int kForm>
constexpr bool kLoadsAhead = kVec && (kForm == kPlainOut ? kP == 4 && sizeof(T) == 2 : kP == 1 || sizeof(T) == 2);
template <typename T, int kP, bool kVec>
constexpr bool kLoadsAheadBack = kVec && kP >= 2 && sizeof(T) == 2;

// Rows stay packed from their sum to the result, opened twice, so that more of them are in flight (24,571 x 1,024 bfloat16 to 8 bits:
// 47 us with rows of floats, 37 packed, 32 with the next row's loads ahead; 96,001 x 512: 98, 62 and 56).
template <typename T, int kP, bool kVec, int kThreads, int kForm>
__global__ void __launch_bounds__(kThreads, kVec && kThreads == 256 ? kBlocks<T, kP, kForm> : 1) pv_norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float shared[2][kThreads / 32][2];
  const int lanes = 1 << a.lanes_log2, lane = threadIdx.x & (lanes - 1);
  const int here = kThreads >> a.lanes_log2, own = threadIdx.x >> a.lanes_log2;
  wait_prior_grid();
  float w[kP][kV];
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    const int c = (j * lanes + lane) * kV;
#pragma unroll
    for (int i = 0; i < kV; ++i) w[j][i] = c + i < a.C ? a.w[c + i] : 0.0f;
  }
  const float inv_c = 1.0f / static_cast<float>(a.C);
  int turn = 0;
  // (Every thread of a block goes round equally often: longer rows meet at barriers.)
  const long long step = static_cast<long long>(gridDim.x) * here, start = static_cast<long long>(blockIdx.x) * here;
  Row8<T, kVec> xn[kP], un[kP];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      const int c = (j * lanes + lane) * kV;
      xn[j].clear();
      if (row >= a.rows || c >= a.C) continue;
      xn[j].load(a.x + row * a.x_row, c, a.C);
      if (a.res) un[j].load(a.res + row * a.res_row, c, a.C);
    }
  };
  constexpr bool kAhead = kLoadsAhead<T, kP, kVec, kForm>;
  if constexpr (kAhead) fetch(start + own);
  for (long long r0 = start; r0 < a.rows; r0 += step) {
    const long long row = r0 + own;
    const bool on = row < a.rows;
    if constexpr (!kAhead) fetch(row);
    Row8<T, kVec> x[kP];
    float v[2] = {};
#pragma unroll
    for (int j = 0; j < kP; ++j) x[j] = xn[j];
    if (a.res && on) {
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        const int c = (j * lanes + lane) * kV;
        if (c >= a.C) continue;
        // Rounded: what is normalised, here and backward, is the sum that is kept.
        float xs[kV], us[kV];
        x[j].open(xs), un[j].open(us);
#pragma unroll
        for (int i = 0; i < kV; i += 2) add2(xs[i], xs[i + 1], xs[i], xs[i + 1], us[i], us[i + 1]);
        x[j].take(xs);
        x[j].open(xs);
        store8<T, kVec>(a.h + row * a.h_row, c, a.C, xs);
      }
    }
    if constexpr (kAhead) fetch(row + step);
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      float xs[kV];
      x[j].open(xs);
#pragma unroll
      for (int i = 0; i < kV; i += 2) fma2(v[0], v[1], xs[i], xs[i + 1], xs[i], xs[i + 1], v[0], v[1]);
    }
    v[0] += v[1];
    join_row<1, false, kThreads>(v, lanes, shared, turn);
    turn ^= 1;
    const float r = 1.0f / sqrtf(fmaf(v[0], inv_c, a.eps));
    auto result = [&](int j, float* y) {
      x[j].open(y);
#pragma unroll
      for (int i = 0; i < kV; i += 2) {
        mul2(y[i], y[i + 1], y[i], y[i + 1], r, r);
        mul2(y[i], y[i + 1], y[i], y[i + 1], w[j][i], w[j][i + 1]);
      }
    };
    if constexpr (kForm == kPlainOut) {
      if (on) {
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          const int c = (j * lanes + lane) * kV;
          if (c >= a.C) continue;
          float y[kV];
          result(j, y);
          store8<T, kVec>(a.y + row * a.y_row, c, a.C, y);
        }
      }
    } else {
      // (Lanes past the last channel hold zeros, which are no one's maximum; with r
      // infinite they hold no numbers, as the row does, and are left out.)
      auto largest = [&](int j, const float* y) {
        float most = 0.0f;
        const int c = (j * lanes + lane) * kV;
#pragma unroll
        for (int i = 0; i < kV; ++i)
          if (kVec || c + i < a.C) most = max_nan(most, fabsf(y[i]));
        return c < a.C ? most : 0.0f;
      };
      auto put = [&](int j, const float* y, float most) {
        const int p = j * lanes + lane, c = p * kV;
        if (!on || c >= a.C) return;
        unsigned short b[kV / 2];
        const Quotients by(most);
        const float scale = by.scale;
        if ((p & ((1 << a.group_lanes_log2) - 1)) == 0 && (a.groups > 1 || p == 0))
          a.scales[row * a.groups + (a.groups > 1 ? p >> a.group_lanes_log2 : 0)] = scale;
        if (by.quick) {
#pragma unroll
          for (int i = 0; i < kV; i += 2) {
            float q0, q1;
            mul2(q0, q1, y[i], y[i + 1], by.low, by.low);
            fma2(q0, q1, y[i], y[i + 1], by.high, by.high, q0, q1);
            b[i / 2] = __nv_cvt_float2_to_fp8x2(make_float2(q0, q1), __NV_SATFINITE, __NV_E4M3);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kV; i += 2) b[i / 2] = __nv_cvt_float2_to_fp8x2(make_float2(y[i] / scale, y[i + 1] / scale), __NV_SATFINITE, __NV_E4M3);
        }
        unsigned char* out = reinterpret_cast<unsigned char*>(a.y + row * a.y_row) + c;
        if constexpr (kVec) {
          *reinterpret_cast<uint2*>(out) = make_uint2(b[0] | static_cast<uint32_t>(b[1]) << 16, b[2] | static_cast<uint32_t>(b[3]) << 16);
        } else {
#pragma unroll
          for (int i = 0; i < kV; ++i)
            if (c + i < a.C) out[i] = static_cast<unsigned char>(b[i / 2] >> (i & 1) * 8);
        }
      };
      if (a.groups > 1) {
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          float y[kV];
          result(j, y);
          float most = largest(j, y);
          for (int o = (1 << a.group_lanes_log2) >> 1; o; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
          put(j, y, most);
        }
      } else {
        float most = 0.0f, y[kV];
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          result(j, y);
          most = max_nan(most, largest(j, y));
        }
        join_row<1, true, kThreads>(&most, lanes, shared, turn);
        turn ^= 1;
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          result(j, y);
          put(j, y, most);
        }
      }
    }
  }
  allow_next_grid();
}

template <typename T, int kP, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 && kP <= 2 ? (kP == 1 ? 4 : 2) : 1) pv_norm_backward_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float shared[2][kThreads / 32][2];
  __shared__ float sums[kThreads * kV];
  const int lanes = 1 << a.lanes_log2, lane = threadIdx.x & (lanes - 1);
  const int here = kThreads >> a.lanes_log2, own = threadIdx.x >> a.lanes_log2;
  wait_prior_grid();
  float w[kP][kV], dw[kP][kV] = {};
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    const int c = (j * lanes + lane) * kV;
#pragma unroll
    for (int i = 0; i < kV; ++i) w[j][i] = c + i < a.C ? a.w[c + i] : 0.0f;
  }
  const float inv_c = 1.0f / static_cast<float>(a.C);
  int turn = 0;
  const long long step = static_cast<long long>(gridDim.x) * here, start = static_cast<long long>(blockIdx.x) * here;
  Row8<T, kVec> xn[kP], gn[kP], en[kP];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      const int c = (j * lanes + lane) * kV;
      xn[j].clear(), gn[j].clear(), en[j].clear();
      if (row >= a.rows || c >= a.C) continue;
      xn[j].load(a.x + row * a.x_row, c, a.C);
      gn[j].load(a.dy + row * a.dy_row, c, a.C);
      if (a.dh) en[j].load(a.dh + row * a.dh_row, c, a.C);
    }
  };
  constexpr bool kAhead = kLoadsAheadBack<T, kP, kVec> && kThreads == 256;
  if constexpr (kAhead) fetch(start + own);
  for (long long r0 = start; r0 < a.rows; r0 += step) {
    const long long row = r0 + own;
    const bool on = row < a.rows;
    if constexpr (!kAhead) fetch(row);
    Row8<T, kVec> x[kP], g[kP], e[kP];
#pragma unroll
    for (int j = 0; j < kP; ++j) x[j] = xn[j], g[j] = gn[j], e[j] = en[j];
    if constexpr (kAhead) fetch(row + step);
    float v[2], u[2] = {}, t[2] = {};
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      float xs[kV], gs[kV];
      x[j].open(xs), g[j].open(gs);
#pragma unroll
      for (int i = 0; i < kV; i += 2) {
        float p0, p1;
        fma2(u[0], u[1], xs[i], xs[i + 1], xs[i], xs[i + 1], u[0], u[1]);
        mul2(p0, p1, gs[i], gs[i + 1], w[j][i], w[j][i + 1]);
        fma2(t[0], t[1], p0, p1, xs[i], xs[i + 1], t[0], t[1]);
      }
    }
    v[0] = u[0] + u[1];
    v[1] = t[0] + t[1];
    join_row<2, false, kThreads>(v, lanes, shared, turn);
    turn ^= 1;
    const float r = 1.0f / sqrtf(fmaf(v[0], inv_c, a.eps));
    const float mean = -(v[1] * inv_c) * r;  // of g n, negated
    if (!on) continue;
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      const int c = (j * lanes + lane) * kV;
      if (c >= a.C) continue;
      float xs[kV], gs[kV], es[kV];
      x[j].open(xs), g[j].open(gs), e[j].open(es);
#pragma unroll
      for (int i = 0; i < kV; i += 2) {
        float n0, n1, p0, p1;
        mul2(n0, n1, xs[i], xs[i + 1], r, r);
        fma2(dw[j][i], dw[j][i + 1], gs[i], gs[i + 1], n0, n1, dw[j][i], dw[j][i + 1]);
        mul2(p0, p1, gs[i], gs[i + 1], w[j][i], w[j][i + 1]);
        fma2(p0, p1, n0, n1, mean, mean, p0, p1);
        fma2(es[i], es[i + 1], p0, p1, r, r, es[i], es[i + 1]);
      }
      store8<T, kVec>(a.h + row * a.h_row, c, a.C, es);
    }
  }
  // The rows that the block has taken in turn, joined in order, pack by pack.
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kV; ++i) sums[i * kThreads + threadIdx.x] = dw[j][i];
    __syncthreads();
    for (int k = threadIdx.x; k < lanes * kV; k += kThreads) {
      const int l = k >> 3, i = k & 7, c = (j * lanes + l) * kV + i;
      float s = 0.0f;
      for (int o = 0; o < here; ++o) s += sums[i * kThreads + o * lanes + l];
      if (c < a.C) a.partial[static_cast<long long>(blockIdx.x) * a.C + c] = s;
    }
  }
  allow_next_grid();
}

// The blocks' sums of the weight's gradient, joined in order: 32 channels a block.
__global__ void __launch_bounds__(1024) pv_norm_weight_kernel(const float* partial, float* dw, int blocks, int C) {
  __shared__ float sums[32][33];
  wait_prior_grid();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float s = 0.0f;
  if (c < C) {
#pragma unroll 8
    for (int b = slice; b < blocks; b += 32) s += partial[static_cast<long long>(b) * C + c];
  }
  sums[slice][threadIdx.x & 31] = s;
  __syncthreads();
  if (slice == 0 && c < C) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sums[i][threadIdx.x];
    dw[c] = s;
  }
  allow_next_grid();
}

// ------------------------------------------------------------ host side

int check_rows(const void* p, int64_t stride, int64_t rows, int64_t C, int elem, int dev, bool written) {
  if (rows == 0) return PV_OK;
  if (!p || !aligned(p, elem) || device_of(p) != dev) return PV_ERR_INVALID;
  if (stride >= C || (rows == 1 && stride >= 0)) return PV_OK;
  return stride == 0 && !written ? PV_OK : PV_ERR_INVALID;
}

// A result in the place of an input has to have its rows, too.
bool in_place(const void* out, int64_t out_stride, const void* in, int64_t in_stride, int64_t rows) {
  return out != in || rows <= 1 || out_stride == in_stride;
}

int check_params(const pv_norm_params* p, int* dev) {
  if (!p || !dtype_size(p->dtype) || p->rows < 0 || p->rows >= (int64_t(1) << 31)) return PV_ERR_INVALID;
  if (p->channels < 1 || p->channels > kMostChannels || !(p->eps >= 0.0f) || !std::isfinite(p->eps)) return PV_ERR_INVALID;
  if (!p->weight || !aligned(p->weight, 4) || (*dev = device_of(p->weight)) < 0) return PV_ERR_INVALID;
  const int elem = dtype_size(p->dtype);
  const int st = check_rows(p->x, p->x_stride, p->rows, p->channels, elem, *dev, false);
  return st == PV_OK && p->residual ? check_rows(p->residual, p->residual_stride, p->rows, p->channels, elem, *dev, false) : st;
}

NormArgs args_of(const pv_norm_params* p) {
  const int elem = dtype_size(p->dtype);
  NormArgs a{};
  a.x = static_cast<const char*>(p->x);
  a.x_row = p->x_stride * elem;
  a.res = static_cast<const char*>(p->residual);
  a.res_row = p->residual_stride * elem;
  a.w = p->weight;
  a.rows = p->rows;
  a.C = static_cast<int>(p->channels);
  a.groups = 1;
  a.eps = p->eps;
  return a;
}

bool wide(const void* p, int64_t stride_bytes) { return !p || (aligned(p, 16) && stride_bytes % 16 == 0); }

// The variant of a row length: how many packs a thread holds (kP), and how many lanes
// share a row, the fewest powers of two that hold it.  One and two packs for the short
// rows of many tokens (more rows in flight); the scalar form has one variant, of four.
template <template <typename, int, bool, int> class Go, typename T>
int pick(NormArgs& a, bool vec, int dev, pv_stream_t stream) {
  const int packs = (a.C + kV - 1) / kV;
  const int kp = !vec ? 4 : packs <= 32 ? 1 : packs <= 64 ? 2 : 4;
  while ((kp << a.lanes_log2) < packs) ++a.lanes_log2;
  a.lanes_log2 = std::max({a.lanes_log2, a.group_lanes_log2, 3});
  const bool longest = a.lanes_log2 > 8;  // 512 lanes
  if (!vec) return longest ? Go<T, 4, false, 512>::go(a, dev, stream) : Go<T, 4, false, 256>::go(a, dev, stream);
  if (kp == 1) return Go<T, 1, true, 256>::go(a, dev, stream);
  if (kp == 2) return Go<T, 2, true, 256>::go(a, dev, stream);
  return longest ? Go<T, 4, true, 512>::go(a, dev, stream) : Go<T, 4, true, 256>::go(a, dev, stream);
}

// Blocks of a launch: as many as are resident at once (`each` on a multiprocessor), or as the rows need.
int blocks_of(const NormArgs& a, int each, int threads, int dev) {
  const int here = threads >> a.lanes_log2;
  return static_cast<int>(std::max<long long>(1, std::min<long long>(static_cast<long long>(each) * sm_count(dev), (a.rows + here - 1) / here)));
}

template <typename K>
int resident(K kernel, int threads) {
  int each = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&each, kernel, threads, 0) == cudaSuccess && each > 0) return each;
  cudaGetLastError();
  return 1;
}

template <typename... K, typename... A>
int launch(void (*kernel)(K...), int blocks, int threads, pv_stream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
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

template <typename T, int kP, bool kVec, int kThreads, int kForm>
int go_forward(const NormArgs& a, int dev, pv_stream_t stream) {
  auto kernel = pv_norm_kernel<T, kP, kVec, kThreads, kForm>;
  static const int each = resident(kernel, kThreads);
  return launch(kernel, blocks_of(a, each, kThreads, dev), kThreads, stream, a);
}
template <typename T, int kP, bool kVec, int kThreads>
struct Forward {
  static int go(const NormArgs& a, int dev, pv_stream_t stream) { return go_forward<T, kP, kVec, kThreads, kPlainOut>(a, dev, stream); }
};
template <typename T, int kP, bool kVec, int kThreads>
struct To8Bit {
  static int go(const NormArgs& a, int dev, pv_stream_t stream) { return go_forward<T, kP, kVec, kThreads, k8Bit>(a, dev, stream); }
};
template <typename T, int kP, bool kVec, int kThreads>
struct Backward {
  static int go(NormArgs& a, int dev, pv_stream_t stream) {
    auto kernel = pv_norm_backward_kernel<T, kP, kVec, kThreads>;
    static const int each = resident(kernel, kThreads);
    const int blocks = blocks_of(a, each, kThreads, dev);
    Scratch scratch;
    int st = scratch.open(dev, stream, kPlain, sizeof(float) * static_cast<size_t>(blocks) * a.C);
    if (st != PV_OK) return st;
    a.partial = static_cast<float*>(scratch.body());
    if ((st = launch(kernel, blocks, kThreads, stream, a)) != PV_OK) return st;
    return launch(pv_norm_weight_kernel, (a.C + 31) / 32, 1024, stream, static_cast<const float*>(a.partial), a.dw, blocks, a.C);
  }
};

template <template <typename, int, bool, int> class Go>
int by_type(NormArgs& a, int dtype, bool vec, int dev, pv_stream_t stream) {
  if (sm_count(dev) < 1) return PV_ERR_CUDA;
  switch (dtype) {
    case PV_F32: return pick<Go, float>(a, vec, dev, stream);
    case PV_BF16: return pick<Go, __nv_bfloat16>(a, vec, dev, stream);
    default: return pick<Go, __half>(a, vec, dev, stream);
  }
}

}  // namespace

extern "C" int pv_rms_norm(const pv_norm_params* params, void* y, int64_t y_stride, void* h, int64_t h_stride,
                           pv_stream_t stream) try {
  int dev = 0, st = check_params(params, &dev);
  if (st != PV_OK) return st;
  const int elem = dtype_size(params->dtype);
  if ((st = check_rows(y, y_stride, params->rows, params->channels, elem, dev, true)) != PV_OK) return st;
  if (params->residual && (st = check_rows(h, h_stride, params->rows, params->channels, elem, dev, true)) != PV_OK) return st;
  if (params->rows == 0) return PV_OK;
  if (!in_place(y, y_stride, params->x, params->x_stride, params->rows)) return PV_ERR_INVALID;
  if (params->residual && (y == h || !in_place(y, y_stride, params->residual, params->residual_stride, params->rows) ||
                           !in_place(h, h_stride, params->x, params->x_stride, params->rows) ||
                           !in_place(h, h_stride, params->residual, params->residual_stride, params->rows)))
    return PV_ERR_INVALID;
  DeviceScope scope(dev);
  if (!scope.ok()) return PV_ERR_CUDA;
  NormArgs a = args_of(params);
  a.y = static_cast<char*>(y);
  a.y_row = y_stride * elem;
  if (a.res) a.h = static_cast<char*>(h), a.h_row = h_stride * elem;
  const bool vec = a.C % kV == 0 && wide(a.x, a.x_row) && wide(a.res, a.res_row) && wide(a.y, a.y_row) && wide(a.h, a.h_row);
  return by_type<Forward>(a, params->dtype, vec, dev, stream);
} catch (...) {
  return caught();
}

extern "C" int pv_rms_norm_8bit(const pv_norm_params* params, int group, void* values, float* scales, void* h,
                                int64_t h_stride, pv_stream_t stream) try {
  int dev = 0, st = check_params(params, &dev);
  if (st != PV_OK) return st;
  if (group != 0 && group != 32 && group != 64 && group != 128) return PV_ERR_INVALID;
  const int elem = dtype_size(params->dtype);
  if ((st = check_rows(values, params->channels, params->rows, params->channels, 1, dev, true)) != PV_OK) return st;
  if (params->residual && (st = check_rows(h, h_stride, params->rows, params->channels, elem, dev, true)) != PV_OK) return st;
  if (params->rows && (!scales || !aligned(scales, 4) || device_of(scales) != dev)) return PV_ERR_INVALID;
  if (params->rows == 0) return PV_OK;
  if (params->residual && (!in_place(h, h_stride, params->x, params->x_stride, params->rows) ||
                           !in_place(h, h_stride, params->residual, params->residual_stride, params->rows)))
    return PV_ERR_INVALID;
  DeviceScope scope(dev);
  if (!scope.ok()) return PV_ERR_CUDA;
  NormArgs a = args_of(params);
  a.y = static_cast<char*>(values);
  a.y_row = a.C;
  a.scales = scales;
  if (a.res) a.h = static_cast<char*>(h), a.h_row = h_stride * elem;
  // A group is 4, 8 or 16 lanes next to one another (a row that one group covers is
  // joined as a row).
  if (group) a.groups = (a.C + group - 1) / group;
  if (a.groups > 1)
    while ((kV << a.group_lanes_log2) < group) ++a.group_lanes_log2;
  const bool vec = a.C % kV == 0 && wide(a.x, a.x_row) && wide(a.res, a.res_row) && wide(a.h, a.h_row) && aligned(values, 8);
  return by_type<To8Bit>(a, params->dtype, vec, dev, stream);
} catch (...) {
  return caught();
}

extern "C" int pv_rms_norm_backward(const pv_norm_params* params, const void* dy, int64_t dy_stride, const void* dh,
                                    int64_t dh_stride, void* dx, int64_t dx_stride, float* dweight, pv_stream_t stream) try {
  int dev = 0, st = check_params(params, &dev);
  if (st != PV_OK) return st;
  if (params->residual) return PV_ERR_INVALID;  // x is the sum
  const int elem = dtype_size(params->dtype);
  if ((st = check_rows(dy, dy_stride, params->rows, params->channels, elem, dev, false)) != PV_OK ||
      (st = check_rows(dx, dx_stride, params->rows, params->channels, elem, dev, true)) != PV_OK ||
      (dh && (st = check_rows(dh, dh_stride, params->rows, params->channels, elem, dev, false)) != PV_OK))
    return st;
  if (!dweight || !aligned(dweight, 4) || device_of(dweight) != dev) return PV_ERR_INVALID;
  if (!in_place(dx, dx_stride, dy, dy_stride, params->rows) || (dh && !in_place(dx, dx_stride, dh, dh_stride, params->rows)) ||
      !in_place(dx, dx_stride, params->x, params->x_stride, params->rows))
    return PV_ERR_INVALID;
  DeviceScope scope(dev);
  if (!scope.ok()) return PV_ERR_CUDA;
  NormArgs a = args_of(params);
  a.dy = static_cast<const char*>(dy);
  a.dy_row = dy_stride * elem;
  a.dh = static_cast<const char*>(dh);
  a.dh_row = dh_stride * elem;
  a.h = static_cast<char*>(dx);
  a.h_row = dx_stride * elem;
  a.dw = dweight;
  const bool vec = a.C % kV == 0 && wide(a.x, a.x_row) && wide(a.dy, a.dy_row) && wide(a.dh, a.dh_row) && wide(a.h, a.h_row);
  return by_type<Backward>(a, params->dtype, vec, dev, stream);
} catch (...) {
  return caught();
}
