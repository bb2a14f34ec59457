// Softmax cross entropy over a large vocabulary whose logits are never kept, and its
// backward pass (pv_cross_entropy, pv_cross_entropy_backward in pv.h).
//
//   z[t][v] = x[t] . w[v];  lse[t] = log sum_v exp(z[t][v]);  loss[t] = lse[t] - z[t][target[t]].
//   G[t][v] = (dloss + dlse) exp(z - lse) - dloss [v = target];  dx = G w;  dw = G^T x.
//
// All three products are matrix products on the tensor cores (bound by them: 2, 2 + 4
// operations for each row, class and channel; the logits of the backward pass are
// computed once more).  Persistent pairs of blocks walk a list of tiles of 256 x 256, each block
// with half of the rows of both operands in its shared memory (a block by itself would
// write and read half as much again): warp 17 loads blocks of 64 of the depth by TMA into a ring, the
// first block's warp 16 issues the products into one of two accumulators in tensor memory, warps 0-15
// take the other one (a row and 64 columns a thread: with 8 warps and 128 columns each an epilogue's
// latencies show).  8,191 rows of 512 channels, 214,272 classes, forward and backward: 5,744 us in single blocks of
// 128 x 256 (1,250 TFLOP/s), 4,951 in pairs with 8 warps, 4,890 with 16, 4,690 to 4,880, from
// board to board, with the gradients' tiles shared out (1,470 to 1,530 TFLOP/s, 76 to 79 % of a matrix product's rate in a
// burst: forward 864 us, G 1,120, its products 2,050, the rest small).
//
// Forward, a tile's epilogue leaves the maximum and the sum of exponentials of its
// part of each row, and a second kernel joins them.  Backward goes through the
// vocabulary in pieces: G of a piece in the tensors' type (so that the tensor cores can
// take it), then its products, dx summed over the pieces in 32 bits.
//
// What G is rounded to: its factors are divided by the largest |dloss + dlse| or |dloss| of the call (and times 2^14 in
// float16, whose exponents end at 2^-24), which the results are multiplied with.  So the usual
// mean over rows gives factors of exactly 1, a target's gradient near -1 loses little, and
// float16 holds probabilities down to 2^-28 whole in rows of the largest weight.  A row of a weight 2^-n of it has them
// whole down to 2^(n - 28) only, and from there on to within 2^-39 of the largest weight: both products take the same G, and the one over
// rows needs one scale for all of them.

#include "pv_attn.cuh"
#include "pv_tc.cuh"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace {

using namespace pvs;

constexpr int kThreads = 576;
constexpr int kEpilogues = 16;  // warps; then one for the products, one for the loads
constexpr int kOwn = 64;        // columns of an epilogue's thread
constexpr int kM = 256, kN = 256, kK = 64;  // rows, columns and depth of a tile's products
constexpr int kHalf = 128;                  // of the rows, and of the columns' operand, in each block of a pair
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum Mode { kStats, kProbs, kGrads };

template <int kMode>
struct Smem {
  static constexpr int kStages = kMode == kStats ? 6 : 5;
  alignas(1024) unsigned char a[kStages][kHalf * kK * 2];
  alignas(1024) unsigned char b[kStages][kHalf * kK * 2];
  alignas(1024) unsigned char out[kMode == kStats ? 1 : kEpilogues][32 * 128];  // a warp's 32 rows of 64 probabilities, or of dw
  float2 sums[2][4][kMode == kStats ? kHalf : 1];  // the rows' sums of 64 columns each
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  uint32_t tmem;
  int given_up;
};

struct LossArgs {
  int tiles, T, V, D;
  // Logits of classes v0 ..: tiles of all rows, a block of classes after another (the
  // rows are the smaller matrix, and stay in the L2 cache).
  int v0, row_blocks;
  float2* part;        // kStats: [class tiles, T] maximum (times log2 e) and sum of 256 classes
  const float4* rows;  // kProbs: factors of the probability and the target, lse (times log2 e), target's bits
  long long piece;     // classes of a piece, a multiple of 256
  // Gradients: dx_tiles tiles of dx (row block, block of channels, part of the depth), then those of dw, `extra` of
  // them for each pair of blocks that has a tile of dx more than others.
  int dx_tiles, d_tiles, parts, extra, first;
  float* acc;          // [parts, T, D]
  const float* mult;
};

// What one tile multiplies: kind 0 x w^T, 1 dx = G w, 2 dw = G^T x.
struct Tile {
  int kind, m0, n0, n, k0, blocks, part;
};

template <int kMode>
__device__ __forceinline__ Tile tile_of(const LossArgs& a, int i) {
  if constexpr (kMode != kGrads) {
    const int v = i / a.row_blocks;
    return {0, (i - v * a.row_blocks) * kM, v * kN, kN, 0, (a.D + kK - 1) / kK, 0};
  } else {
    const int classes = static_cast<int>(min(static_cast<long long>(a.V - a.v0), a.piece));
    Tile t;
    if (i < a.dx_tiles) {
      t.kind = 1;
      t.part = i % a.parts;
      i /= a.parts;
      const int all = (classes + kK - 1) / kK, each = (all + a.parts - 1) / a.parts;
      t.k0 = min(t.part * each, all);
      t.blocks = min(each, all - t.k0);
    } else {
      t.kind = 2;
      t.part = 0;
      i -= a.dx_tiles;
      t.k0 = 0;
      t.blocks = (a.T + kK - 1) / kK;
    }
    const int m = i / a.d_tiles;
    t.m0 = m * kM;
    t.n0 = (i - m * a.d_tiles) * kN;
    t.n = a.D - t.n0 > 128 ? kN : 128;  // (blocks of 64 columns in each block of the pair)
    return t;
  }
}

// The n-th tile of a pair of blocks, -1 past its last.
template <int kMode>
__device__ __forceinline__ int nth_tile(const LossArgs& a, int pair, int pairs, int n) {
  if constexpr (kMode != kGrads) {
    const int i = pair + n * pairs;
    return i < a.tiles ? i : -1;
  } else {
    const int each = a.dx_tiles / pairs, more = a.dx_tiles - each * pairs;
    const bool has = pair < more;
    const int m = n - each - (has ? 1 : 0);
    if (m < 0) return pair + n * pairs;
    if (has && m >= a.extra) return -1;
    const int i = a.dx_tiles + (has ? m * more + pair : a.extra * more + m * (pairs - more) + pair - more);
    return i < a.tiles ? i : -1;
  }
}

// Maximum (times log2 e) and sum of exponentials of two parts of a row.  (A maximum ignores what
// is no number; the sums do not.)
__device__ __forceinline__ float2 joined(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  const float x = a.x == m ? 1.0f : exp2_fast(a.x - m), y = b.x == m ? 1.0f : exp2_fast(b.x - m);
  return make_float2(m, a.y * x + b.y * y);
}

template <typename T, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    pv_loss_kernel(const __grid_constant__ LossArgs a, const __grid_constant__ CUtensorMap m0, const __grid_constant__ CUtensorMap m1,
                   const __grid_constant__ CUtensorMap m2, const __grid_constant__ CUtensorMap m3,
                   const __grid_constant__ CUtensorMap m4) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) unsigned char raw[];
  using S = Smem<kMode>;
  constexpr int kStages = S::kStages;
  S& sm = *reinterpret_cast<S*>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    sm.given_up = 0;
    for (int i = 0; i < kStages; ++i) bar_init(&sm.full[i], 1), bar_init(&sm.empty[i], 1);
    for (int i = 0; i < 2; ++i) bar_init(&sm.acc_full[i], 1), bar_init(&sm.acc_empty[i], 2 * kEpilogues);
    fence_bar_init();
  }
  if (warp == kEpilogues) tmem_alloc_pair<512>(&sm.tmem);
  tc_before();
  __syncthreads();
  cluster_sync();
  tc_after();
  const int rank = static_cast<int>(cluster_rank()), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const uint32_t tm = sm.tmem;
  volatile int* given_up = &sm.given_up;
  // (Logits backward need nothing of the kernel ahead, which allows this one when its own wait is over; their
  // epilogues need its factors, and the place that G is written to.)
  if constexpr (kMode != kProbs) wait_prior_grid();

  if (warp == kEpilogues + 1) {
    // ---- loads: this block's halves, counted by the first block's barrier
    if (lane == 0) {
      int slot = 0, parity = 1;
      unsigned int sent = 0;
      bool ok = true;
      for (int n = 0, i; ok && (i = nth_tile<kMode>(a, pair, pairs, n)) >= 0; ++n) {
        const Tile t = tile_of<kMode>(a, i);
        const int row = t.m0 + rank * kHalf, col = t.n0 + rank * (t.n / 2), cols = t.n / 128;
        for (int k = t.k0; k < t.k0 + t.blocks; ++k) {
          if (!(ok = bar_wait(&sm.empty[slot], parity, given_up))) break;
          unsigned char *pa = sm.a[slot], *pb = sm.b[slot];
          const uint32_t bar = in_first(&sm.full[slot]);
          if (rank == 0) bar_expect(&sm.full[slot], 2 * (kHalf + t.n / 2) * kK * 2);
          if (kMode != kGrads) {
            tma_load4_pair(pa, &m0, k * kK, 0, 0, row, bar);
            tma_load4_pair(pb, &m1, k * kK, 0, 0, a.v0 + col, bar);
          } else if (t.kind == 1) {
            tma_load4_pair(pa, &m0, k * kK, 0, 0, row, bar);
            for (int c = 0; c < cols; ++c) tma_load4_pair(pb + c * 8192, &m1, col + 64 * c, 0, 0, a.v0 + k * kK, bar);
          } else {
            for (int c = 0; c < 2; ++c) tma_load4_pair(pa + c * 8192, &m2, row + 64 * c, 0, 0, k * kK, bar);
            for (int c = 0; c < cols; ++c) tma_load4_pair(pb + c * 8192, &m3, col + 64 * c, 0, 0, k * kK, bar);
          }
          ++sent;
          if (++slot == kStages) slot = 0, parity ^= 1;
        }
      }
      // (The first block's barriers tell when both blocks' loads have landed, but not of loads that it has not come to
      // itself, if it has given up; those of the second block have landed, too, when the products are done with them.)
      bars_drain(rank == 0 ? sm.full : sm.empty, kStages, sent);
    }
    __syncwarp();
  } else if (warp == kEpilogues) {
    // ---- products, by the first block
    if (rank == 0 && elect_one()) {
      int slot = 0, parity = 0;
      bool ok = true;
      for (int n = 0, i; ok && (i = nth_tile<kMode>(a, pair, pairs, n)) >= 0; ++n) {
        const Tile t = tile_of<kMode>(a, i);
        const bool a_mn = t.kind == 2, b_mn = t.kind != 0;
        const uint32_t word = mma_word(kBf16, kM, 0, a_mn, b_mn) | (static_cast<uint32_t>(t.n >> 3) << 17);
        const uint32_t oa = operand(smem_addr(sm.a[0]), a_mn ? 8192 : 16), ob = operand(smem_addr(sm.b[0]), b_mn ? 8192 : 16);
        const uint32_t sa = a_mn ? 2048 >> 4 : 2, sb = b_mn ? 2048 >> 4 : 2;  // 16 of the depth further
        const uint32_t d = tm + (n & 1) * kN;
        if (!(ok = bar_wait(&sm.acc_empty[n & 1], ((n >> 1) & 1) ^ 1, given_up))) break;
        for (int k = 0; k < t.blocks; ++k) {
          if (!(ok = bar_wait(&sm.full[slot], parity, given_up))) break;
          tc_after();
          const uint32_t xa = oa + slot * (kHalf * kK * 2 >> 4), xb = ob + slot * (kHalf * kK * 2 >> 4);
#pragma unroll
          for (int x = 0; x < kK / 16; ++x) mma_ss_pair(d, xa + x * sa, xb + x * sb, word, k > 0 || x > 0);
          mma_commit_pair(&sm.empty[slot]);
          if (++slot == kStages) slot = 0, parity ^= 1;
        }
        if (ok) mma_commit_pair(&sm.acc_full[n & 1]);
      }
    }
    __syncwarp();
  } else {
    // ---- epilogues: a row and 64 of the columns a thread
    if constexpr (kMode == kProbs) wait_prior_grid();
    const int quarter = warp >> 2, row = rank * kHalf + (warp & 3) * 32 + lane;
    const uint32_t acc_empty[2] = {in_first(&sm.acc_empty[0]), in_first(&sm.acc_empty[1])};
    // A warp whose wait has run out gives nothing back, and all that it writes from there on is NaN: the products stop
    // at the accumulator that it keeps, and no other warp, of either block, finds another tile's in the place of its own.
    bool ok = true;
    auto release = [&](int buf) {
      __syncwarp();
      if (ok && lane == 0) bar_arrive_at(acc_empty[buf]);
    };
    const uint32_t own = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16) + quarter * kOwn;
    for (int n = 0, i; (i = nth_tile<kMode>(a, pair, pairs, n)) >= 0; ++n) {
      const Tile t = tile_of<kMode>(a, i);
      const int buf = n & 1;
      float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (kMode == kProbs && t.m0 + row < a.T) r = a.rows[t.m0 + row];
      ok = ok && warp_wait(&sm.acc_full[buf], (n >> 1) & 1, given_up);
      tc_after();
      const int c0 = t.n0 + quarter * kOwn;
      if constexpr (kMode != kGrads) {
        float v[kOwn];
        tmem_read64(own + buf * kN, v);
        tc_before();
        release(buf);
        const int at = t.m0 + row, left = a.V - a.v0 - c0;  // classes from here on
        if constexpr (kMode == kStats) {
          if (left < kOwn) {
#pragma unroll
            for (int c = 0; c < kOwn; ++c)
              if (c >= left) v[c] = -INFINITY;
          }
          float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int c = 4; c < kOwn - 4; c += 8)
#pragma unroll
            for (int j = 0; j < 4; ++j) top[j] = max3(top[j], v[c + j], v[c + 4 + j]);
#pragma unroll
          for (int j = 0; j < 4; ++j) top[j] = fmaxf(top[j], v[kOwn - 4 + j]);
          const float most = fmaxf(max3(top[0], top[1], top[2]), top[3]) * kLog2e;
          const float off = most == -INFINITY ? 0.0f : -most;
          float sum[4] = {};
#pragma unroll
          for (int c = 0; c < kOwn; c += 4) {
            float e[4];
#pragma unroll
            for (int j = 0; j < 4; j += 2) fma2(e[j], e[j + 1], v[c + j], v[c + j + 1], kLog2e, kLog2e, off, off);
#pragma unroll
            for (int j = 0; j < 4; j += 2)
              add2(sum[j], sum[j + 1], sum[j], sum[j + 1], exp2_fast(e[j]), exp2_fast(e[j + 1]));
          }
          const float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
          // The four warps of these rows join theirs (the next tile's go to the other place).
          const int r = row - rank * kHalf;
          sm.sums[n & 1][quarter][r] = ok ? make_float2(most, s) : make_float2(NAN, NAN);
          asm volatile("bar.sync %0, 128;" ::"r"(1 + (warp & 3)) : "memory");
          if (quarter == (n & 3) && at < a.T) {
            float2 all = sm.sums[n & 1][0][r];
#pragma unroll
            for (int q = 1; q < 4; ++q) all = joined(all, sm.sums[n & 1][q][r]);
            a.part[static_cast<long long>((a.v0 + t.n0) / kN) * a.T + at] = all;
          }
        } else {
          // Through shared memory and out by TMA: rows by themselves would be written in pieces of 16
          // bytes (a piece of 9,728 classes: 103 us for what takes 38 to multiply, 60 like this).
          const int target = __float_as_int(r.w) - a.v0 - c0;
          if (r.x == 0.0f && r.y == 0.0f) {  // no gradient, whatever the logits are (an infinity times 0 is no number)
            r.z = 0.0f;
#pragma unroll
            for (int c = 0; c < kOwn; ++c) v[c] = 0.0f;
          }
          if (!ok) r.x = 1.0f, r.z = NAN;  // (and with it every exponential)
          if (lane == 0) tma_stores_read();
          __syncwarp();
#pragma unroll
          for (int c = 0; c < kOwn; c += 8) {
            float e[8];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              fma2(e[j], e[j + 1], v[c + j], v[c + j + 1], kLog2e, kLog2e, -r.z, -r.z);
              mul2(e[j], e[j + 1], exp2_fast(e[j]), exp2_fast(e[j + 1]), r.x, r.x);
            }
            if ((target & ~7) == c) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (target == c + j) e[j] -= r.y;
            }
            if (left < kOwn) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (c + j >= left) e[j] = 0.0f;
            }
            Pack<T>::store(sm.out[warp] + lane * 128 + (((c >> 3) ^ (lane & 7)) << 4), e);
          }
          fence_to_async();
          __syncwarp();
          if (lane == 0) {
            // (Rows past the last are left out by the map.)
            tma_store4(&m2, sm.out[warp], c0, 0, 0, at);
            tma_store_group();
          }
        }
      } else {
        const int at = t.m0 + row;
        if (t.kind == 2) {
          // By TMA, as the probabilities are: rows by themselves would be written in pieces of 16 bytes
          // (40 rows, 214,272 classes of 512, backward: 233 us with rows stored by their threads, 163 like this).
          if (quarter * kOwn < t.n) {
            const float by = ok ? *a.mult : NAN;
            float v[kOwn];
            tmem_read64(own + buf * kN, v);
            tc_before();
            release(buf);
            if (lane == 0) tma_stores_read();
            __syncwarp();
#pragma unroll
            for (int c = 0; c < kOwn; c += 8) {
#pragma unroll
              for (int x = 0; x < 8; x += 2) mul2(v[c + x], v[c + x + 1], v[c + x], v[c + x + 1], by, by);
              Pack<T>::store(sm.out[warp] + lane * 128 + (((c >> 3) ^ (lane & 7)) << 4), v + c);
            }
            fence_to_async();
            __syncwarp();
            // (Classes past the last and channels past the last are left out by the map.)
            if (lane == 0 && c0 < a.D) {
              tma_store4(&m4, sm.out[warp], c0, 0, 0, a.v0 + at - lane);
              tma_store_group();
            }
          } else {
            tc_before();
            release(buf);
          }
          continue;
        }
#pragma unroll 1
        for (int c = 0; c < kOwn && quarter * kOwn + c < t.n; c += 32) {
          float v[32];
          tmem_read32(own + buf * kN + c, v);
          if (t.blocks == 0 || !ok) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = ok ? 0.0f : NAN;
          }
          if (at < a.T) {
            float* out = a.acc + (static_cast<long long>(t.part) * a.T + at) * a.D + c0 + c;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              if (c0 + c + j >= a.D) continue;
              float4 s = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
              if (!a.first) {
                const float4 o = *reinterpret_cast<const float4*>(out + j);
                s = make_float4(s.x + o.x, s.y + o.y, s.z + o.z, s.w + o.w);
              }
              *reinterpret_cast<float4*>(out + j) = s;
            }
          }
          __syncwarp();
        }
        tc_before();
        release(buf);
      }
    }
  }
  if (kMode != kStats && warp < kEpilogues && lane == 0) tma_stores_done();
  // Neither block goes while the other one may read, write or signal its shared memory.
  tc_before();
  __syncthreads();
  cluster_sync();
  tc_after();
  allow_next_grid();
  if (warp == kEpilogues) tmem_free_pair<512>(tm);
}

// ------------------------------------------------------------ few rows

// Up to 32 rows: the classes are the products' rows, and the rows of x, all of their depth in shared
// memory, their columns.  The weights are read once, which bounds it.  A thread keeps the
// maximum and the sum of its classes for every row of x, and the block joins them at its end.
constexpr int kFew = 32, kFewThreads = 192, kFewStages = 9;
constexpr int kFewBlocks = 16;  // blocks of 64 of the depth that there is room for

struct SmemFew {
  alignas(1024) unsigned char w[kFewStages][128 * kK * 2];
  alignas(1024) unsigned char x[kFewBlocks][kFew * kK * 2];
  uint64_t full[kFewStages], empty[kFewStages], x_full, acc_full[2], acc_empty[2];
  uint32_t tmem;
  int given_up;
};

template <typename T>
__global__ void __launch_bounds__(kFewThreads, 1)
    pv_loss_few_kernel(const __grid_constant__ LossArgs a, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) unsigned char raw[];
  SmemFew& sm = *reinterpret_cast<SmemFew*>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    sm.given_up = 0;
    for (int i = 0; i < kFewStages; ++i) bar_init(&sm.full[i], 1), bar_init(&sm.empty[i], 1);
    bar_init(&sm.x_full, 1);
    for (int i = 0; i < 2; ++i) bar_init(&sm.acc_full[i], 1), bar_init(&sm.acc_empty[i], 4);
    fence_bar_init();
  }
  if (warp == 4) tmem_alloc<64>(&sm.tmem);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = sm.tmem;
  volatile int* given_up = &sm.given_up;
  wait_prior_grid();
  const int blocks = (a.D + kK - 1) / kK;
  if (warp == 5) {
    if (lane == 0) {
      bar_expect(&sm.x_full, blocks * kFew * kK * 2);
      for (int k = 0; k < blocks; ++k) tma_load4(sm.x[k], &mx, k * kK, 0, 0, 0, &sm.x_full);
      int slot = 0, parity = 1;
      unsigned int sent = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < a.tiles; i += gridDim.x)
        for (int k = 0; k < blocks; ++k) {
          if (!(ok = bar_wait(&sm.empty[slot], parity, given_up))) break;
          bar_expect(&sm.full[slot], 128 * kK * 2);
          tma_load4(sm.w[slot], &mw, k * kK, 0, 0, i * 128, &sm.full[slot]);
          ++sent;
          if (++slot == kFewStages) slot = 0, parity ^= 1;
        }
      bars_drain(&sm.x_full, 1, 1);
      bars_drain(sm.full, kFewStages, sent);
    }
    __syncwarp();
  } else if (warp == 4) {
    if (elect_one()) {
      const uint32_t word = mma_word(kBf16, 128, kFew, false, false);
      const uint32_t ow = operand(smem_addr(sm.w[0]), 16), ox = operand(smem_addr(sm.x[0]), 16);
      int slot = 0, parity = 0, n = 0;
      bool ok = bar_wait(&sm.x_full, 0, given_up);
      for (int i = blockIdx.x; ok && i < a.tiles; i += gridDim.x, ++n) {
        if (!(ok = bar_wait(&sm.acc_empty[n & 1], ((n >> 1) & 1) ^ 1, given_up))) break;
        for (int k = 0; k < blocks; ++k) {
          if (!(ok = bar_wait(&sm.full[slot], parity, given_up))) break;
          tc_after();
          const uint32_t w = ow + slot * (128 * kK * 2 >> 4), x = ox + k * (kFew * kK * 2 >> 4);
#pragma unroll
          for (int j = 0; j < kK / 16; ++j) mma_ss(tm + (n & 1) * kFew, w + 2 * j, x + 2 * j, word, k > 0 || j > 0);
          mma_commit(&sm.empty[slot]);
          if (++slot == kFewStages) slot = 0, parity ^= 1;
        }
        if (ok) mma_commit(&sm.acc_full[n & 1]);
      }
    }
    __syncwarp();
  } else {
    float top[kFew], sum[kFew];
#pragma unroll
    for (int j = 0; j < kFew; ++j) top[j] = -INFINITY, sum[j] = 0.0f;
    bool ok = true;
    int n = 0;
    for (int i = blockIdx.x; i < a.tiles; i += gridDim.x, ++n) {
      ok = ok && warp_wait(&sm.acc_full[n & 1], (n >> 1) & 1, given_up);
      tc_after();
      float z[kFew];
      tmem_read32(tm + (static_cast<uint32_t>(warp * 32) << 16) + (n & 1) * kFew, z);
      tc_before();
      if (ok) warp_arrive(&sm.acc_empty[n & 1]);
      if (i * 128 + warp * 32 + lane < a.V) {
#pragma unroll
        for (int j = 0; j < kFew; ++j) {
          // (An infinite maximum makes no number of the sum, as in the other kernel.)
          const float u = z[j] * kLog2e, m = fmaxf(top[j], u), off = m == -INFINITY ? 0.0f : m;
          sum[j] = fmaf(sum[j], exp2_fast(top[j] - off), exp2_fast(u - off));
          top[j] = m;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kFew; ++j) {
      if (j >= a.T) break;
      float m = top[j];
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      float s = sum[j] * (top[j] == m ? 1.0f : exp2_fast(top[j] - m));
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      if (lane == 0) a.part[static_cast<long long>(blockIdx.x * 4 + warp) * a.T + j] = ok ? make_float2(m, s) : make_float2(NAN, NAN);
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  allow_next_grid();
  if (warp == 4) tmem_free<64>(tm);
}

// ------------------------------------------------------------ what is around the products

// Joins the parts of eight rows' softmax sums, in order, and takes the target's logit from its
// two rows.  Four slices of the parts in a warp; 32 warps where the parts are many, 8 where they are
// few (4,071 rows of 33 parts: 8.9 us with 32 warps, 5.3 with 8).
template <typename T, int kWarps>
__global__ void __launch_bounds__(32 * kWarps)
    pv_loss_join_kernel(const float2* part, int parts, int rows, int V, int D, const char* x, long long x_row, const char* w,
                        long long w_row, const long long* target, float* loss, float* lse) {
  constexpr int kEach = kWarps / 8;  // warps for a row's target
  __shared__ float2 sums[kWarps][8];
  __shared__ float dots[kWarps];
  wait_prior_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane & 7, row = blockIdx.x * 8 + r;
  const int own = blockIdx.x * 8 + warp / kEach;
  const long long t = own < rows ? target[own] : -1;
  float2 own_sum = make_float2(-INFINITY, 0.0f);
  if (row < rows) {
#pragma unroll 4
    for (int p = warp * 4 + (lane >> 3); p < parts; p += 4 * kWarps) own_sum = joined(own_sum, part[static_cast<long long>(p) * rows + row]);
  }
  float dot = 0.0f;
  if (t >= 0 && t < V) {
    const char *px = x + own * x_row, *pw = w + t * w_row;
#pragma unroll 2
    for (int c = ((warp % kEach) * 32 + lane) * 8; c < D; c += 256 * kEach) {
      float u[8], v[8];
      Pack<T>::load(px + 2 * c, u);
      Pack<T>::load(pw + 2 * c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) dot = fmaf(u[j], v[j], dot);
    }
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    const float2 other = make_float2(__shfl_xor_sync(0xFFFFFFFFu, own_sum.x, o), __shfl_xor_sync(0xFFFFFFFFu, own_sum.y, o));
    // (The same order on both sides, so that all lanes hold the same bits.)
    own_sum = lane & o ? joined(other, own_sum) : joined(own_sum, other);
  }
  if (lane < 8) sums[warp][lane] = own_sum;
#pragma unroll
  for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
  if (lane == 0) dots[warp] = dot;
  __syncthreads();
  if (threadIdx.x < 8 && row < rows) {
    float2 all = sums[0][r];
    for (int i = 1; i < kWarps; ++i) all = joined(all, sums[i][r]);
    const float l = all.y == 0.0f ? -INFINITY : (all.x + log2f(all.y)) * kLn2;
    const long long v = target[row];
    float z = dots[kEach * r];
    for (int i = 1; i < kEach; ++i) z += dots[kEach * r + i];
    lse[row] = l;
    // A target that no class has is a mistake, and shows; a negative one says that there is none.
    loss[row] = v < 0 ? 0.0f : v < V ? l - z : NAN;
  }
  allow_next_grid();
}

// What the rows' gradients are scaled by: the factors over the largest finite one (and
// times `up`); *mult, what that takes out of the results.  One block.
__global__ void __launch_bounds__(1024)
    pv_loss_rows_kernel(const float* dloss, const float* dlse, const float* lse, const long long* target, int rows, int V, float up,
                        float4* out, float* mult) {
  __shared__ float most[32];
  wait_prior_grid();
  allow_next_grid();
  auto of = [&](int t, float& c1, float& c2) {
    const long long v = target[t];
    const float l = dloss[t], s = dlse ? dlse[t] : 0.0f;
    c2 = v < 0 ? 0.0f : v < V ? l : NAN;
    c1 = c2 + s;
    return static_cast<int>(v < 0 || v >= V ? -1 : v);
  };
  float top = 0.0f;
#pragma unroll 8
  for (int t = threadIdx.x; t < rows; t += 1024) {
    float c1, c2;
    of(t, c1, c2);
    top = fmaxf(top, isfinite(c1) ? fabsf(c1) : 0.0f);
    top = fmaxf(top, isfinite(c2) ? fabsf(c2) : 0.0f);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = top;
  __syncthreads();
  for (int i = 0; i < 32; ++i) top = fmaxf(top, most[i]);
  if (threadIdx.x == 0) *mult = top / up;
#pragma unroll 8
  for (int t = threadIdx.x; t < rows; t += 1024) {
    float c1, c2;
    const int v = of(t, c1, c2);
    // (With nothing but zeros, or nothing finite, the factors are what they are.)
    out[t] = make_float4(top > 0.0f ? c1 / top * up : c1, top > 0.0f ? c2 / top * up : c2, lse[t] * kLog2e, __int_as_float(v));
  }
}

// dx: the parts joined in order, scaled and rounded; four elements a thread.
template <typename T>
__global__ void __launch_bounds__(256)
    pv_loss_dx_kernel(const float* acc, int parts, int rows, int D, const float* mult, char* dx, long long dx_row) {
  wait_prior_grid();
  const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 4, all = static_cast<long long>(rows) * D;
  if (i < all) {
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int p = 0; p < parts; ++p) {
      const float4 v = *reinterpret_cast<const float4*>(acc + p * all + i);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const float by = *mult;
    const long long t = i / D;
    *reinterpret_cast<uint2*>(dx + t * dx_row + (i - t * D) * 2) = make_uint2(Pack<T>::two(s.x * by, s.y * by), Pack<T>::two(s.z * by, s.w * by));
  }
  allow_next_grid();
}

// ------------------------------------------------------------ host side

// How the tiles of the gradients go to the pairs of blocks: those of dx in turn, cut into parts of their depth, the
// classes; those of dw so that pairs with a tile of dx less have more of them.  `cost`: blocks of the
// depth that the longest pair goes through, a tile's change counted as one, no tile as less than five (its epilogue,
// 40 rows, 214,272 classes of 512, backward: 219 us without), and the last epilogue as eight.
// (All tiles in turn: 8,191 rows, 214,272 classes of 512, forward and backward 4,855 us, 4,760 like this;
// 2,048 rows, 32,000 classes of 512, backward 157 and 147; 4,071 rows, 8,193 classes of 128, forward and backward 75 and 73.)
struct Plan {
  int parts, extra;
  int64_t cost;
};

Plan shared_out(int64_t x_tiles, int64_t x_blocks, int64_t parts, int64_t w_tiles, int64_t w_blocks, int most_pairs) {
  const int64_t x = x_tiles * parts, pairs = std::min<int64_t>(most_pairs, x + w_tiles), more = x % pairs, less = pairs - more;
  const int64_t each = std::max<int64_t>((x_blocks + parts - 1) / parts + 1, 5), w = std::max<int64_t>(w_blocks + 1, 5), mine = x / pairs * each;
  Plan best{static_cast<int>(parts), 0, INT64_MAX};
  const int64_t even = more ? std::max<int64_t>(0, (w_tiles * w - less * each) / (pairs * w)) : 0;
  for (int64_t extra = even; extra <= even + (more ? 1 : 0); ++extra) {
    const int64_t rest = std::max<int64_t>(0, w_tiles - extra * more);
    const int64_t cost = std::max(more ? mine + each + extra * w : 0, mine + (rest + less - 1) / less * w) + 8;
    if (cost < best.cost) best.extra = static_cast<int>(extra), best.cost = cost;
  }
  return best;
}

Plan plan_of(int64_t x_tiles, int64_t x_blocks, int64_t w_tiles, int64_t w_blocks, int most_pairs) {
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(2 * most_pairs / x_tiles, x_blocks / 4));
  Plan best{1, 0, INT64_MAX};
  for (int64_t parts = 1; parts <= most; ++parts) {
    const Plan p = shared_out(x_tiles, x_blocks, parts, w_tiles, w_blocks, most_pairs);
    if (p.cost < best.cost) best = p;
  }
  return best;
}

// Classes of a piece: as many pieces as these bytes of G ask for, or one or two more if equal ones are done
// sooner.  (Each piece costs some 15 us, 40 blocks of the depth, more than its products: 8,191 rows of 512 channels, 214,272
// classes, backward 4,883 us with pieces of 80 MB that stay in the L2 cache, 3,766 with 160, 3,442 with 640, 3,400 with
// 1,280; with 64 channels 3,510, 2,671, 2,110 and 2,044.)
constexpr int64_t kPieceBytes = int64_t(768) << 20;

int64_t piece_of(int64_t T, int64_t V, int64_t D, int pairs) {
  const int64_t all = (V + kN - 1) / kN, most = std::max<int64_t>(1, kPieceBytes / (2 * T * kN)), d_tiles = (D + kN - 1) / kN;
  const int64_t fewest = (all + most - 1) / most, x_tiles = (T + kM - 1) / kM * d_tiles;
  int64_t best = all, least = INT64_MAX;
  for (int64_t n = fewest; fewest > 1 && n <= fewest + 2; ++n) {
    const int64_t c = (all + n - 1) / n, cost = n * (plan_of(x_tiles, c * (kN / kK), c * d_tiles, (T + kK - 1) / kK, pairs).cost + 40);
    if (cost < least) least = cost, best = c;
  }
  return best * kN;
}

int check_matrix(const void* p, int64_t stride, int64_t rows, int64_t D, int dev) {
  if (rows == 0) return PV_OK;
  if (!p || !aligned(p, 16) || stride % 8 || device_of(p) != dev) return PV_ERR_INVALID;
  return stride >= D || (rows == 1 && stride >= 0) ? PV_OK : PV_ERR_INVALID;
}

int check_params(const pv_loss_params* p, int* dev) {
  if (!p || (p->dtype != PV_BF16 && p->dtype != PV_F16)) return PV_ERR_INVALID;
  if (p->rows < 0 || p->classes < 1 || p->channels < 8 || p->channels % 8) return PV_ERR_INVALID;
  if (p->rows > PV_LOSS_MAX_ROWS || p->classes > PV_LOSS_MAX_CLASSES || p->channels > PV_LOSS_MAX_CHANNELS) return PV_ERR_TOO_LARGE;
  if (!p->weight || (*dev = device_of(p->weight)) < 0) return PV_ERR_INVALID;
  int st = check_matrix(p->x, p->x_stride, p->rows, p->channels, *dev);
  if (st == PV_OK) st = check_matrix(p->weight, p->weight_stride, p->classes, p->channels, *dev);
  if (st != PV_OK || p->rows == 0) return st;
  return p->targets && aligned(p->targets, 8) && device_of(p->targets) == *dev ? PV_OK : PV_ERR_INVALID;
}

bool floats_on(const float* p, int dev) { return p && aligned(p, 4) && device_of(p) == dev; }

int map_of(CUtensorMap* m, const void* p, int64_t stride, int dtype, int64_t rows, int64_t cols, int box) {
  View v{static_cast<char*>(const_cast<void*>(p)), stride * 2, 0};
  return make_map(m, v, dtype, static_cast<int>(cols), 1, 1, rows, box);
}

template <typename T, int kMode>
int launch_products(const LossArgs& a, const CUtensorMap (&m)[5], int sms, cudaStream_t s) {
  auto kernel = pv_loss_kernel<T, kMode>;
  const int smem = static_cast<int>(sizeof(Smem<kMode>)) + 1024;
  const int st = allow_smem(kernel, smem);
  if (st != PV_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * std::min(a.tiles, sms / 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, a, m[0], m[1], m[2], m[3], m[4]) != cudaSuccess) {
    cudaGetLastError();
    return PV_ERR_CUDA;
  }
  return PV_OK;
}

template <typename T>
int forward(const pv_loss_params* p, float* loss, float* lse, int dev, pv_stream_t stream) {
  const int sms = sm_count(dev);
  if (sms < 1) return PV_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  LossArgs a{};
  a.T = static_cast<int>(p->rows), a.V = static_cast<int>(p->classes), a.D = static_cast<int>(p->channels);
  // Few rows (whose depth fits beside the ring) are read by every block, and the classes walked through; more go
  // in tiles of both (8 rows, 214,272 classes of 512: 67 us in tiles, 40 like this, 82 % of the memory's rate).
  const bool few = a.T <= kFew && a.D <= kFewBlocks * kK;
  int parts;
  Scratch scratch;
  int st;
  CUtensorMap m[5];
  if (few) {
    a.tiles = (a.V + 127) / 128;
    const int blocks = std::min(a.tiles, sms);
    parts = 4 * blocks;
    if ((st = scratch.open(dev, stream, kPlain, sizeof(float2) * parts * a.T)) != PV_OK) return st;
    a.part = static_cast<float2*>(scratch.body());
    if ((st = map_of(&m[0], p->x, p->x_stride, p->dtype, a.T, a.D, kFew)) != PV_OK ||
        (st = map_of(&m[1], p->weight, p->weight_stride, p->dtype, a.V, a.D, 128)) != PV_OK)
      return st;
    const int smem = static_cast<int>(sizeof(SmemFew)) + 1024;
    if ((st = allow_smem(pv_loss_few_kernel<T>, smem)) != PV_OK ||
        (st = launch_pdl(pv_loss_few_kernel<T>, dim3(blocks), kFewThreads, smem, s, a, m[0], m[1])) != PV_OK)
      return st;
  } else {
    a.row_blocks = (a.T + kM - 1) / kM;
    const int64_t class_tiles = (a.V + kN - 1) / kN, tiles = class_tiles * a.row_blocks;
    if (tiles >= (int64_t(1) << 31) - sms) return PV_ERR_TOO_LARGE;
    a.tiles = static_cast<int>(tiles);
    parts = static_cast<int>(class_tiles);
    if ((st = scratch.open(dev, stream, kPlain, sizeof(float2) * class_tiles * a.T)) != PV_OK) return st;
    a.part = static_cast<float2*>(scratch.body());
    if ((st = map_of(&m[0], p->x, p->x_stride, p->dtype, a.T, a.D, kHalf)) != PV_OK ||
        (st = map_of(&m[1], p->weight, p->weight_stride, p->dtype, a.V, a.D, kHalf)) != PV_OK)
      return st;
    m[2] = m[3] = m[4] = m[0];
    if ((st = launch_products<T, kStats>(a, m, sms, s)) != PV_OK) return st;
  }
  const bool many = parts > 128;
  return launch_pdl(many ? pv_loss_join_kernel<T, 32> : pv_loss_join_kernel<T, 8>, dim3((a.T + 7) / 8), many ? 1024 : 256, 0, s,
                    static_cast<const float2*>(a.part), parts, a.T, a.V, a.D, static_cast<const char*>(p->x),
                    static_cast<long long>(p->x_stride * 2), static_cast<const char*>(p->weight),
                    static_cast<long long>(p->weight_stride * 2), reinterpret_cast<const long long*>(p->targets), loss, lse);
}

template <typename T>
int backward(const pv_loss_params* p, const float* dloss, const float* dlse, const float* lse, void* dx, int64_t dx_stride, void* dw,
             int64_t dw_stride, int dev, pv_stream_t stream) {
  const int sms = sm_count(dev);
  if (sms < 1) return PV_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  LossArgs a{};
  a.T = static_cast<int>(p->rows), a.V = static_cast<int>(p->classes), a.D = static_cast<int>(p->channels);
  a.row_blocks = (a.T + kM - 1) / kM;
  a.d_tiles = (a.D + kN - 1) / kN;
  a.piece = piece_of(a.T, a.V, a.D, sms / 2);
  const int64_t dx_tiles = static_cast<int64_t>(a.row_blocks) * a.d_tiles;
  const int64_t w_blocks = (a.T + kK - 1) / kK;
  a.parts = plan_of(dx_tiles, a.piece / kK, a.piece / kM * a.d_tiles, w_blocks, sms / 2).parts;
  const int64_t logit_tiles = static_cast<int64_t>(a.row_blocks) * (a.piece / kN), dw_tiles = a.piece / kM * a.d_tiles;
  if (std::max(logit_tiles, dx_tiles * a.parts + dw_tiles) >= (int64_t(1) << 31) - sms) return PV_ERR_TOO_LARGE;
  const size_t rows = round_up(sizeof(float4) * a.T, 1024), g = round_up(2 * static_cast<size_t>(a.T) * a.piece, 1024);
  Scratch scratch;
  int st = scratch.open(dev, stream, kPlain, 1024 + rows + g + sizeof(float) * a.parts * static_cast<size_t>(a.T) * a.D);
  if (st != PV_OK) return st;
  char* at = static_cast<char*>(scratch.body());
  float* mult = reinterpret_cast<float*>(at);
  a.mult = mult;
  float4* rows_out = reinterpret_cast<float4*>(at + 1024);
  a.rows = rows_out;
  void* const g_at = at + 1024 + rows;
  a.acc = reinterpret_cast<float*>(at + 1024 + rows + g);
  const float up = p->dtype == PV_F16 ? 16384.0f : 1.0f;
  if ((st = launch_pdl(pv_loss_rows_kernel, dim3(1), 1024, 0, s, dloss, dlse, lse, reinterpret_cast<const long long*>(p->targets), a.T,
                       a.V, up, rows_out, mult)) != PV_OK)
    return st;
  CUtensorMap z[5], m[5];
  if ((st = map_of(&z[0], p->x, p->x_stride, p->dtype, a.T, a.D, kHalf)) != PV_OK ||
      (st = map_of(&z[1], p->weight, p->weight_stride, p->dtype, a.V, a.D, kHalf)) != PV_OK ||
      (st = map_of(&m[0], g_at, a.piece, p->dtype, a.T, a.piece, kHalf)) != PV_OK ||
      (st = map_of(&m[1], p->weight, p->weight_stride, p->dtype, a.V, a.D, kK)) != PV_OK ||
      (st = map_of(&m[2], g_at, a.piece, p->dtype, a.T, a.piece, kK)) != PV_OK ||
      (st = map_of(&m[3], p->x, p->x_stride, p->dtype, a.T, a.D, kK)) != PV_OK ||
      (st = map_of(&m[4], dw, dw_stride, p->dtype, a.V, a.D, 32)) != PV_OK)
    return st;
  if ((st = map_of(&z[2], g_at, a.piece, p->dtype, a.T, a.piece, 32)) != PV_OK) return st;
  z[3] = z[4] = z[0];
  a.first = 1;
  for (int64_t v0 = 0; v0 < a.V; v0 += a.piece) {
    a.v0 = static_cast<int>(v0);
    const int64_t classes = std::min<int64_t>(a.piece, a.V - v0);
    a.tiles = static_cast<int>(a.row_blocks * ((classes + kN - 1) / kN));
    if ((st = launch_products<T, kProbs>(a, z, sms, s)) != PV_OK) return st;
    a.dx_tiles = static_cast<int>(dx_tiles * a.parts);
    const int64_t w_tiles = (classes + kM - 1) / kM * a.d_tiles;
    a.tiles = a.dx_tiles + static_cast<int>(w_tiles);
    a.extra = shared_out(dx_tiles, (classes + kK - 1) / kK, a.parts, w_tiles, w_blocks, sms / 2).extra;
    if ((st = launch_products<T, kGrads>(a, m, sms, s)) != PV_OK) return st;
    a.first = 0;
  }
  const int64_t packs = static_cast<int64_t>(a.T) * a.D / 4;
  return launch_pdl(pv_loss_dx_kernel<T>, dim3(static_cast<unsigned>((packs + 255) / 256)), 256, 0, s, static_cast<const float*>(a.acc),
                    a.parts, a.T, a.D, static_cast<const float*>(mult), static_cast<char*>(dx), static_cast<long long>(dx_stride * 2));
}

}  // namespace

extern "C" int pv_cross_entropy(const pv_loss_params* params, float* loss, float* lse, pv_stream_t stream) try {
  int dev = 0, st = check_params(params, &dev);
  if (st != PV_OK || params->rows == 0) return st;
  if (!floats_on(loss, dev) || !floats_on(lse, dev)) return PV_ERR_INVALID;
  DeviceScope scope(dev);
  if (!scope.ok()) return PV_ERR_CUDA;
  return params->dtype == PV_BF16 ? forward<__nv_bfloat16>(params, loss, lse, dev, stream)
                                  : forward<__half>(params, loss, lse, dev, stream);
} catch (...) {
  return caught();
}

extern "C" int pv_cross_entropy_backward(const pv_loss_params* params, const float* dloss, const float* dlse, const float* lse,
                                         void* dx, int64_t dx_stride, void* dweight, int64_t dweight_stride,
                                         pv_stream_t stream) try {
  int dev = 0, st = check_params(params, &dev);
  if (st != PV_OK) return st;
  if ((st = check_matrix(dx, dx_stride, params->rows, params->channels, dev)) != PV_OK ||
      (st = check_matrix(dweight, dweight_stride, params->classes, params->channels, dev)) != PV_OK)
    return st;
  if (params->rows && (!floats_on(dloss, dev) || !floats_on(lse, dev) || (dlse && !floats_on(dlse, dev)))) return PV_ERR_INVALID;
  DeviceScope scope(dev);
  if (!scope.ok()) return PV_ERR_CUDA;
  if (params->rows == 0) {
    const int64_t pitch = 2 * std::max(dweight_stride, params->channels);  // (a single class may come with any stride)
    if (cudaMemset2DAsync(dweight, pitch, 0, params->channels * 2, params->classes, reinterpret_cast<cudaStream_t>(stream)) ==
        cudaSuccess)
      return PV_OK;
    cudaGetLastError();
    return PV_ERR_CUDA;
  }
  return params->dtype == PV_BF16
             ? backward<__nv_bfloat16>(params, dloss, dlse, lse, dx, dx_stride, dweight, dweight_stride, dev, stream)
             : backward<__half>(params, dloss, dlse, lse, dx, dx_stride, dweight, dweight_stride, dev, stream);
} catch (...) {
  return caught();
}
