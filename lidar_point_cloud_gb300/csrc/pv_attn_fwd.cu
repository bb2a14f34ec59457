// Attention inside frames, forward, on the tensor cores.
//
// A block takes two tiles of 128 query rows and walks the frame's keys in
// tiles of 128.  Warps 0-3 and 4-7 own a query tile each, one row a thread: they
// read the scores from tensor memory, keep the row's running maximum and sum,
// and write the probabilities back over the scores as the next product's
// operand.  Warp 8 issues the products, warp 9 the TMA loads of keys and values
// into a ring of shared-memory slots, warp 10 puts key positions there, warp 11
// clears what a frame's last tile holds of the next frame.  While
// one tile's scores go through the exponential, the other tile's products run.
//
// Rows are (query, head) pairs of the heads that share a key head (the largest
// power of two of them), so that one query of many heads fills a tile as far as
// it can, and its keys are read once for all of them.
//
// With few rows the keys are split over blocks: each leaves its unnormalised
// output, maximum and sum, and a second kernel joins them in order.
//
// The running maximum moves only when a row's scores rise by more than 2^8 over
// it: sums and outputs then stay below 2^8 times what they would be, well
// inside 32 bits (and probabilities inside float16), and the output in tensor
// memory is rescaled a few times per row instead of at every tile.
// Probabilities are rounded to the storage type for the second product, as the
// tensor cores take it; their sum is taken before rounding, in 32 bits.

#include "pv_attn.cuh"
#include "pv_tc.cuh"

#include <type_traits>

namespace pvs {

namespace {

constexpr int kThreads = 384;
// Registers of a thread: 168 at launch (384 x 168 = 64,512 of a multiprocessor's
// 65,536); the softmax warpgroups take what the other one gives back: 256 x 208 +
// 128 x 80 = 63,488.
constexpr int kRegsSoftmax = 208, kRegsOther = 80;
constexpr int kRows = 128;      // rows of a query tile, keys of a key tile
constexpr int kPosSlots = 4;
constexpr float kLazy = 8.0f;   // log2 of how far scores may rise over the kept maximum
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int kBlocks>  // 64-element blocks of a head: 1 or 2
struct Smem {
  static constexpr int kTile = kRows * 128 * kBlocks;  // bytes of 128 rows of a head
  static constexpr int kSlots = kBlocks == 1 ? 8 : 4;
  alignas(1024) unsigned char q[2][kTile];
  alignas(1024) unsigned char kv[kSlots][kTile];
  float pos[kPosSlots][3][kRows];
  uint64_t q_full, dirty, clean, kv_full[kSlots], kv_empty[kSlots], s_full[2], p_full[2], o_full[2], pos_full[kPosSlots], pos_empty[kPosSlots];
  uint32_t tmem;
  int given_up;
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return Pack<T>::two(a, b);
}

template <typename T, int kBlocks>
__global__ void __launch_bounds__(kThreads, 1)
    pv_attn_fwd_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using S = Smem<kBlocks>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) unsigned char raw[];
  S& sm = *reinterpret_cast<S*>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- which rows, which keys
  const int tile = blockIdx.x / a.heads, place = frame_of(a.tile0, a.frames, tile), f = a.order[place];
  const int nq = a.q0[f + 1] - a.q0[f], nk = a.k0[f + 1] - a.k0[f];
  const int pack = 1 << a.pack_log2;
  const int mblocks = (((nq << a.pack_log2) + 2 * kRows - 1) / (2 * kRows));
  const int local = tile - a.tile0[place];
  // Later rows see more keys under a causal mask: they go first.
  const int mb = mblocks - 1 - local % mblocks, split = local / mblocks;
  const int hb = blockIdx.x - tile * a.heads;  // block of `pack` heads
  const int kh = (hb << a.pack_log2) / a.G;
  // Keys that query i sees: all below this.
  auto limit = [&](int i) { return a.causal ? max(min(max(i + nk - nq + 1, a.prefix[f]), nk), 0) : nk; };
  const int js = split * a.chunk;
  int first[2], last_j[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    first[t] = (mb * 2 + t) * (kRows >> a.pack_log2);  // its first query
    const int end = min(first[t] + (kRows >> a.pack_log2), nq);
    const int tiles = first[t] < nq ? (limit(end - 1) + kRows - 1) / kRows : 0;
    last_j[t] = max(min(tiles, js + a.chunk), js);
  }
  const int je = max(last_j[0], last_j[1]);

  // ---- set up
  if (threadIdx.x == 0) {
    sm.given_up = 0;
    bar_init(&sm.q_full, 1);
    bar_init(&sm.dirty, 1);
    bar_init(&sm.clean, 1);
    for (int i = 0; i < S::kSlots; ++i) bar_init(&sm.kv_full[i], 1), bar_init(&sm.kv_empty[i], 1);
    for (int t = 0; t < 2; ++t) bar_init(&sm.s_full[t], 1), bar_init(&sm.p_full[t], kRows / 32), bar_init(&sm.o_full[t], 1);
    for (int i = 0; i < kPosSlots; ++i) bar_init(&sm.pos_full[i], 1), bar_init(&sm.pos_empty[i], 2 * kRows / 32);
    fence_bar_init();
    tma_prefetch(&mq);
    tma_prefetch(&mk);
    tma_prefetch(&mv);
  }
  if (warp == 8) tmem_alloc<512>(&sm.tmem);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = sm.tmem;
  volatile int* given_up = &sm.given_up;
  const int heads_k = a.k.head ? kh : 0, heads_v = a.v.head ? kh : 0;
  wait_prior_grid();

  if (warp >= 8) regs_down<kRegsOther>();
  if (warp == 9) {
    // ---- loads
    if (lane == 0 && je > js) {
      const bool two = last_j[1] > js;
      bar_expect(&sm.q_full, (two ? 2 : 1) * S::kTile);
      for (int t = 0; t < (two ? 2 : 1); ++t)
        for (int b = 0; b < kBlocks; ++b)
          tma_load4(sm.q[t] + b * kRows * 128, &mq, b * 64, 0, a.q.head ? hb : 0, a.q0[f] + first[t], &sm.q_full);
      for (int n = 0; n < 2 * (je - js); ++n) {
        const int slot = n % S::kSlots;
        if (!bar_wait(&sm.kv_empty[slot], ((n / S::kSlots) & 1) ^ 1, given_up)) break;
        bar_expect(&sm.kv_full[slot], S::kTile);
        const CUtensorMap* m = n & 1 ? &mv : &mk;
        for (int b = 0; b < kBlocks; ++b)
          tma_load4(sm.kv[slot] + b * kRows * 128, m, b * 64, 0, n & 1 ? heads_v : heads_k,
                    a.k0[f] + (js + (n >> 1)) * kRows, &sm.kv_full[slot]);
      }
    }
  } else if (warp == 8) {
    // ---- products: one thread, with little to do between them (the tensor cores
    // take few in advance, and its scheduler is shared)
    if (elect_one() && je > js) {
      const uint32_t word_s = mma_word(kBf16, 128, 128, false, false);
      const uint32_t word_o = mma_word(kBf16, 128, 0, false, true) | (static_cast<uint32_t>(a.Dn >> 3) << 17);
      const int ksteps = (a.D + 15) / 16;
      const uint32_t q_op = operand(smem_addr(sm.q[0]), 16), k_op = operand(smem_addr(sm.kv[0]), 16);
      const uint32_t v_op = operand(smem_addr(sm.kv[0]), kRows * 128);
      constexpr uint32_t kStep = S::kTile >> 4;
      auto scores = [&](int t, int slot) {  // S_t = Q_t K^T
        const uint32_t q = q_op + t * kStep, k = k_op + slot * kStep;
#pragma unroll
        for (int x = 0; x < 4 * kBlocks; ++x) {
          const uint32_t off = ((x >> 2) * kRows * 128 + (x & 3) * 32) >> 4;
          if (x < ksteps) mma_ss(tm + t * 128, q + off, k + off, word_s, x > 0);
        }
        mma_commit(&sm.s_full[t]);
      };
      // Keys lie in the even slots of the ring, values in the odd ones.
      int slot = 0, parity = 0;
      bool ok = bar_wait(&sm.q_full, 0, given_up) && bar_wait(&sm.kv_full[0], 0, given_up);
      if (ok) {
        tc_after();
        for (int t = 0; t < 2; ++t)
          if (last_j[t] > js) scores(t, 0);
        mma_commit(&sm.kv_empty[0]);
      }
      for (int j = js; ok && j < je; ++j) {
        const int sv = slot + 1;
        if (!(ok = bar_wait(&sm.kv_full[sv], parity, given_up))) break;
        if ((j + 1) * kRows > nk) {
          bar_arrive(&sm.dirty);
          if (!(ok = bar_wait(&sm.clean, 0, given_up))) break;
        }
        slot += 2;
        if (slot == S::kSlots) slot = 0, parity ^= 1;
        if (j + 1 < je && !(ok = bar_wait(&sm.kv_full[slot], parity, given_up))) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || j >= last_j[t]) continue;
          if (!(ok = bar_wait(&sm.p_full[t], (j - js) & 1, given_up))) continue;
          tc_after();
          const uint32_t v = v_op + sv * kStep;
#pragma unroll
          for (int x = 0; x < kRows / 16; ++x)
            mma_ts(tm + 256 + t * 64 * kBlocks, tm + t * 128 + x * 8, v + x * (2048 >> 4), word_o, j > js || x > 0);
          if (j + 1 < last_j[t])
            scores(t, slot);
          else
            mma_commit(&sm.o_full[t]);
        }
        if (ok) {
          mma_commit(&sm.kv_empty[sv]);
          if (j + 1 < je) mma_commit(&sm.kv_empty[slot]);
        }
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    // ---- rows past the frame's end are another frame's: whatever they hold must
    // not meet the zero probabilities of these places
    if (je > js && je * kRows > nk) {
      const int n = 2 * (je - 1 - js) + 1, have = nk - (je - 1) * kRows;
      if (warp_wait(&sm.dirty, 0, given_up)) {
        uint4* v = reinterpret_cast<uint4*>(sm.kv[n % S::kSlots]);
        for (int b = 0; b < kBlocks; ++b)
          for (int i = have * 8 + lane; i < kRows * 8; i += 32) v[b * kRows * 8 + i] = make_uint4(0, 0, 0, 0);
        fence_to_async();
        warp_arrive(&sm.clean);
      }
    }
  } else if (warp == 10) {
    // ---- key positions, each tile's loaded while the last one's are handed over
    if (a.slopes && je > js) {
      int next[3][4];
      auto load = [&](int j) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = j * kRows + x * 32 + lane;
          const int32_t* p = a.kpos + static_cast<long long>(a.k0[f] + min(key, nk - 1)) * a.kpos_stride;
#pragma unroll
          for (int c = 0; c < 3; ++c)
            if (c < a.axes) next[c][x] = p[c];
        }
      };
      load(js);
      for (int j = js; j < je; ++j) {
        const int n = j - js, slot = n % kPosSlots;
        float now[3][4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int c = 0; c < 3; ++c)
            if (c < a.axes) now[c][x] = static_cast<float>(next[c][x]);
        if (j + 1 < je) load(j + 1);
        if (!warp_wait(&sm.pos_empty[slot], ((n / kPosSlots) & 1) ^ 1, given_up)) break;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int c = 0; c < 3; ++c)
            if (c < a.axes) sm.pos[slot][c][x * 32 + lane] = now[c][x];
        warp_arrive(&sm.pos_full[slot]);
      }
    }
  } else if (warp < 8) {
    // ---- softmax: 32 rows a warp, in fragments: four rows and 32 of their keys a thread
    regs_up<kRegsSoftmax>();
    const int t = warp >> 2, r0 = (warp & 3) * 32, quad = lane & 3;
    const uint32_t mine = tm + (static_cast<uint32_t>(r0) << 16), high = mine + (16u << 16);
    const uint32_t sc = t * 128, oc = 256 + t * 64 * kBlocks;  // columns
    // Row `x` of the thread is r0 + 8 x + lane / 4.
    int lim[4];
    float slope[4], qp[3][4];
    // What a score (the raw product, or tanh of it if capped) is multiplied by to
    // be in units of log2.
    const float mul = (a.cap > 0.0f ? a.cap : a.scale) * kLog2e;
    const float cap_in = a.cap > 0.0f ? 2.0f * a.scale * kLog2e / a.cap : 0.0f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = r0 + 8 * x + (lane >> 2), i = first[t] + (r >> a.pack_log2);
      lim[x] = i < nq ? limit(i) : nk;
      slope[x] = 0.0f;
#pragma unroll
      for (int c = 0; c < 3; ++c) qp[c][x] = 0.0f;
      if (a.slopes && i < nq) {
        slope[x] = -a.slopes[(hb << a.pack_log2) + (r & (pack - 1))] * kLog2e / mul;
#pragma unroll
        for (int c = 0; c < 3; ++c)
          if (c < a.axes) qp[c][x] = -static_cast<float>(a.qpos[static_cast<long long>(a.q0[f] + i) * a.qpos_stride + c]);
      }
    }
    const int clear = first[t] < nq ? limit(first[t]) : nk;  // tiles that end at or below this are seen whole
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, sum[4] = {};
    bool ok = true;
    for (int j = js; j < last_j[t]; ++j) {
      const int n = j - js;
      if (!(ok = warp_wait(&sm.s_full[t], n & 1, given_up))) break;
      tc_after();
      float u[2][64];
      tmem_ld_16x256b_x16(mine + sc, reinterpret_cast<uint32_t*>(u[0]));
      tmem_ld_16x256b_x16(high + sc, reinterpret_cast<uint32_t*>(u[1]));
      tc_wait_ld<64>(reinterpret_cast<uint32_t*>(u[0]));
      tc_wait_ld<64>(reinterpret_cast<uint32_t*>(u[1]));
      if (a.cap > 0.0f) {
#pragma unroll
        for (int x = 0; x < 128; ++x) u[x >> 6][x & 63] = tanh_half(u[x >> 6][x & 63] * cap_in);
      }
      if (a.slopes) {
        if (!(ok = warp_wait(&sm.pos_full[n % kPosSlots], (n / kPosSlots) & 1, given_up))) break;
        const float* pos = &sm.pos[n % kPosSlots][0][2 * quad];
        if (a.axes == 1)
          lower<1, 16>(u, pos, kRows, qp, slope);
        else if (a.axes == 2)
          lower<2, 16>(u, pos, kRows, qp, slope);
        else
          lower<3, 16>(u, pos, kRows, qp, slope);
        warp_arrive(&sm.pos_empty[n % kPosSlots]);
      }
      if ((j + 1) * kRows > clear) {
#pragma unroll
        for (int x = 0; x < 128; ++x) {
          const int row = (x >> 6) * 2 + ((x >> 1) & 1), col = ((x & 63) >> 2) * 8 + (x & 1);
          u[x >> 6][x & 63] = col < lim[row] - j * kRows - 2 * quad ? u[x >> 6][x & 63] : -INFINITY;
        }
      }
      float most[4];
#pragma unroll
      for (int row = 0; row < 4; ++row) {
        const float* x = u[row >> 1] + 2 * (row & 1);
        float m0 = fmaxf(x[0], x[1]), m1 = fmaxf(x[4], x[5]);
#pragma unroll
        for (int k = 2; k < 16; k += 2) {
          m0 = max3(m0, x[4 * k], x[4 * k + 1]);
          m1 = max3(m1, x[4 * k + 4], x[4 * k + 5]);
        }
        most[row] = fmaxf(m0, m1) * mul;
      }
      // -inf + 8 is -inf: any first score is a rise.  Only if some thread's own share of a
      // row rises are the shares of a row joined.
      const bool rise = most[0] > top[0] + kLazy || most[1] > top[1] + kLazy || most[2] > top[2] + kLazy || most[3] > top[3] + kLazy;
      if (__any_sync(0xFFFFFFFFu, rise)) {
        float by[4];
#pragma unroll
        for (int row = 0; row < 4; ++row) {
          most[row] = fmaxf(most[row], __shfl_xor_sync(0xFFFFFFFFu, most[row], 1));
          most[row] = fmaxf(most[row], __shfl_xor_sync(0xFFFFFFFFu, most[row], 2));
          const bool up = most[row] > top[row] + kLazy;
          by[row] = up ? exp2_fast(top[row] - most[row]) : 1.0f;
          if (up) top[row] = most[row];
          sum[row] *= by[row];
        }
        if (j > js)
          for (int x = 0; x < a.Dn; x += 16) {
            uint32_t o[2][8];
            tmem_ld_16x256b_x2(mine + oc + x, o[0]);
            tmem_ld_16x256b_x2(high + oc + x, o[1]);
            tc_wait_ld<8>(o[0]);
            tc_wait_ld<8>(o[1]);
#pragma unroll
            for (int y = 0; y < 16; ++y)
              o[y >> 3][y & 7] = __float_as_uint(__uint_as_float(o[y >> 3][y & 7]) * by[(y >> 3) * 2 + ((y >> 1) & 1)]);
            tmem_st_16x256b_x2(mine + oc + x, o[0]);
            tmem_st_16x256b_x2(high + oc + x, o[1]);
          }
      }
      float base[4];
#pragma unroll
      for (int row = 0; row < 4; ++row) base[row] = top[row] == -INFINITY ? 0.0f : -top[row];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p[32];
        float s[4] = {};
#pragma unroll
        for (int x = 0; x < 64; x += 2) {
          const int row = 2 * h + ((x >> 1) & 1);
          float e0, e1;
          fma2(e0, e1, u[h][x], u[h][x + 1], mul, mul, base[row], base[row]);
          e0 = exp2_fast(e0);
          e1 = exp2_fast(e1);
          add2(s[x & 2], s[(x & 2) + 1], s[x & 2], s[(x & 2) + 1], e0, e1);
          p[x >> 1] = pack2<T>(e0, e1);
        }
        tmem_st_16x128b_x16((h ? high : mine) + sc, p);
        sum[2 * h] += s[0] + s[1];
        sum[2 * h + 1] += s[2] + s[3];
      }
      tc_wait_st();
      tc_before();
      warp_arrive(&sm.p_full[t]);
    }
    // A tile that ends earlier lets go of the other tile's key positions.
    if (a.slopes)
      for (int j = last_j[t]; ok && j < je; ++j) {
        const int n = j - js;
        if ((ok = warp_wait(&sm.pos_full[n % kPosSlots], (n / kPosSlots) & 1, given_up))) warp_arrive(&sm.pos_empty[n % kPosSlots]);
      }
    // ---- output: one row a thread, its statistics fetched from the fragments' threads
    const bool any = last_j[t] > js;
    float row_sum = 0.0f, row_top = 0.0f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      sum[x] += __shfl_xor_sync(0xFFFFFFFFu, sum[x], 1);
      sum[x] += __shfl_xor_sync(0xFFFFFFFFu, sum[x], 2);
      const float s = __shfl_sync(0xFFFFFFFFu, sum[x], (lane & 7) * 4), m = __shfl_sync(0xFFFFFFFFu, top[x], (lane & 7) * 4);
      if (lane >> 3 == x) row_sum = s, row_top = m;
    }
    const int r = r0 + lane, i = first[t] + (r >> a.pack_log2), h = (hb << a.pack_log2) + (r & (pack - 1));
    const bool live = i < nq;
    const long long qrow = a.q0[f] + i;
    if (any && ok) ok = warp_wait(&sm.o_full[t], 0, given_up);
    tc_after();
    const bool parts = a.part_o != nullptr;
    float by = parts ? 1.0f : row_sum > 0.0f ? 1.0f / row_sum : 0.0f;
    if (!ok || *given_up) by = __int_as_float(0x7FFFFFFF);  // a wait ran out: nothing here is an answer
    char* out = a.o.data + qrow * a.o.row + h * a.o.head;
    float* part = parts ? a.part_o + ((static_cast<long long>(split) * a.queries + qrow) * a.H + h) * a.D : nullptr;
    for (int x = 0; x < a.Dn; x += 16) {
      uint32_t o[16];
      float v[16];
      if (any) {
        tmem_ld16(mine + oc + x, o);
        tc_wait_ld<16>(o);
      }
#pragma unroll
      for (int y = 0; y < 16; ++y) v[y] = any ? __uint_as_float(o[y]) * by : 0.0f * by;
#pragma unroll
      for (int y = 0; y < 16; y += 8) {
        if (!live || x + y >= a.D) continue;
        if (parts) {
          Pack<float>::store(part + x + y, v + y);
          Pack<float>::store(part + x + y + 4, v + y + 4);
        } else {
          Pack<T>::store(out + (x + y) * 2, v + y);
        }
      }
      __syncwarp();
    }
    if (live) {
      const long long at = static_cast<long long>(h) * a.queries + qrow;
      if (parts)
        a.part_ml[(static_cast<long long>(split) * a.queries + qrow) * a.H + h] = make_float2(row_top, row_sum);
      else if (a.lse)
        a.lse[at] = row_sum > 0.0f ? (row_top + log2f(row_sum)) * kLn2 : -INFINITY;
    }
    tc_before();
  }
  __syncthreads();
  if (warp == 8) {
    if (*given_up) {
      // Loads and products still in flight end in this block's shared and tensor
      // memory: two milliseconds are a thousand times what they take.
      const unsigned long long until = now_ns() + 2000000ull;
      while (now_ns() < until) {
      }
      __syncwarp();
    }
    tc_after();
    tmem_free<512>(tm);
  }
  allow_next_grid();
}

// Joins the parts of a row: weights 2^(top - highest top), in order.
template <typename T>
__global__ void __launch_bounds__(128) pv_attn_join_kernel(const __grid_constant__ AttnArgs a) {
  wait_prior_grid();
  const long long w = (static_cast<long long>(blockIdx.x) * 128 + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w < static_cast<long long>(a.queries) * a.H) {
    const int row = static_cast<int>(w / a.H), h = static_cast<int>(w % a.H);
    const int f = frame_of(a.q0, a.frames, row);
    const int nk = a.k0[f + 1] - a.k0[f];
    const int splits = max(1, ((nk + kRows - 1) / kRows + a.chunk - 1) / a.chunk);
    float top = -INFINITY;
    for (int s = 0; s < splits; ++s) top = fmaxf(top, a.part_ml[(static_cast<long long>(s) * a.queries + row) * a.H + h].x);
    float sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < splits; ++s) {
      const long long at = (static_cast<long long>(s) * a.queries + row) * a.H + h;
      const float2 ml = a.part_ml[at];
      const float by = ml.x == -INFINITY ? 0.0f : exp2_fast(ml.x - top);
      sum = fmaf(ml.y, by, sum);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (lane * 4 + x < a.D) v[x] = fmaf(a.part_o[at * a.D + lane * 4 + x], by, v[x]);
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    T* out = reinterpret_cast<T*>(a.o.data + row * a.o.row + h * a.o.head);
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (lane * 4 + x < a.D) out[lane * 4 + x] = Pack<T>::one(v[x] * inv);
    if (a.lse && lane == 0)
      a.lse[static_cast<long long>(h) * a.queries + row] = sum > 0.0f ? (top + log2f(sum)) * kLn2 : -INFINITY;
  }
  allow_next_grid();
}

template <typename T, int kBlocks>
int launch_fwd(const AttnArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, dim3 grid, cudaStream_t s) {
  auto kernel = pv_attn_fwd_kernel<T, kBlocks>;
  const int smem = static_cast<int>(sizeof(Smem<kBlocks>)) + 1024;
  static bool ready[64];  // set once per device; a second set does no harm
  int dev = 0;
  cudaGetDevice(&dev);
  if (!ready[dev & 63]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
      cudaGetLastError();
      return PV_ERR_CUDA;
    }
    ready[dev & 63] = true;
  }
  return launch_pdl(kernel, grid, kThreads, smem, s, a, q, k, v);
}

}  // namespace

int attn_forward(AttnArgs& a, int dtype, const AttnMaps& m, dim3 grid, cudaStream_t s) {
  const bool wide = a.D > 64;
  int st;
  if (dtype == PV_BF16)
    st = wide ? launch_fwd<__nv_bfloat16, 2>(a, m.q, m.k, m.v, grid, s) : launch_fwd<__nv_bfloat16, 1>(a, m.q, m.k, m.v, grid, s);
  else
    st = wide ? launch_fwd<__half, 2>(a, m.q, m.k, m.v, grid, s) : launch_fwd<__half, 1>(a, m.q, m.k, m.v, grid, s);
  if (st != PV_OK || !a.part_o) return st;
  const long long warps = static_cast<long long>(a.queries) * a.H;
  const dim3 g(static_cast<unsigned int>((warps + 3) / 4));
  return dtype == PV_BF16 ? launch_pdl(pv_attn_join_kernel<__nv_bfloat16>, g, 128, 0, s, a)
                          : launch_pdl(pv_attn_join_kernel<__half>, g, 128, 0, s, a);
}

}  // namespace pvs
