// Attention inside frames, forward, on the tensor cores.
//
// A block takes two tiles of 128 query rows and walks the frame's keys in
// tiles of 128.  Warps 0-3 and 4-7 own a query tile each: they read the scores from
// tensor memory (a row a thread, or, with distances, fragments of four rows), keep
// the rows' running maxima and sums, and write the probabilities back over the
// scores as the next product's operand.  Warp 8 issues the products, warp 9 the TMA loads of keys and values
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
// The running maximum moves only when a row's scores rise by more than 2^32 over
// it (2^15 for float16, whose probabilities have to stay below 2^16): sums and
// outputs then stay that far below what they would be, well inside 32 bits, and the
// output in tensor memory is rescaled once or twice per row instead of at every
// tile.  With distances, whose nearest keys come anywhere in a frame, that
// matters: 8 ragged frames took 667 us with 2^8, 619 us with 2^32.
// Probabilities are rounded to the storage type for the second product, as the
// tensor cores take it; their sum is taken before rounding, in 32 bits.
//
// Measured: 24,571 causal tokens, 8 heads over 2 of 128, bf16, 743 us by itself (1,665
// TFLOP/s), 795 to 820 us in a row, at the power limit (1,510 to 1,560): bound by the tensor
// cores.  8 ragged frames of up to 6,000, 8 heads of 64: 414 us,
// with distances 594 us: bound by the arithmetic between the products (two warps a
// scheduler, 53 % of issue slots; four softmax warpgroups have too few registers, and
// loading the scores in two or four pieces hides nothing: 601 and 660 us).  A cap is two more
// special-function operations a score: 4,071 tokens, 4 heads of 32, f16, 51 us.

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
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int kBlocks>  // 64-element blocks of a head: 1 or 2
struct Smem {
  static constexpr int kTile = kRows * 128 * kBlocks;  // bytes of 128 rows of a head
  static constexpr int kSlots = kBlocks == 1 ? 8 : 4;
  // Tensor memory holds two outputs of 64 or 128 columns, and as many score
  // tiles of 128 columns as then fit: three are a ring that both query tiles take
  // from in turn (8 ragged distance-biased frames, 64-element heads: 672 -> 619 us), two
  // are one each.
  static constexpr int kBufs = kBlocks == 1 ? 3 : 2;
  static constexpr bool kRing = kBufs == 3;
  static constexpr int kOut = kBufs * 128;
  alignas(1024) unsigned char q[2][kTile];
  alignas(1024) unsigned char kv[kSlots][kTile];
  float pos[kPosSlots][3][kRows];
  uint64_t q_full, dirty, clean, kv_full[kSlots], kv_empty[kSlots], s_full[kBufs], p_full[kBufs], pv_done[2][2], o_full[2], pos_full[kPosSlots], pos_empty[kPosSlots];
  uint32_t tmem;
  int given_up;
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return Pack<T>::two(a, b);
}

// The logarithm of a row's sum (-inf if it sees nothing, no number if its sum is none).
__device__ __forceinline__ float log_sum(float top, float sum) { return sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2; }

template <typename T, int kBlocks, int kCap, bool kSlopes>
__global__ void __launch_bounds__(kThreads, 1)
    pv_attn_fwd_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using S = Smem<kBlocks>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr float kLazy = kBf16 ? 32.0f : 15.0f;  // log2 of how far scores may rise over the kept maximum
  extern __shared__ __align__(1024) unsigned char raw[];
  S& sm = *reinterpret_cast<S*>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- which rows, which keys
  const int tile = blockIdx.x / a.heads, place = frame_of(a.tile0, a.frames, tile), f = a.order[place];
  const int nq = a.q0[f + 1] - a.q0[f], nk = a.k0[f + 1] - a.k0[f];
  const int pack = 1 << a.pack_log2;
  const int per_block = 2 * kRows >> a.pack_log2;  // queries of a block
  const int mblocks = (nq + per_block - 1) / per_block;
  const int local = tile - a.tile0[place];
  // Later rows see more keys under a causal mask: they go first.
  const int mb = mblocks - 1 - local % mblocks, split = local / mblocks;
  const int hb = blockIdx.x - tile * a.heads;  // block of `pack` heads
  const int kh = (hb << a.pack_log2) / a.G;
  // Keys that query i sees: all below this.
  auto limit = [&](int i) { return a.causal ? max(min(max(i - nq + nk + 1, a.prefix[f]), nk), 0) : nk; };
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
    for (int b = 0; b < S::kBufs; ++b) bar_init(&sm.s_full[b], 1), bar_init(&sm.p_full[b], kRows / 32);
    for (int t = 0; t < 2; ++t) bar_init(&sm.pv_done[t][0], 1), bar_init(&sm.pv_done[t][1], 1), bar_init(&sm.o_full[t], 1);
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
      if constexpr (S::kRing) {
        const int count[2] = {last_j[0] - js, last_j[1] - js}, tiles = je - js;
        // The two query tiles' steps in turn (a tile that ends earlier drops out).
        struct Turn {
          int t, n;
        };
        auto next = [&](Turn& x) {
          do {
            x.n += x.t;
            x.t ^= 1;
          } while (x.n >= count[x.t] && x.n < tiles);
        };
        // A key tile's operands are used by the first and then the second query tile.
        auto opens = [&](Turn x) { return x.t == 0 || x.n >= count[0]; };
        auto closes = [&](Turn x) { return x.t == 1 || x.n >= count[1]; };
        Turn ahead{count[0] > 0 ? 0 : 1, 0}, now = ahead;
        int buf = 0, buf_at = 0, parity = 0;  // the score buffers of `ahead` and of `now`, and its parity
        bool ok = bar_wait(&sm.q_full, 0, given_up);
        // S = Q K^T of the turn `ahead`: what it needs, and the products.
        uint32_t s_q = 0, s_k = 0;
        int s_slot = 0;
        auto prepare = [&]() {
          const int i = 2 * ahead.n;
          s_slot = i % S::kSlots;
          s_q = q_op + ahead.t * kStep;
          s_k = k_op + s_slot * kStep;
          return !opens(ahead) || bar_wait(&sm.kv_full[s_slot], (i / S::kSlots) & 1, given_up);
        };
        auto scores = [&]() {
#pragma unroll
          for (int x = 0; x < 4 * kBlocks; ++x) {
            const uint32_t off = ((x >> 2) * kRows * 128 + (x & 3) * 32) >> 4;
            if (x < ksteps) mma_ss(tm + buf * 128, s_q + off, s_k + off, word_s, x > 0);
          }
          mma_commit(&sm.s_full[buf]);
          if (closes(ahead)) mma_commit(&sm.kv_empty[s_slot]);
          if (++buf == S::kBufs) buf = 0;
          next(ahead);
        };
        const int total = count[0] + count[1];
        for (int i = 0; ok && i < min(total, S::kBufs); ++i) {
          if (!(ok = prepare())) break;
          tc_after();
          scores();
        }
        for (int i = 0; ok && i < total; ++i) {
          const int iv = 2 * now.n + 1, slot = iv % S::kSlots;
          if (opens(now)) {
            if (!(ok = bar_wait(&sm.kv_full[slot], (iv / S::kSlots) & 1, given_up))) break;
            if ((js + now.n + 1) * kRows > nk) {
              bar_arrive(&sm.dirty);
              if (!(ok = bar_wait(&sm.clean, 0, given_up))) break;
            }
          }
          // Nothing is left to be done between this turn's product and the next scores.
          const bool more = i + S::kBufs < total;
          if (more && !(ok = prepare())) break;
          const uint32_t v = v_op + slot * kStep, out = tm + S::kOut + now.t * 64 * kBlocks, p = tm + buf_at * 128;
          uint64_t* const done = now.n + 1 == count[now.t] ? &sm.o_full[now.t] : &sm.pv_done[now.t][now.n & 1];
          const bool add = now.n > 0, close = closes(now);
          if (!(ok = bar_wait(&sm.p_full[buf_at], parity, given_up))) break;
          tc_after();
#pragma unroll
          for (int x = 0; x < kRows / 16; ++x) mma_ts(out, p + x * 8, v + x * (2048 >> 4), word_o, add || x > 0);
          mma_commit(done);
          if (close) mma_commit(&sm.kv_empty[slot]);
          if (more) scores();
          if (++buf_at == S::kBufs) buf_at = 0, parity ^= 1;
          next(now);
        }
      } else {
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
              mma_ts(tm + S::kOut + t * 64 * kBlocks, tm + t * 128 + x * 8, v + x * (2048 >> 4), word_o, j > js || x > 0);
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
    if (kSlopes && je > js) {
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
    // ---- softmax: 32 rows a warp
    regs_up<kRegsSoftmax>();
    const int t = warp >> 2, r0 = (warp & 3) * 32;
    const uint32_t mine = tm + (static_cast<uint32_t>(r0) << 16);
    const uint32_t oc = S::kOut + t * 64 * kBlocks;  // the output's columns
    const int other_count = last_j[1 - t] - js;
    const int r = r0 + lane, i = first[t] + (r >> a.pack_log2), h = (hb << a.pack_log2) + (r & (pack - 1));
    const bool live = i < nq;
    const long long qrow = a.q0[f] + i;
    const int clear = first[t] < nq ? limit(first[t]) : nk;  // tiles that end at or below this are seen whole
    // What a score (the raw product, or tanh of it if capped) is multiplied by to
    // be in units of log2.
    const float mul = (kCap ? a.cap : a.scale) * kLog2e;
    const float cap_in = kCap ? 2.0f * a.scale * kLog2e / a.cap : 0.0f;
    bool ok = true;
    // The score buffer of step n, and the phase of its barriers: with a ring, steps of
    // both tiles before this one count.
    auto buffer = [&](int n, uint32_t* phase) {
      const int turn = S::kRing ? n + min(n + t, other_count) : 2 * n + t;
      *phase = (turn / S::kBufs) & 1;
      return turn % S::kBufs;
    };
    float row_sum = 0.0f, row_top = 0.0f;  // of the thread's own row
    if constexpr (kSlopes) {
      // In fragments, four rows and 32 of their keys a thread: a key's position is loaded
      // once for four rows, by lanes that load different keys.  (With a row a thread
      // every lane loads the same one, at the same cost to the shared memory as 512
      // different bytes: 166 us for two frames of 4,096, 157 us in fragments.)
      const int quad = lane & 3;
      const uint32_t high = mine + (16u << 16);
      // Row `x` of the thread is r0 + 8 x + lane / 4.
      int lim[4];
      float slope[4], qp[3][4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int r = r0 + 8 * x + (lane >> 2), i = first[t] + (r >> a.pack_log2);
        lim[x] = i < nq ? limit(i) : nk;
        slope[x] = 0.0f;
#pragma unroll
        for (int c = 0; c < 3; ++c) qp[c][x] = 0.0f;
        if (i < nq) {
          slope[x] = -a.slopes[(hb << a.pack_log2) + (r & (pack - 1))] * kLog2e / mul;
#pragma unroll
          for (int c = 0; c < 3; ++c)
            if (c < a.axes) qp[c][x] = -static_cast<float>(a.qpos[static_cast<long long>(a.q0[f] + i) * a.qpos_stride + c]);
        }
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, sum[4] = {};
      for (int j = js; j < last_j[t]; ++j) {
        const int n = j - js;
        uint32_t phase;
        const int buf = buffer(n, &phase);
        const uint32_t sc = buf * 128;
        if (!(ok = warp_wait(&sm.s_full[buf], phase, given_up))) break;
        tc_after();
        float u[2][64];
        tmem_ld_16x256b_x16(mine + sc, reinterpret_cast<uint32_t*>(u[0]));
        tmem_ld_16x256b_x16(high + sc, reinterpret_cast<uint32_t*>(u[1]));
        tc_wait_ld<64>(reinterpret_cast<uint32_t*>(u[0]));
        tc_wait_ld<64>(reinterpret_cast<uint32_t*>(u[1]));
        if (kCap) {
#pragma unroll
          for (int x = 0; x < 128; ++x) u[x >> 6][x & 63] = capped<kCap>(u[x >> 6][x & 63] * cap_in);
        }
        {
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
        // -inf + kLazy is -inf: any first score is a rise.  Only if some thread's own share of a
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
          if (n > 0) {
            // With a ring the last step's product may still be adding to the output.  (These
            // scores were issued after the product of two or three steps ago: with a barrier each
            // for even and odd steps, the phase awaited is never two away.)
            if (S::kRing && !(ok = warp_wait(&sm.pv_done[t][(n - 1) & 1], ((n - 1) >> 1) & 1, given_up))) break;
            tc_after();
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
        warp_arrive(&sm.p_full[buf]);
      }
      // A tile that ends earlier lets go of the other tile's key positions.
      for (int j = last_j[t]; ok && j < je; ++j) {
        const int n = j - js;
        if ((ok = warp_wait(&sm.pos_full[n % kPosSlots], (n / kPosSlots) & 1, given_up))) warp_arrive(&sm.pos_empty[n % kPosSlots]);
      }
      // Each row's statistics to the thread that writes it.
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        sum[x] += __shfl_xor_sync(0xFFFFFFFFu, sum[x], 1);
        sum[x] += __shfl_xor_sync(0xFFFFFFFFu, sum[x], 2);
        const float s = __shfl_sync(0xFFFFFFFFu, sum[x], (lane & 7) * 4), m = __shfl_sync(0xFFFFFFFFu, top[x], (lane & 7) * 4);
        if (lane >> 3 == x) row_sum = s, row_top = m;
      }
    } else {
      // A row a thread: no maximum or sum is joined across threads (two sequences of 4,096,
      // 128-element heads: 115 us in fragments, 108 us so).
      const int lim = live ? limit(i) : nk;
      float top = -INFINITY, sum = 0.0f;
      for (int j = js; j < last_j[t]; ++j) {
        const int n = j - js;
        uint32_t phase;
        const int buf = buffer(n, &phase);
        const uint32_t sc = mine + buf * 128;
        if (!(ok = warp_wait(&sm.s_full[buf], phase, given_up))) break;
        tc_after();
        float u[kRows];
        uint32_t* ur = reinterpret_cast<uint32_t*>(u);
#pragma unroll
        for (int x = 0; x < kRows; x += 32) tmem_ld32(sc + x, ur + x);
        tc_wait_ld<kRows>(ur);
        if (kCap) {
#pragma unroll
          for (int x = 0; x < kRows; ++x) u[x] = capped<kCap>(u[x] * cap_in);
        }
        if ((j + 1) * kRows > clear) {
          const int seen = lim - j * kRows;
#pragma unroll
          for (int x = 0; x < kRows; ++x) u[x] = x < seen ? u[x] : -INFINITY;
        }
        float m[4] = {u[0], u[1], u[2], u[3]};
#pragma unroll
        for (int x = 4; x < kRows; x += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (x + 2 * y + 1 < kRows) m[y] = max3(m[y], u[x + 2 * y], u[x + 2 * y + 1]);
        const float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * mul;
        const bool rise = most > top + kLazy;  // -inf + kLazy is -inf: any first score is a rise
        if (j == js) {
          if (rise) top = most;
        } else if (__any_sync(0xFFFFFFFFu, rise)) {
          // (As above.)
          if (S::kRing && !(ok = warp_wait(&sm.pv_done[t][(n - 1) & 1], ((n - 1) >> 1) & 1, given_up))) break;
          tc_after();
          const float by = rise ? exp2_fast(top - most) : 1.0f;
          if (rise) top = most;
          sum *= by;
          for (int x = 0; x < a.Dn; x += 16) {
            uint32_t o[16];
            tmem_ld16(mine + oc + x, o);
            tc_wait_ld<16>(o);
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * by);
            tmem_st16(mine + oc + x, o);
          }
        }
        const float base = top == -INFINITY ? 0.0f : -top;
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int y = 0; y < kRows; y += 64) {
          uint32_t p[32];
#pragma unroll
          for (int x = 0; x < 64; x += 2) {
            float e0, e1;
            fma2(e0, e1, u[y + x], u[y + x + 1], mul, mul, base, base);
            e0 = exp2_fast(e0);
            e1 = exp2_fast(e1);
            add2(s0, s1, s0, s1, e0, e1);
            p[x >> 1] = pack2<T>(e0, e1);
          }
          tmem_st32(sc + (y >> 1), p);
        }
        sum += s0 + s1;
        tc_wait_st();
        tc_before();
        warp_arrive(&sm.p_full[buf]);
      }
      row_sum = sum;
      row_top = top;
    }
    // ---- output: one row a thread
    const bool any = last_j[t] > js;
    if (any && ok) ok = warp_wait(&sm.o_full[t], 0, given_up);
    tc_after();
    const bool parts = a.part_o != nullptr;
    float by = parts ? 1.0f : row_sum == 0.0f ? 0.0f : 1.0f / row_sum;
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
        a.lse[at] = log_sum(row_top, row_sum);
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

// Joins the parts of a row: weights 2^(top - highest top), in order.  kLanes lanes a row,
// four elements a lane; a part's maximum and sum are read by one of them, the outputs
// eight parts at a time.
template <typename T, int kLanes>
__global__ void __launch_bounds__(128) pv_attn_join_kernel(const __grid_constant__ AttnArgs a) {
  wait_prior_grid();
  const long long step = static_cast<long long>(a.queries) * a.H;
  const long long first = (static_cast<long long>(blockIdx.x) * 128 + threadIdx.x) / kLanes;
  const int lane = threadIdx.x % kLanes;
  const bool any = first < step, on = any && lane * 4 < a.D;
  const int row = any ? static_cast<int>(first / a.H) : 0, h = any ? static_cast<int>(first % a.H) : 0;
  const int f = frame_of(a.q0, a.frames, row);
  const int tiles = (a.k0[f + 1] - a.k0[f] + kRows - 1) / kRows;
  const int parts = any ? max(1, (tiles + a.chunk - 1) / a.chunk) : 0;
  const float* at = a.part_o + first * a.D + lane * 4;
  float top = -INFINITY, sum = 0.0f, v[4] = {};
  for (int x = 0; __any_sync(0xFFFFFFFFu, x < parts); x += kLanes) {
    const float2 ml = x + lane < parts ? a.part_ml[first + (x + lane) * step] : make_float2(-INFINITY, 0.0f);
    float m = fmaxf(top, ml.x);
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float keep = top == -INFINITY ? 0.0f : exp2_fast(top - m), by = ml.x == -INFINITY ? 0.0f : exp2_fast(ml.x - m);
    float s = ml.y * by;
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    top = m;
    sum = fmaf(sum, keep, s);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] *= keep;
#pragma unroll 1
    for (int p0 = 0; p0 < kLanes && __any_sync(0xFFFFFFFFu, x + p0 < parts); p0 += 8) {
      float4 o[8];
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (on && x + p0 + p < parts) o[p] = *reinterpret_cast<const float4*>(at + (x + p0 + p) * step * a.D);
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const float b = __shfl_sync(0xFFFFFFFFu, by, p0 + p, kLanes);
        if (on && x + p0 + p < parts) {
          v[0] = fmaf(o[p].x, b, v[0]);
          v[1] = fmaf(o[p].y, b, v[1]);
          v[2] = fmaf(o[p].z, b, v[2]);
          v[3] = fmaf(o[p].w, b, v[3]);
        }
      }
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (on)
    *reinterpret_cast<uint2*>(a.o.data + row * a.o.row + h * a.o.head + lane * 8) =
        make_uint2(pack2<T>(v[0] * inv, v[1] * inv), pack2<T>(v[2] * inv, v[3] * inv));
  if (any && a.lse && lane == 0)
    a.lse[static_cast<long long>(h) * a.queries + row] = log_sum(top, sum);
  allow_next_grid();
}

template <int kLanes>
int launch_join(const AttnArgs& a, cudaStream_t s) {
  const long long threads = static_cast<long long>(a.queries) * a.H * kLanes;
  return launch_pdl(pv_attn_join_kernel<Storage, kLanes>, dim3(static_cast<unsigned>((threads + 127) / 128)), 128, 0, s, a);
}

template <int kBlocks, int kCap, bool kSlopes>
int launch_fwd(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s) {
  auto kernel = pv_attn_fwd_kernel<Storage, kBlocks, kCap, kSlopes>;
  const int smem = static_cast<int>(sizeof(Smem<kBlocks>)) + 1024;
  const int st = allow_smem(kernel, smem);
  return st == PV_OK ? launch_pdl(kernel, grid, kThreads, smem, s, a, m.q, m.k, m.v) : st;
}

template <int kBlocks>
int with_scores(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s) {
  if (a.cap > kSmallCap) return a.slopes ? launch_fwd<kBlocks, kAny, true>(a, m, grid, s) : launch_fwd<kBlocks, kAny, false>(a, m, grid, s);
  if (a.cap > 0.0f) return a.slopes ? launch_fwd<kBlocks, kSmall, true>(a, m, grid, s) : launch_fwd<kBlocks, kSmall, false>(a, m, grid, s);
  return a.slopes ? launch_fwd<kBlocks, kNoCap, true>(a, m, grid, s) : launch_fwd<kBlocks, kNoCap, false>(a, m, grid, s);
}

}  // namespace

int PV_ATTN_NAME(attn_forward)(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s) {
  const int st = a.D > 64 ? with_scores<2>(a, m, grid, s) : with_scores<1>(a, m, grid, s);
  if (st != PV_OK || !a.part_o) return st;
  return a.D > 64 ? launch_join<32>(a, s) : a.D > 32 ? launch_join<16>(a, s) : launch_join<8>(a, s);
}

}  // namespace pvs
