// Attention inside frames, backward, on the tensor cores.
//
// Two kernels of one form, so that every sum is taken in a fixed order and
// none needs atomics.  A block owns 128 rows (queries for dq, keys for dk and
// dv), held in shared memory, and walks the other side in tiles of 128 rows:
//   S = own1 other1^T, dP = own2 other2^T     (scores and do.v, or transposed)
//   P = exp(score - lse), dS = P (dP - delta) d(score)/d(s)
//   acc2 += P other,  acc1 += dS other1
// with own = (q, do), other = (k, v) for dq, and the other way round for dk
// (acc1) and dv (acc2 += P^T do).  P replaces S in tensor memory and dS dP, as
// the next products' operands.  Four warpgroups take 32 columns each; one warp
// issues the products, one the loads, one puts what belongs to the other side's
// rows (lse, delta, positions) into shared memory, one clears the rows of a last tile
// that belong to the next frame.
//
// The arithmetic reads S and dP in fragments (four rows and eight columns a
// thread), not a row a thread: what belongs to a column is then loaded once for
// four rows, by lanes that load different columns.  With a row a thread all lanes
// load the same column, which takes the shared memory, that the products are fed
// from, as long as a load of 512 different bytes.
//
// The accumulators of 128-element heads leave room for one S and one dP only,
// so the work is staggered: while the threads make dS of a tile, the tensor cores
// run acc2 and the next tile's S, and while they make the next P, acc1 and the
// next dP.  A product of 128 columns from shared memory takes 64 cycles, as much as
// one of 64 columns (55 measured): tiles of 64 columns with two buffers, tried
// first, left the tensor cores 1.4 times the work.
//
// delta = do.o of the rounded o would leave each row's dS with a sum that is
// not zero: an error of P times the rounding of o, which for a row that few
// keys share is larger than all other roundings.  The dq kernel therefore takes
// that delta as a first guess, sums P dP in 32 bits on the way (which is delta as
// the products have it), and mends dq by the difference times acc2 = P k; it
// leaves the summed delta (with the queries' lse and positions, laid out for bulk
// copies) for the dk, dv kernel.  That is one product more than
// the four that dq needs least, and no more exponentials.
//
// Measured: 4 ragged frames of up to 4,000, 8 heads of 64, distances, bf16: dq 207 us,
// dk and dv 202 us; 12,289 causal tokens, capped, 8 heads over 2 of 128, f16: 600 and
// 615 us.  Tensor cores 34 and 45 %, issue slots 50 to 61 %: products and arithmetic take
// turns.  At 128 elements that is for want of tensor memory; heads of 64 or less leave 128
// columns of it, where a second S would fit, which is not done.
//
// P and dS are held 2^kUp times their values in the storage type.  Float16 runs out of
// exponent below 2^-14, where the probabilities of some thousand keys lie, and ends at
// 65,504: a factor of 1,024 keeps P whole down to 2^-24, and leaves room for one of 60 (of a
// score so large that 32 bits hold it badly).  How large
// dS is goes by dout, too, which a loss scale moves anywhere:
// there dS has a power of two by |dP - delta| <= 2 |dout| |v|, so that 2^15 bounds it: for dq the
// row's own, with the largest v of the frame, for dk, whose sums go over the queries, the
// frame's, with the largest dout, too.  One small kernel reads dout and v for that.

#include "pv_attn.cuh"
#include "pv_tc.cuh"

#include <algorithm>
#include <type_traits>

namespace pvs {

namespace {

constexpr int kGroups = 4;                      // warpgroups of arithmetic
constexpr int kMath = kGroups * 128;
constexpr int kThreads = kMath + 128;
// Registers of a thread: 96 at launch (640 x 96 = 61,440); 512 x 104 + 128 x 64 = 61,440.
constexpr int kRegsMath = 104, kRegsOther = 64;
constexpr int kOwn = 128;    // rows of a block
constexpr int kOther = 128;  // rows of a step
constexpr int kCols = kOther / kGroups;  // columns of a thread
constexpr int kSides = 3;    // slots of what belongs to the other side's rows
constexpr float kLog2e = 1.4426950408889634f;
constexpr bool kHalf = std::is_same<Storage, __half>::value;
constexpr float kUp = kHalf ? 10.0f : 4.0f;  // log2 of the factor on P (and, in bfloat16, dS)
constexpr float kDown = kHalf ? 0x1p-10f : 0x1p-4f;

template <int kBlocks>
struct Smem {
  static constexpr int kTile = kOwn * 128 * kBlocks;  // bytes of 128 rows of a head
  static constexpr int kSlots = kBlocks == 1 ? 4 : 2;
  alignas(1024) unsigned char own[2][kTile];
  alignas(1024) unsigned char other[2][kSlots][kTile];
  alignas(16) float side[kSides][5][kOther];  // lse (as an offset of the exponent), delta (negated), positions
  float rest[kGroups][kOwn];      // dq: each warpgroup's sum of P (dP - delta)
  float guess[kOwn];              // dq: do.o of the rounded o
  float up[kOwn];                 // dq, float16: the rows' factors
  uint64_t own_full, dirty[2], clean[2], full[2][kSlots], empty[2][kSlots], s_full, dp_full, p_full, ds_full, acc_full, side_full[kSides],
      side_empty[kSides];
  uint32_t tmem;
  int given_up;
};

// All threads of the arithmetic.
__device__ __forceinline__ void math_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kMath) : "memory"); }

// A thread's four rows: 8 x + lane / 4 of its warp's 32.
struct Rows {
  float pos[3][4];         // negated
  float slope[4], mul;     // exponent = mul * (score + slope * distance) + off
  float cap_in;            // score = tanh of half this times the raw one, if capped
  float off[4], delta[4];  // dq: the rows' own (delta negated, times `up`); dk, dv: the columns', in shared memory
  float up[4];             // float16: dS is `up` times 2^kUp times its value
  float total[4];          // dq: sums of 2^kUp P (dP - delta), times `up`
  int lo[4], hi[4];        // of the thread's first column, columns seen: lo <= column < hi
};

// The power of two for gradients of rows of these norms; 1 where they are 0 or not finite.
__device__ __forceinline__ float factor(float dout, float v) {
  const float bound = 2.0f * dout * v;
  int e = 15 - static_cast<int>(kUp);
  if (bound > 0.0f && bound < INFINITY) frexpf(bound, &e);  // bound < 2^e
  return ldexpf(1.0f, 15 - static_cast<int>(kUp) - e);
}

constexpr int kElems = kCols / 2;  // of two of the four rows: registers of one 16-lane fragment
__device__ __forceinline__ constexpr int row_of(int h, int x) { return 2 * h + ((x >> 1) & 1); }
__device__ __forceinline__ constexpr int col_of(int x) { return (x >> 2) * 8 + (x & 1); }

// 32 rows' scores of 32 columns, from column `at` of tensor memory on, to P there, in
// the storage type.  `side` points to what belongs to the thread's first column.
// u keeps what dS is made of: P times the cap's slope; with a cap, dq takes that
// for acc2 too, and what the slope took from P, for the sum of P dP, goes to `rest`
// as half pairs (a small share, of which the rounding does not show).  One operation
// after the other over all elements: an element's chain is long, 32 of them hide it.
template <typename T, bool kDkv, int kCap, bool kSlopes, bool kMask>
__device__ __forceinline__ void probabilities(uint32_t at, const float* side, int axes, const Rows& row, float (*u)[kElems],
                                              uint32_t (*rest)[kElems / 2]) {
  tmem_ld_16x256b_x4(at, reinterpret_cast<uint32_t*>(u[0]));
  tmem_ld_16x256b_x4(at + (16u << 16), reinterpret_cast<uint32_t*>(u[1]));
  tc_wait_ld<kElems>(reinterpret_cast<uint32_t*>(u[0]));
  tc_wait_ld<kElems>(reinterpret_cast<uint32_t*>(u[1]));
  float steep[2][kCap ? kElems : 1];
  if (kCap) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int x = 0; x < kElems; ++x) {
        u[h][x] = capped<kCap>(u[h][x] * row.cap_in);
        steep[h][x] = fmaf(-u[h][x], u[h][x], 1.0f);
      }
  }
  if (kSlopes) {
    if (axes == 1) lower<1, kCols / 8>(u, side + 2 * kOther, kOther, row.pos, row.slope);
    if (axes == 2) lower<2, kCols / 8>(u, side + 2 * kOther, kOther, row.pos, row.slope);
    if (axes == 3) lower<3, kCols / 8>(u, side + 2 * kOther, kOther, row.pos, row.slope);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int x = 0; x < kElems; x += 2) {
      const int r = row_of(h, x);
      float2 l = make_float2(row.off[r], row.off[r]);
      if (kDkv) l = *reinterpret_cast<const float2*>(side + col_of(x));
      fma2(u[h][x], u[h][x + 1], u[h][x], u[h][x + 1], row.mul, row.mul, l.x, l.y);
    }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int x = 0; x < kElems; ++x) {
      u[h][x] = exp2_fast(u[h][x]);
      if (kMask) u[h][x] = col_of(x) >= row.lo[row_of(h, x)] && col_of(x) < row.hi[row_of(h, x)] ? u[h][x] : 0.0f;
    }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p[kElems / 2];
    if (!kCap || kDkv) {
#pragma unroll
      for (int x = 0; x < kElems; x += 2) p[x >> 1] = Pack<T>::two(u[h][x], u[h][x + 1]);
    }
    if (kCap) {
#pragma unroll
      for (int x = 0; x < kElems; x += 2) {
        const float e0 = u[h][x] * steep[h][x], e1 = u[h][x + 1] * steep[h][x + 1];
        if (!kDkv) {
          rest[h][x >> 1] = Pack<__half>::two(u[h][x] - e0, u[h][x + 1] - e1);
          p[x >> 1] = Pack<T>::two(e0, e1);
        }
        u[h][x] = e0;
        u[h][x + 1] = e1;
      }
    }
    tmem_st_16x128b_x4(at + (h ? 16u << 16 : 0u), p);
  }
}

// dP at column `at` to dS there.
template <typename T, bool kDkv, int kCap, bool kMask>
__device__ __forceinline__ void gradients(uint32_t at, const float* side, Rows& row, const float (*e)[kElems],
                                          const uint32_t (*rest)[kElems / 2]) {
  float g[2][kElems];
  tmem_ld_16x256b_x4(at, reinterpret_cast<uint32_t*>(g[0]));
  tmem_ld_16x256b_x4(at + (16u << 16), reinterpret_cast<uint32_t*>(g[1]));
  tc_wait_ld<kElems>(reinterpret_cast<uint32_t*>(g[0]));
  tc_wait_ld<kElems>(reinterpret_cast<uint32_t*>(g[1]));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t s[kElems / 2];
    float t[4] = {};
#pragma unroll
    for (int x = 0; x < kElems; x += 2) {
      const int r = row_of(h, x);
      float2 d = make_float2(row.delta[r], row.delta[r]);
      if (kDkv) d = *reinterpret_cast<const float2*>(side + kOther + col_of(x));
      if (std::is_same<T, __half>::value)
        fma2(g[h][x], g[h][x + 1], g[h][x], g[h][x + 1], row.up[kDkv ? 0 : r], row.up[kDkv ? 0 : r], d.x, d.y);
      else
        add2(g[h][x], g[h][x + 1], g[h][x], g[h][x + 1], d.x, d.y);
      // (A hidden place has e = 0, but what stands at it need not be finite.)
      const bool seen0 = !kMask || (col_of(x) >= row.lo[r] && col_of(x) < row.hi[r]);
      const bool seen1 = !kMask || (col_of(x + 1) >= row.lo[r] && col_of(x + 1) < row.hi[r]);
      float v0 = seen0 ? g[h][x] * e[h][x] : 0.0f, v1 = seen1 ? g[h][x + 1] * e[h][x + 1] : 0.0f;
      s[x >> 1] = Pack<T>::two(v0, v1);
      if (!kDkv) {
        if (kCap) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&rest[h][x >> 1]));
          v0 = seen0 ? g[h][x] * (e[h][x] + f.x) : 0.0f;
          v1 = seen1 ? g[h][x + 1] * (e[h][x + 1] + f.y) : 0.0f;
        }
        add2(t[x & 2], t[(x & 2) + 1], t[x & 2], t[(x & 2) + 1], v0, v1);
      }
    }
    tmem_st_16x128b_x4(at + (h ? 16u << 16 : 0u), s);
    if (!kDkv) {
      row.total[2 * h] += t[0] + t[1];
      row.total[2 * h + 1] += t[2] + t[3];
    }
  }
}

// The cap and the slopes are compile-time choices: code that a launch does not run
// still costs it instruction fetches (2 x 4096 tokens, 64-element heads, forward and
// backward: 411 us with both as branches, 375 us so).
template <typename T, int kBlocks, bool kDkv, int kCap, bool kSlopes>
__global__ void __launch_bounds__(kThreads, 1)
    pv_attn_bwd_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ CUtensorMap mdo) {
  using S = Smem<kBlocks>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kIssue = kMath / 32;  // the first warp after those of the arithmetic
  extern __shared__ __align__(1024) unsigned char raw[];
  S& sm = *reinterpret_cast<S*>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- which rows
  const int tile = blockIdx.x / a.heads, place = frame_of(a.tile0, a.frames, tile), f = a.order[place];
  const int head = blockIdx.x - tile * a.heads;
  const int nq = a.q0[f + 1] - a.q0[f], nk = a.k0[f + 1] - a.k0[f], shift = nk - nq;
  const int local = tile - a.tile0[place], tiles = a.tile0[place + 1] - a.tile0[place];
  // Under a causal mask late queries and early keys have the most work: they go first.
  const int own0 = (kDkv ? local : tiles - 1 - local) * kOwn;
  auto limit = [&](int i) { return a.causal ? max(min(max(i + shift + 1, a.prefix[f]), nk), 0) : nk; };
  // dk, dv: the query heads of a key head may be cut into parts, a block each.
  const int own_head = kDkv ? head / a.head_parts : head;
  const int heads = kDkv ? a.G / a.head_parts : 1;
  const int head0 = kDkv ? head * heads : own_head / a.G;
  int other_tile0 = 0, per_head;
  if (kDkv) {
    const int begin = a.causal && own0 >= a.prefix[f] ? max(own0 - shift, 0) : 0;
    other_tile0 = begin / kOther;
    per_head = max((nq + kOther - 1) / kOther - other_tile0, 0);
  } else {
    per_head = (limit(min(own0 + kOwn, nq) - 1) + kOther - 1) / kOther;
  }
  const int steps = per_head * heads;
  const int own_rows = kDkv ? nk : nq, other_rows = kDkv ? nq : nk;

  // ---- set up
  if (threadIdx.x == 0) {
    sm.given_up = 0;
    bar_init(&sm.own_full, 1);
    bar_init(&sm.acc_full, 1);
    for (int s = 0; s < 2; ++s) bar_init(&sm.dirty[s], 1), bar_init(&sm.clean[s], 1);
    for (int s = 0; s < 2; ++s)
      for (int i = 0; i < S::kSlots; ++i) bar_init(&sm.full[s][i], 1), bar_init(&sm.empty[s][i], 1);
    bar_init(&sm.s_full, 1);
    bar_init(&sm.dp_full, 1);
    bar_init(&sm.p_full, kMath / 32);
    bar_init(&sm.ds_full, kMath / 32);
    for (int i = 0; i < kSides; ++i) bar_init(&sm.side_full[i], 1), bar_init(&sm.side_empty[i], kMath / 32);
    fence_bar_init();
    tma_prefetch(&mq);
    tma_prefetch(&mk);
    tma_prefetch(&mv);
    tma_prefetch(&mdo);
  }
  if (warp == kIssue) tmem_alloc<512>(&sm.tmem);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = sm.tmem;  // columns: S 0, dP 128, acc1 256, acc2 256 + 64 kBlocks
  volatile int* given_up = &sm.given_up;
  constexpr bool sides = kDkv || kSlopes;
  wait_prior_grid();

  if (warp >= kIssue) regs_down<kRegsOther>();
  if (warp == kIssue + 1) {
    // ---- loads
    if (lane == 0 && steps > 0) {
      const CUtensorMap* own_map[2] = {kDkv ? &mk : &mq, kDkv ? &mv : &mdo};
      const CUtensorMap* other_map[2] = {kDkv ? &mq : &mk, kDkv ? &mdo : &mv};
      const bool own_heads[2] = {(kDkv ? a.k.head : a.q.head) != 0, (kDkv ? a.v.head : a.dout.head) != 0};
      const bool other_heads[2] = {(kDkv ? a.q.head : a.k.head) != 0, (kDkv ? a.dout.head : a.v.head) != 0};
      const int own_base = (kDkv ? a.k0[f] : a.q0[f]) + own0, other_base = kDkv ? a.q0[f] : a.k0[f];
      bar_expect(&sm.own_full, 2 * S::kTile);
#pragma unroll
      for (int s = 0; s < 2; ++s)
        for (int b = 0; b < kBlocks; ++b)
          tma_load4(sm.own[s] + b * kOwn * 128, own_map[s], b * 64, 0, own_heads[s] ? own_head : 0, own_base, &sm.own_full);
      int slot = 0, phase = 1, h = head0, left = per_head;
      const int first_row = other_base + other_tile0 * kOther;
      int row = first_row;
      bool ok = true;
      for (int n = 0; ok && n < steps; ++n) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!ok || !(ok = bar_wait(&sm.empty[s][slot], phase, given_up))) continue;
          bar_expect(&sm.full[s][slot], S::kTile);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
            tma_load4(sm.other[s][slot] + b * kOther * 128, other_map[s], b * 64, 0, other_heads[s] ? h : 0, row,
                      &sm.full[s][slot]);
        }
        row += kOther;
        if (--left == 0) left = per_head, row = first_row, ++h;
        if (++slot == S::kSlots) slot = 0, phase ^= 1;
      }
    }
  } else if (warp == kIssue) {
    // ---- products: one thread, with little to do between them.  It shares its
    // scheduler with four warps of arithmetic, and the tensor cores take few
    // products in advance: what it does between two of them, they wait for.
    if (elect_one() && steps > 0) {
      const uint32_t word_s = mma_word(kBf16, 128, kOther, false, false);
      const uint32_t word_a = mma_word(kBf16, 128, 0, false, true) | (static_cast<uint32_t>(a.Dn >> 3) << 17);
      const int ksteps = (a.D + 15) / 16;
      const uint32_t own_op = operand(smem_addr(sm.own[0]), 16), row_op = operand(smem_addr(sm.other[0][0]), 16);
      const uint32_t col_op = operand(smem_addr(sm.other[0][0]), kOther * 128);
      constexpr uint32_t kStep = S::kTile >> 4, kSide = S::kSlots * kStep;
      // The slot and its parity of the tile that S and dP (0, 1) come to next.
      int slot[2] = {0, 0}, parity[2] = {0, 0}, left[2] = {per_head, per_head}, cleaned[2] = {0, 0};
      const bool ragged = other_rows < (other_tile0 + per_head) * kOther;
      // Whether the tile's operand is there (its rows past the frame's end cleared).
      auto arrived = [&](int s) {
        if (!bar_wait(&sm.full[s][slot[s]], parity[s], given_up)) return false;
        if (--left[s] == 0) {
          left[s] = per_head;
          if (ragged) {
            bar_arrive(&sm.dirty[s]);
            if (!bar_wait(&sm.clean[s], cleaned[s], given_up)) return false;
            cleaned[s] ^= 1;
          }
        }
        return true;
      };
      auto scores = [&](int s) {  // S or dP of that tile
        const uint32_t own = own_op + s * kStep, other = row_op + s * kSide + slot[s] * kStep;
#pragma unroll
        for (int x = 0; x < 4 * kBlocks; ++x) {
          const uint32_t off = ((x >> 2) * kOwn * 128 + (x & 3) * 32) >> 4;
          if (x < ksteps) mma_ss(tm + s * 128, own + off, other + off, word_s, x > 0);
        }
        mma_commit(s ? &sm.dp_full : &sm.s_full);
        if (!kDkv && s) mma_commit(&sm.empty[1][slot[1]]);  // dq: nothing else needs v
        if (++slot[s] == S::kSlots) slot[s] = 0, parity[s] ^= 1;
      };
      // acc2 += P other (s = 0), acc1 += dS other1 (s = 1), of the tile in slot `at`.
      auto sums = [&](int s, int at, bool add) {
        const uint32_t b = col_op + (kDkv && s == 0 ? kSide : 0) + at * kStep;
        const uint32_t acc = tm + 256 + (s ? 0 : 64 * kBlocks), left = tm + s * 128;
#pragma unroll
        for (int x = 0; x < kOther / 16; ++x)  // a warpgroup's 32 columns lie in 16 of its own
          mma_ts(acc, left + x / (kCols / 16) * kCols + x % (kCols / 16) * 8, b + x * (2048 >> 4), word_a, add || x > 0);
        if (kDkv && s == 0) mma_commit(&sm.empty[1][at]);
        if (s == 1) mma_commit(&sm.empty[0][at]);
      };
      bool ok = bar_wait(&sm.own_full, 0, given_up) && arrived(0) && arrived(1);
      if (ok) {
        tc_after();
        scores(0);
        scores(1);
      }
      for (int n = 0, at = 0; ok && n < steps; ++n) {
        const bool more = n + 1 < steps;
        if (more && !(ok = arrived(0))) break;
        if (!(ok = bar_wait(&sm.p_full, n & 1, given_up))) break;
        tc_after();
        sums(0, at, n > 0);
        if (more) scores(0);
        if (more && !(ok = arrived(1))) break;
        if (!(ok = bar_wait(&sm.ds_full, n & 1, given_up))) break;
        tc_after();
        sums(1, at, n > 0);
        if (more)
          scores(1);
        else
          mma_commit(&sm.acc_full);
        if (++at == S::kSlots) at = 0;
      }
    }
    __syncwarp();
  } else if (warp == kIssue + 3) {
    // ---- rows past the frame's end are another frame's, whatever they hold
    const int have = other_rows - (other_tile0 + per_head - 1) * kOther;
    if (per_head > 0 && have < kOther) {
      bool ok = true;
      for (int n = per_head - 1, k = 0; ok && n < steps; n += per_head, k ^= 1) {
        const int slot = n % S::kSlots;
        for (int s = 0; ok && s < 2; ++s) {
          if (!(ok = warp_wait(&sm.dirty[s], k, given_up))) break;
          uint4* v = reinterpret_cast<uint4*>(sm.other[s][slot]);
          for (int c = 0; c < kBlocks; ++c)
            for (int i = have * 8 + lane; i < kOther * 8; i += 32) v[c * kOther * 8 + i] = make_uint4(0, 0, 0, 0);
          fence_to_async();
          warp_arrive(&sm.clean[s]);
        }
      }
    }
  } else if (warp == kIssue + 2) {
    // ---- what belongs to the other side's rows
    if (kDkv) {
      // The dq kernel left it as it is needed: whole pieces, past a frame's end too (what
      // is there is hidden).
      if (lane == 0 && steps > 0) {
        int slot = 0, phase = 1, h = head0, left = per_head;
        const int first_row = a.side0[f] + other_tile0 * kOther;
        const float* const pos = a.sides + 2 * a.H * a.sides_row;
        int row = first_row;
        for (int n = 0; n < steps; ++n) {
          if (!bar_wait(&sm.side_empty[slot], phase, given_up)) break;
          bar_expect(&sm.side_full[slot], (2 + (kSlopes ? a.axes : 0)) * kOther * 4);
          const float* const off = a.sides + h * a.sides_row + row;
          tma_copy(sm.side[slot][0], off, kOther * 4, &sm.side_full[slot]);
          tma_copy(sm.side[slot][1], off + a.H * a.sides_row, kOther * 4, &sm.side_full[slot]);
          for (int c = 0; kSlopes && c < a.axes; ++c)
            tma_copy(sm.side[slot][2 + c], pos + c * a.sides_row + row, kOther * 4, &sm.side_full[slot]);
          row += kOther;
          if (--left == 0) left = per_head, row = first_row, ++h;
          if (++slot == kSides) slot = 0, phase ^= 1;
        }
      }
    } else if (kSlopes && steps > 0) {
      // Positions, each tile's loaded while the last one's are handed over.
      int pos[3][4];
      auto load = [&](int tile) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const long long row = a.k0[f] + min(tile * kOther + x * 32 + lane, nk - 1);
#pragma unroll
          for (int c = 0; c < 3; ++c)
            if (c < a.axes) pos[c][x] = a.kpos[row * a.kpos_stride + c];
        }
      };
      load(0);
      for (int n = 0; n < steps; ++n) {
        const int slot = n % kSides;
        float now[3][4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int c = 0; c < 3; ++c)
            if (c < a.axes) now[c][x] = static_cast<float>(pos[c][x]);
        if (n + 1 < steps) load(n + 1);
        if (!warp_wait(&sm.side_empty[slot], ((n / kSides) & 1) ^ 1, given_up)) break;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int c = 0; c < 3; ++c)
            if (c < a.axes) sm.side[slot][2 + c][x * 32 + lane] = now[c][x];
        warp_arrive(&sm.side_full[slot]);
      }
    }
  } else if (warp < kIssue) {
    // ---- probabilities and gradients: 32 own rows a warp, in fragments: four rows and
    // 8 of the warpgroup's 32 columns a thread
    regs_up<kRegsMath>();
    const int wg = warp >> 2, r0 = (warp & 3) * 32, quad = lane & 3;
    const uint32_t mine = tm + (static_cast<uint32_t>(r0) << 16);
    // Outputs, and the first guess of delta: one row a thread.
    const int r = r0 + lane, own = own0 + r;
    const bool live = own < own_rows;
    const long long own_row = (kDkv ? a.k0[f] : a.q0[f]) + own;
    if (!kDkv) {
      if (wg == 0) {
        float delta = 0.0f, norm = 0.0f;
        if (live) {
          const char* o = a.o.data + own_row * a.o.row + own_head * a.o.head;
          const char* g = a.dout.data + own_row * a.dout.row + own_head * a.dout.head;
          for (int d = 0; d < a.D; d += 8) {
            float x[8], y[8];
            Pack<T>::load(o + d * 2, x);
            Pack<T>::load(g + d * 2, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) delta = fmaf(x[e], y[e], delta);
            if (!kBf16) {
#pragma unroll
              for (int e = 0; e < 8; ++e) norm = fmaf(y[e], y[e], norm);
            }
          }
        }
        sm.guess[r] = delta;
        if (!kBf16) sm.up[r] = a.up ? factor(sqrtf(norm), a.up[f].y) : 1.0f;
      }
      math_sync();
    }
    Rows row{};
    const float up_frame = !kBf16 && a.up ? a.up[f].x : 1.0f;
    if (kDkv) row.up[0] = up_frame;
    row.mul = (kCap ? a.cap : a.scale) * kLog2e;
    row.cap_in = kCap ? 2.0f * a.scale * kLog2e / a.cap : 0.0f;
    // A place is seen if its column is at least `from` and below `to`.
    int from[4], to[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int rx = r0 + 8 * x + (lane >> 2), ox = own0 + rx;
      const bool in = ox < own_rows;
      const long long at = (kDkv ? a.k0[f] : a.q0[f]) + ox;
      from[x] = 0;
      to[x] = other_rows;
      if (a.causal) {
        if (kDkv)
          from[x] = ox < a.prefix[f] ? 0 : ox - shift;
        else
          to[x] = in ? limit(ox) : 0;
      }
      if (!kDkv) {
        if (in) row.off[x] = fmaf(-kLog2e, a.lse[static_cast<long long>(own_head) * a.queries + at], kUp);
        if (!kBf16) row.up[x] = sm.up[rx];
        row.delta[x] = kBf16 ? -sm.guess[rx] : -sm.guess[rx] * row.up[x];
      }
      if (kSlopes && in) {
        if (!kDkv) row.slope[x] = -a.slopes[own_head] * kLog2e / row.mul;
#pragma unroll
        for (int c = 0; c < 3; ++c)
          if (c < a.axes)
            row.pos[c][x] = -static_cast<float>(kDkv ? a.kpos[at * a.kpos_stride + c] : a.qpos[at * a.qpos_stride + c]);
      }
    }
    const int c0 = wg * kCols;
    const uint32_t s_at = mine + c0, dp_at = mine + 128 + c0;
    bool ok = true;
    // One step, with the mask a compile-time choice.
    auto step = [&](auto mask, int n, const float* side) {
      constexpr bool kMask = decltype(mask)::value;
      float e[2][kElems];
      uint32_t rest[2][kElems / 2];
      probabilities<T, kDkv, kCap, kSlopes, kMask>(s_at, side, a.axes, row, e, rest);
      tc_wait_st();
      tc_before();
      warp_arrive(&sm.p_full);
      if (!(ok = warp_wait(&sm.dp_full, n & 1, given_up))) return;
      tc_after();
      gradients<T, kDkv, kCap, kMask>(dp_at, side, row, e, rest);
      tc_wait_st();
      tc_before();
      warp_arrive(&sm.ds_full);
    };
    int next_head = head0, left = 0, row0 = 0;  // dk, dv: the other side's next head, and the tiles to come of this one
    for (int n = 0; n < steps; ++n, row0 += kOther) {
      const int slot = n % kSides;
      if (left-- == 0) {
        left = per_head - 1;
        row0 = other_tile0 * kOther;
        if (kDkv && kSlopes) {
          const float slope = -a.slopes[next_head] * kLog2e / row.mul;
#pragma unroll
          for (int x = 0; x < 4; ++x) row.slope[x] = slope;
        }
        ++next_head;
      }
      if (sides && !(ok = warp_wait(&sm.side_full[slot], (n / kSides) & 1, given_up))) break;
      // Seen whole: nothing of the tile is hidden from any of the block's rows.
      const bool whole = row0 + kOther <= other_rows &&
                         (!a.causal || (kDkv ? limit(row0) >= min(own0 + kOwn, nk) : limit(own0) >= row0 + kOther));
      if (!whole) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          row.lo[x] = from[x] - row0 - c0 - 2 * quad;
          row.hi[x] = to[x] - row0 - c0 - 2 * quad;
        }
      }
      if (!(ok = warp_wait(&sm.s_full, n & 1, given_up))) break;
      tc_after();
      const float* side = &sm.side[slot][0][c0 + 2 * quad];
      if (whole)
        step(std::false_type{}, n, side);
      else
        step(std::true_type{}, n, side);
      if (!ok) break;
      if (sides) warp_arrive(&sm.side_empty[slot]);
    }
    // ---- outputs
    const bool any = steps > 0;
    if (any && ok) ok = warp_wait(&sm.acc_full, 0, given_up);
    tc_after();
    // dq: the sum of P (dP - delta) is what delta is off by (here `up` times that).
    float total = 0.0f;
    if (!kDkv) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        row.total[x] += __shfl_xor_sync(0xFFFFFFFFu, row.total[x], 1);
        row.total[x] += __shfl_xor_sync(0xFFFFFFFFu, row.total[x], 2);
        if (quad == 0) sm.rest[wg][r0 + 8 * x + (lane >> 2)] = row.total[x];
      }
      math_sync();
      total = ((sm.rest[0][r] + sm.rest[1][r]) + (sm.rest[2][r] + sm.rest[3][r])) * kDown;
      if (live && wg == 0) {
        float* const side = a.sides + own_head * a.sides_row + a.side0[f] + own;
        side[0] = fmaf(-kLog2e, a.lse[static_cast<long long>(own_head) * a.queries + own_row], kUp);
        side[a.H * a.sides_row] = kBf16 ? -(sm.guess[r] + total) : -fmaf(sm.guess[r], up_frame, total * (up_frame / sm.up[r]));
        if (own_head == 0)
          for (int c = 0; c < a.axes; ++c)
            side[(2 * a.H + c) * a.sides_row] = static_cast<float>(a.qpos[own_row * a.qpos_stride + c]);
      }
    }
    const float bad = !ok || *given_up ? __int_as_float(0x7FFFFFFF) : 1.0f;  // a wait ran out: nothing here is an answer
    const int which = wg & 1;  // dk, dv: 0 and 1
    const View& out = kDkv ? (which ? a.dv : a.dk) : a.dq;
    char* to_row = out.data + own_row * out.row + own_head * out.head;
    const bool parts = kDkv && a.head_parts > 1;
    float* part = parts ? a.part_o + (((static_cast<long long>(head % a.head_parts) * 2 + which) * a.keys + own_row) * a.Hk + own_head) * a.D
                        : nullptr;
    const float k1 = (kDkv && which ? 1.0f : kBf16 ? a.scale : a.scale / (kDkv ? up_frame : sm.up[r])) * kDown * bad;
    const uint32_t acc = mine + 256 + (kDkv && which ? 64 * kBlocks : 0);
    for (int x = (kDkv ? wg >> 1 : wg) * 16; x < a.Dn; x += kDkv ? 32 : 64) {
      uint32_t c[16], d[16];
      float v[16];
      if (any) {
        tmem_ld16(acc + x, c);
        if (!kDkv) tmem_ld16(acc + 64 * kBlocks + x, d);
        tc_wait_ld<16>(c);
        if (!kDkv) tc_wait_ld<16>(d);
      }
#pragma unroll
      for (int y = 0; y < 16; ++y) {
        float w = any ? __uint_as_float(c[y]) : 0.0f;
        if (!kDkv && any) w = fmaf(-total, __uint_as_float(d[y]), w);
        v[y] = w * k1;
      }
#pragma unroll
      for (int y = 0; y < 16; y += 8) {
        if (!live || x + y >= a.D) continue;
        if (parts) {
          Pack<float>::store(part + x + y, v + y);
          Pack<float>::store(part + x + y + 4, v + y + 4);
        } else {
          Pack<T>::store(to_row + (x + y) * 2, v + y);
        }
      }
      __syncwarp();
    }
    tc_before();
  }
  __syncthreads();
  if (warp == kIssue) {
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

#ifdef PV_ATTN_HALF
// A frame's `up` (block: frame blockIdx.y, every gridDim.x-th stretch of its rows' heads, as
// many lanes a head as it has pieces of 16 bytes).  Rows that are not finite do not count: they
// spoil their own gradients, not the frame's.  Bound by its loads' latency: 33 MB (8,192 tokens
// of 8 heads of 128) take 15 us from DRAM, a few hundred tokens 6 us; the gradients of
// 12,289 capped tokens take 24 us more in all with it (1,646 -> 1,670 us with the forward pass).
constexpr int kNormThreads = 256;

template <int kLanes>
__global__ void __launch_bounds__(kNormThreads) pv_attn_up_kernel(const __grid_constant__ AttnArgs a) {
  __shared__ float2 warps[kNormThreads / 32];
  __shared__ bool last;
  wait_prior_grid();
  const int f = blockIdx.y, lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  constexpr int kRows = kNormThreads / kLanes;
  auto largest = [&](const View& view, int row0, int rows, int heads) {
    const int step = gridDim.x * kRows, step_t = step / heads, step_h = step - step_t * heads;
    const int first = blockIdx.x * kRows + group;
    long long t = first / heads;
    int h = first - static_cast<int>(t) * heads;
    float most = 0.0f;
    constexpr int kAhead = 4;
    for (long long i = static_cast<long long>(blockIdx.x) * kRows; i < static_cast<long long>(rows) * heads; i += kAhead * step) {
      uint4 raw[kAhead] = {};
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        if (t < rows && lane * 8 < a.D)
          raw[x] = *reinterpret_cast<const uint4*>(view.data + (row0 + t) * view.row + h * view.head + lane * 16);
        t += step_t;
        h += step_h;
        if (h >= heads) h -= heads, ++t;
      }
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        float v[8], s = 0.0f;
        Pack<Storage>::open(raw[x], v);
#pragma unroll
        for (int y = 0; y < 8; ++y) s = fmaf(v[y], v[y], s);
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (s < INFINITY) most = fmaxf(most, s);
      }
    }
    return most;
  };
  auto block_most = [&](float2 m) {  // for thread 0
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      m.x = fmaxf(m.x, __shfl_xor_sync(0xFFFFFFFFu, m.x, o));
      m.y = fmaxf(m.y, __shfl_xor_sync(0xFFFFFFFFu, m.y, o));
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = m;
    __syncthreads();
    for (int w = 0; w < kNormThreads / 32; ++w) m = make_float2(fmaxf(m.x, warps[w].x), fmaxf(m.y, warps[w].y));
    return m;
  };
  const float2 mine = block_most(make_float2(largest(a.dout, a.q0[f], a.q0[f + 1] - a.q0[f], a.H),
                                             largest(a.v, a.k0[f], a.k0[f + 1] - a.k0[f], a.Hk)));
  float2* const parts = a.norms + static_cast<long long>(f) * gridDim.x;
  if (threadIdx.x == 0) {
    parts[blockIdx.x] = mine;
    __threadfence();
    last = atomicAdd(a.norms_done + f, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (last) {
    __threadfence();
    float2 m = make_float2(0.0f, 0.0f);
    for (int p = threadIdx.x; p < static_cast<int>(gridDim.x); p += kNormThreads) {
      const float2 x = __ldcg(parts + p);
      m = make_float2(fmaxf(m.x, x.x), fmaxf(m.y, x.y));
    }
    m = block_most(m);
    if (threadIdx.x == 0) {
      a.up[f] = make_float2(factor(sqrtf(m.x), sqrtf(m.y)), sqrtf(m.y));
      a.norms_done[f] = 0;
    }
  }
  allow_next_grid();
}
#endif

// dk and dv of a key head whose query heads were cut into parts: the parts' sum, in order.
template <typename T>
__global__ void __launch_bounds__(256) pv_attn_bwd_join_kernel(const __grid_constant__ AttnArgs a) {
  wait_prior_grid();
  const long long per = static_cast<long long>(a.keys) * a.Hk * a.D / 8;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < 2 * per; i += static_cast<long long>(gridDim.x) * 256) {
    const int wg = i >= per;
    const long long at = (i - wg * per) * 8;
    float v[8] = {};
    for (int p = 0; p < a.head_parts; ++p) {
      const float* part = a.part_o + (static_cast<long long>(p) * 2 + wg) * per * 8 + at;
      float x[8];
      Pack<float>::load(part, x);
      Pack<float>::load(part + 4, x + 4);
#pragma unroll
      for (int y = 0; y < 8; ++y) v[y] += x[y];
    }
    const long long d = at % a.D, head = at / a.D % a.Hk, r = at / a.D / a.Hk;
    const View& out = wg ? a.dv : a.dk;
    Pack<T>::store(out.data + r * out.row + head * out.head + d * 2, v);
  }
  allow_next_grid();
}

template <int kBlocks, bool kDkv, int kCap, bool kSlopes>
int launch_bwd(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s) {
  if (grid.x == 0) return PV_OK;
  auto kernel = pv_attn_bwd_kernel<Storage, kBlocks, kDkv, kCap, kSlopes>;
  const int smem = static_cast<int>(sizeof(Smem<kBlocks>)) + 1024;
  const int st = allow_smem(kernel, smem);
  return st == PV_OK ? launch_pdl(kernel, grid, kThreads, smem, s, a, m.q, m.k, m.v, m.dout) : st;
}

template <int kBlocks, bool kDkv>
int with_scores(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s) {
  if (a.cap > kSmallCap)
    return a.slopes ? launch_bwd<kBlocks, kDkv, kAny, true>(a, m, grid, s) : launch_bwd<kBlocks, kDkv, kAny, false>(a, m, grid, s);
  if (a.cap > 0.0f)
    return a.slopes ? launch_bwd<kBlocks, kDkv, kSmall, true>(a, m, grid, s) : launch_bwd<kBlocks, kDkv, kSmall, false>(a, m, grid, s);
  return a.slopes ? launch_bwd<kBlocks, kDkv, kNoCap, true>(a, m, grid, s) : launch_bwd<kBlocks, kDkv, kNoCap, false>(a, m, grid, s);
}

}  // namespace

#ifdef PV_ATTN_HALF
int attn_backward_up_half(const AttnArgs& a, cudaStream_t s) {
  const dim3 grid(a.norm_parts, a.frames);
  if (a.D > 64) return launch_pdl(pv_attn_up_kernel<16>, grid, kNormThreads, 0, s, a);
  return a.D > 32 ? launch_pdl(pv_attn_up_kernel<8>, grid, kNormThreads, 0, s, a)
                  : launch_pdl(pv_attn_up_kernel<4>, grid, kNormThreads, 0, s, a);
}
#endif

int PV_ATTN_NAME(attn_backward_dq)(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s) {
  return a.D > 64 ? with_scores<2, false>(a, m, grid, s) : with_scores<1, false>(a, m, grid, s);
}

int PV_ATTN_NAME(attn_backward_dkv)(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s) {
  const int st = a.D > 64 ? with_scores<2, true>(a, m, grid, s) : with_scores<1, true>(a, m, grid, s);
  if (st != PV_OK || a.head_parts < 2 || grid.x == 0) return st;
  const long long words = static_cast<long long>(a.keys) * a.Hk * a.D / 4;
  const dim3 g(static_cast<unsigned int>(std::min<long long>((words + 255) / 256, 4096)));
  return launch_pdl(pv_attn_bwd_join_kernel<Storage>, g, 256, 0, s, a);
}

}  // namespace pvs
