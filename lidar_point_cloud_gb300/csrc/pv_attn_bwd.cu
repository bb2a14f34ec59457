// Attention inside frames, backward, on the tensor cores.
//
// Two kernels of one form, so that every sum is taken in a fixed order and
// none needs atomics.  A block owns 128 rows (queries for dq, keys for dk and
// dv), held in shared memory, and walks the other side in tiles of 64 rows:
//   S = own1 other1^T, dP = own2 other2^T     (scores and do.v, or transposed)
//   P = exp(score - lse), dS = P (dP - delta) d(score)/d(s)
//   acc1 += dS other1,  acc2 += P other
// with own = (q, do), other = (k, v) for dq, and the other way round for dk
// (acc1) and dv (acc2 += P^T do).  S and dP are double-buffered in tensor memory;
// P and dS replace them there, as the next products' operands.  Warps 0-3 and
// 4-7 take the two buffers in turn, one row a thread; warp 8 issues the
// products, warp 9 the loads, warp 10 puts what belongs to the other side's
// rows (lse, delta, positions) into shared memory.
//
// delta = do.o of the rounded o would leave each row's dS with a sum that is
// not zero: an error of P times the rounding of o, which for a row that few
// keys share is larger than all other roundings.  The dq kernel therefore takes
// that delta as a first guess, sums P dP in 32 bits on the way (which is delta as
// the products have it), and mends dq by the difference times acc2 = P k; it
// leaves the summed delta for the dk, dv kernel.  That is one product more than
// the four that dq needs least, and no more exponentials.
//
// P and dS are held 16 times their values in the storage type: float16 runs out
// of exponent below 2^-14, where the probabilities of some thousand keys lie.

#include "pv_attn.cuh"
#include "pv_tc.cuh"

#include <type_traits>

namespace pvs {

namespace {

constexpr int kThreads = 384;
constexpr int kRegsMath = 208, kRegsOther = 80;  // 256 x 208 + 128 x 80 = 63,488 of 384 x 168 = 64,512
constexpr int kOwn = 128;    // rows of a block
constexpr int kOther = 64;   // rows of a step
constexpr int kSides = 4;    // slots of what belongs to the other side's rows
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kUp = 4.0f;  // log2 of the factor on P and dS
constexpr float kDown = 0.0625f;

template <int kBlocks>
struct Smem {
  static constexpr int kOwnBytes = kOwn * 128 * kBlocks;
  static constexpr int kOtherBytes = kOther * 128 * kBlocks;
  static constexpr int kSlots = kBlocks == 1 ? 6 : 4;
  alignas(1024) unsigned char own[2][kOwnBytes];
  alignas(1024) unsigned char other[kSlots][2][kOtherBytes];
  float side[kSides][5][kOther];  // lse (as an offset of the exponent), delta (negated), positions
  float rest[2][kOwn];            // dq: each warpgroup's sum of P dP
  uint64_t own_full, full[kSlots], empty[kSlots], sp_full[2], pd_full[2], acc_full, side_full[kSides], side_empty[kSides];
  uint32_t tmem;
  int given_up;
};

struct Row {
  float pos[3];        // negated
  float slope, mul;    // exponent = mul * (score + slope * distance) + off
  float cap_in;        // score = tanh of half this times the raw one, if capped
  float off, delta;    // dq: the row's own (delta negated); dk, dv: a column's, in shared memory
  float total;         // dq: sum of 16 P (dP - delta)
  int lo, hi;          // columns seen: lo <= column < hi
};

// One row's 64 scores and dP, at column `at` and 64 after it, to 16 P and 16 dS
// in the storage type in their place (dq with a cap: P times the cap's slope
// for P).  32 columns at a time, one operation after the other over all of
// them: an element's chain is long, 32 of them hide it.
template <typename T, bool kDkv, bool kCap, bool kMask>
__device__ __forceinline__ void tile(uint32_t at, const float (*side)[kOther], int axes, Row& row) {
  float u[2][32], g[2][32];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    tmem_ld32(at + h * 32, reinterpret_cast<uint32_t*>(u[h]));
    tmem_ld32(at + 64 + h * 32, reinterpret_cast<uint32_t*>(g[h]));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    tc_wait_ld<32>(reinterpret_cast<uint32_t*>(u[h]));
    tc_wait_ld<32>(reinterpret_cast<uint32_t*>(g[h]));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float steep[kCap ? 32 : 1];
    if (kCap) {
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        u[h][x] = tanh_half(u[h][x] * row.cap_in);
        steep[x] = fmaf(-u[h][x], u[h][x], 1.0f);
      }
    }
    if (axes == 1) lower<1, 32>(u[h], &side[2][h * 32], kOther, row.pos, row.slope);
    if (axes == 2) lower<2, 32>(u[h], &side[2][h * 32], kOther, row.pos, row.slope);
    if (axes == 3) lower<3, 32>(u[h], &side[2][h * 32], kOther, row.pos, row.slope);
#pragma unroll
    for (int x = 0; x < 32; x += 4) {
      float4 l = make_float4(row.off, row.off, row.off, row.off), d = make_float4(row.delta, row.delta, row.delta, row.delta);
      if (kDkv) {
        l = *reinterpret_cast<const float4*>(&side[0][h * 32 + x]);
        d = *reinterpret_cast<const float4*>(&side[1][h * 32 + x]);
      }
      fma2(u[h][x], u[h][x + 1], u[h][x], u[h][x + 1], row.mul, row.mul, l.x, l.y);
      fma2(u[h][x + 2], u[h][x + 3], u[h][x + 2], u[h][x + 3], row.mul, row.mul, l.z, l.w);
      add2(g[h][x], g[h][x + 1], g[h][x], g[h][x + 1], d.x, d.y);
      add2(g[h][x + 2], g[h][x + 3], g[h][x + 2], g[h][x + 3], d.z, d.w);
    }
#pragma unroll
    for (int x = 0; x < 32; ++x) u[h][x] = exp2_fast(u[h][x]);
#pragma unroll
    for (int x = 0; x < 32; ++x) {
      g[h][x] *= u[h][x];
      if (kMask) {
        const bool seen = h * 32 + x >= row.lo && h * 32 + x < row.hi;
        u[h][x] = seen ? u[h][x] : 0.0f;
        g[h][x] = seen ? g[h][x] : 0.0f;
      }
    }
    if (!kDkv) {
      float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
      for (int x = 0; x < 32; x += 4) {
        add2(s0, s1, s0, s1, g[h][x], g[h][x + 1]);
        add2(s2, s3, s2, s3, g[h][x + 2], g[h][x + 3]);
      }
      row.total += (s0 + s1) + (s2 + s3);
    }
    if (kCap) {
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        g[h][x] *= steep[x];
        if (!kDkv) u[h][x] *= steep[x];
      }
    }
    uint32_t p[16], s[16];
#pragma unroll
    for (int x = 0; x < 32; x += 2) {
      p[x >> 1] = Pack<T>::two(u[h][x], u[h][x + 1]);
      s[x >> 1] = Pack<T>::two(g[h][x], g[h][x + 1]);
    }
    tmem_st16(at + h * 16, p);
    tmem_st16(at + 64 + h * 16, s);
  }
}

template <typename T, int kBlocks, bool kDkv>
__global__ void __launch_bounds__(kThreads, 1)
    pv_attn_bwd_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ CUtensorMap mdo) {
  using S = Smem<kBlocks>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) unsigned char raw[];
  S& sm = *reinterpret_cast<S*>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- which rows
  const int f = frame_of(a.tile0, a.frames, blockIdx.x);
  const int nq = a.q0[f + 1] - a.q0[f], nk = a.k0[f + 1] - a.k0[f], shift = nk - nq;
  const int local = blockIdx.x - a.tile0[f], tiles = a.tile0[f + 1] - a.tile0[f];
  // Under a causal mask late queries and early keys have the most work: they go first.
  const int own0 = (kDkv ? local : tiles - 1 - local) * kOwn;
  auto limit = [&](int i) { return a.causal ? max(min(max(i + shift + 1, a.prefix[f]), nk), 0) : nk; };
  int other_tile0, per_head, steps;
  if (kDkv) {
    const int begin = a.causal && own0 >= a.prefix[f] ? max(own0 - shift, 0) : 0;
    other_tile0 = begin / kOther;
    per_head = max((nq + kOther - 1) / kOther - other_tile0, 0);
    steps = per_head * a.G;
  } else {
    other_tile0 = 0;
    per_head = steps = (limit(min(own0 + kOwn, nq) - 1) + kOther - 1) / kOther;
  }
  const int own_rows = kDkv ? nk : nq, other_rows = kDkv ? nq : nk;
  const int own_head = blockIdx.y;
  // Head of the other side at step n, and its first row.
  auto other_head = [&](int n) { return kDkv ? own_head * a.G + n / per_head : own_head / a.G; };
  auto other_row = [&](int n) { return (other_tile0 + (kDkv ? n % per_head : n)) * kOther; };

  // ---- set up
  if (threadIdx.x == 0) {
    sm.given_up = 0;
    bar_init(&sm.own_full, 1);
    bar_init(&sm.acc_full, 1);
    for (int i = 0; i < S::kSlots; ++i) bar_init(&sm.full[i], 1), bar_init(&sm.empty[i], 1);
    for (int b = 0; b < 2; ++b) bar_init(&sm.sp_full[b], 1), bar_init(&sm.pd_full[b], kOwn);
    for (int i = 0; i < kSides; ++i) bar_init(&sm.side_full[i], 32), bar_init(&sm.side_empty[i], kOwn);
    fence_bar_init();
    tma_prefetch(&mq);
    tma_prefetch(&mk);
    tma_prefetch(&mv);
    tma_prefetch(&mdo);
  }
  if (warp == 8) tmem_alloc<512>(&sm.tmem);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = sm.tmem;
  volatile int* given_up = &sm.given_up;
  const bool sides = kDkv || a.slopes != nullptr;
  wait_prior_grid();

  if (warp >= 8) regs_down<kRegsOther>();
  if (warp == 9) {
    // ---- loads
    if (lane == 0 && steps > 0) {
      const CUtensorMap* o1 = kDkv ? &mk : &mq;
      const CUtensorMap* o2 = kDkv ? &mv : &mdo;
      const CUtensorMap* t1 = kDkv ? &mq : &mk;
      const CUtensorMap* t2 = kDkv ? &mdo : &mv;
      const View& v1 = kDkv ? a.k : a.q;
      const View& v2 = kDkv ? a.v : a.dout;
      const View& w1 = kDkv ? a.q : a.k;
      const View& w2 = kDkv ? a.dout : a.v;
      const int own_base = (kDkv ? a.k0[f] : a.q0[f]) + own0, other_base = kDkv ? a.q0[f] : a.k0[f];
      // The second half of the own rows may lie past the last row of all: it is
      // then left out (nothing of those rows is written).
      const int halves = own0 + kOther < own_rows ? 2 : 1;
      bar_expect(&sm.own_full, 2 * halves * kOther * 128 * kBlocks);
      for (int b = 0; b < kBlocks; ++b)
        for (int x = 0; x < halves; ++x) {
          tma_load4(sm.own[0] + b * kOwn * 128 + x * kOther * 128, o1, b * 64, 0, v1.head ? own_head : 0,
                    own_base + x * kOther, &sm.own_full);
          tma_load4(sm.own[1] + b * kOwn * 128 + x * kOther * 128, o2, b * 64, 0, v2.head ? own_head : 0,
                    own_base + x * kOther, &sm.own_full);
        }
      for (int n = 0; n < steps; ++n) {
        const int slot = n % S::kSlots;
        if (!bar_wait(&sm.empty[slot], ((n / S::kSlots) & 1) ^ 1, given_up)) break;
        bar_expect(&sm.full[slot], 2 * S::kOtherBytes);
        const int h = other_head(n), row = other_base + other_row(n);
        for (int b = 0; b < kBlocks; ++b) {
          tma_load4(sm.other[slot][0] + b * kOther * 128, t1, b * 64, 0, w1.head ? h : 0, row, &sm.full[slot]);
          tma_load4(sm.other[slot][1] + b * kOther * 128, t2, b * 64, 0, w2.head ? h : 0, row, &sm.full[slot]);
        }
      }
    }
  } else if (warp == 8) {
    // ---- products
    const uint32_t word_s = mma_word(kBf16, 128, kOther, false, false);
    const uint32_t word_a = mma_word(kBf16, 128, 0, false, true) | (static_cast<uint32_t>(a.Dn >> 3) << 17);
    const int ksteps = (a.D + 15) / 16;
    const uint32_t acc1 = tm + 256, acc2 = tm + 256 + 64 * kBlocks;
    bool ok = steps > 0 && warp_wait(&sm.own_full, 0, given_up);
    auto scores = [&](int n) {
      const int slot = n % S::kSlots, b = n & 1;
      if (!warp_wait(&sm.full[slot], (n / S::kSlots) & 1, given_up)) return false;
      const int have = other_rows - other_row(n);
      if (have < kOther) {
        // Rows past the frame's end are another frame's, whatever they hold.
        for (int s = 0; s < 2; ++s) {
          uint4* v = reinterpret_cast<uint4*>(sm.other[slot][s]);
          for (int c = 0; c < kBlocks; ++c)
            for (int i = have * 8 + lane; i < kOther * 8; i += 32) v[c * kOther * 8 + i] = make_uint4(0, 0, 0, 0);
        }
        fence_to_async();
        __syncwarp();
      }
      tc_after();
      if (elect_one()) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t own = operand(smem_addr(sm.own[s]), 16), other = operand(smem_addr(sm.other[slot][s]), 16);
#pragma unroll
          for (int x = 0; x < 4 * kBlocks; ++x)
            if (x < ksteps)
              mma_ss(tm + b * 128 + s * 64, own + (((x >> 2) * kOwn * 128 + (x & 3) * 32) >> 4),
                     other + (((x >> 2) * kOther * 128 + (x & 3) * 32) >> 4), word_s, x > 0);
        }
        mma_commit(&sm.sp_full[b]);
      }
      __syncwarp();
      return true;
    };
    for (int n = 0; ok && n < min(steps, 2); ++n) ok = scores(n);
    for (int n = 0; ok && n < steps; ++n) {
      const int slot = n % S::kSlots, b = n & 1;
      if (!(ok = warp_wait(&sm.pd_full[b], (n >> 1) & 1, given_up))) break;
      tc_after();
      if (elect_one()) {
        const uint32_t b1 = operand(smem_addr(sm.other[slot][0]), kOther * 128);
        const uint32_t b2 = kDkv ? operand(smem_addr(sm.other[slot][1]), kOther * 128) : b1;
#pragma unroll
        for (int x = 0; x < kOther / 16; ++x)
          mma_ts(acc1, tm + b * 128 + 64 + x * 8, b1 + x * (2048 >> 4), word_a, n > 0 || x > 0);
#pragma unroll
        for (int x = 0; x < kOther / 16; ++x)
          mma_ts(acc2, tm + b * 128 + x * 8, b2 + x * (2048 >> 4), word_a, n > 0 || x > 0);
        mma_commit(&sm.empty[slot]);
        if (n == steps - 1) mma_commit(&sm.acc_full);
      }
      __syncwarp();
      if (n + 2 < steps) ok = scores(n + 2);
    }
  } else if (warp == 10) {
    // ---- what belongs to the other side's rows
    if (sides) {
      for (int n = 0; n < steps; ++n) {
        const int slot = n % kSides;
        if (!warp_wait(&sm.side_empty[slot], ((n / kSides) & 1) ^ 1, given_up)) break;
        const int h = other_head(n), row0 = other_row(n);
        for (int x = lane; x < kOther; x += 32) {
          const bool in = row0 + x < other_rows;
          const long long row = (kDkv ? a.q0[f] : a.k0[f]) + row0 + x;
          if (kDkv) {
            sm.side[slot][0][x] = in ? fmaf(-kLog2e, a.lse[static_cast<long long>(h) * a.queries + row], kUp) : 0.0f;
            sm.side[slot][1][x] = in ? -a.delta[static_cast<long long>(h) * a.queries + row] : 0.0f;
          }
          for (int c = 0; c < a.axes; ++c)
            sm.side[slot][2 + c][x] =
                in ? static_cast<float>(kDkv ? a.qpos[row * a.qpos_stride + c] : a.kpos[row * a.kpos_stride + c]) : 0.0f;
        }
        bar_arrive(&sm.side_full[slot]);
      }
    }
  } else if (warp < 8) {
    // ---- probabilities and gradients: one own row a thread
    regs_up<kRegsMath>();
    const int wg = warp >> 2, r = threadIdx.x & (kOwn - 1);
    const int own = own0 + r;
    const bool live = own < own_rows;
    const long long own_row = (kDkv ? a.k0[f] : a.q0[f]) + own;
    const uint32_t mine = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    Row row{};
    if (a.slopes && live)
#pragma unroll
      for (int c = 0; c < 3; ++c)
        if (c < a.axes) row.pos[c] = -static_cast<float>(kDkv ? a.kpos[own_row * a.kpos_stride + c] : a.qpos[own_row * a.qpos_stride + c]);
    row.mul = (a.cap > 0.0f ? a.cap : a.scale) * kLog2e;
    row.cap_in = a.cap > 0.0f ? 2.0f * a.scale * kLog2e / a.cap : 0.0f;
    row.slope = a.slopes && !kDkv ? -a.slopes[own_head] * kLog2e / row.mul : 0.0f;
    float delta = 0.0f;
    if (!kDkv && live) {
      row.off = fmaf(-kLog2e, a.lse[static_cast<long long>(own_head) * a.queries + own_row], kUp);
      const char* o = a.o.data + own_row * a.o.row + own_head * a.o.head;
      const char* g = a.dout.data + own_row * a.dout.row + own_head * a.dout.head;
      for (int d = 0; d < a.D; d += 8) {
        float x[8], y[8];
        Pack<T>::load(o + d * 2, x);
        Pack<T>::load(g + d * 2, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) delta = fmaf(x[e], y[e], delta);
      }
      row.delta = -delta;
    }
    // A place is seen if its column is at least `from` and below `to`.
    int from = 0, to = other_rows;
    if (a.causal) {
      if (kDkv)
        from = own < a.prefix[f] ? 0 : own - shift;
      else
        to = live ? limit(own) : 0;
    }
    bool ok = true;
    for (int n = wg; n < steps; n += 2) {
      if (!(ok = warp_wait(&sm.sp_full[wg], (n >> 1) & 1, given_up))) break;
      const int slot = n % kSides;
      if (sides && !(ok = warp_wait(&sm.side_full[slot], (n / kSides) & 1, given_up))) break;
      if (kDkv && a.slopes) row.slope = -a.slopes[other_head(n)] * kLog2e / row.mul;
      tc_after();
      const int row0 = other_row(n);
      const float(*side)[kOther] = sm.side[slot];
      // Seen whole: nothing of the tile is hidden from any of the block's rows.
      const bool whole = row0 + kOther <= other_rows &&
                         (!a.causal || (kDkv ? limit(row0) >= min(own0 + kOwn, nk) : limit(own0) >= row0 + kOther));
      row.lo = from - row0;
      row.hi = to - row0;
      const uint32_t at = mine + wg * 128;
      if (a.cap > 0.0f) {
        if (whole)
          tile<T, kDkv, true, false>(at, side, a.axes, row);
        else
          tile<T, kDkv, true, true>(at, side, a.axes, row);
      } else {
        if (whole)
          tile<T, kDkv, false, false>(at, side, a.axes, row);
        else
          tile<T, kDkv, false, true>(at, side, a.axes, row);
      }
      if (sides) bar_arrive(&sm.side_empty[slot]);
      tc_wait_st();
      tc_before();
      bar_arrive(&sm.pd_full[wg]);
    }
    // ---- outputs
    const bool any = steps > 0;
    if (any && ok) ok = warp_wait(&sm.acc_full, 0, given_up);
    tc_after();
    // dq: the sum of P (dP - delta) is what delta is off by.
    if (!kDkv) {
      sm.rest[wg][r] = row.total;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      row.total = (sm.rest[0][r] + sm.rest[1][r]) * kDown;
      if (live && wg == 0) a.delta[static_cast<long long>(own_head) * a.queries + own_row] = delta + row.total;
    }
    const float bad = !ok || *given_up ? __int_as_float(0x7FFFFFFF) : 1.0f;  // a wait ran out: nothing here is an answer
    const View& out = kDkv ? (wg ? a.dv : a.dk) : a.dq;
    char* to_row = out.data + own_row * out.row + own_head * out.head;
    const float k1 = (kDkv && wg ? 1.0f : a.scale) * kDown * bad;
    const uint32_t acc = mine + 256 + (kDkv && wg ? 64 * kBlocks : 0);
    for (int x = kDkv ? 0 : wg * 16; x < a.Dn; x += kDkv ? 16 : 32) {
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
        if (!kDkv && any) w = fmaf(-row.total, __uint_as_float(d[y]), w);
        v[y] = w * k1;
      }
#pragma unroll
      for (int y = 0; y < 16; y += 8)
        if (live && x + y < a.D) Pack<T>::store(to_row + (x + y) * 2, v + y);
      __syncwarp();
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

template <typename T, int kBlocks, bool kDkv>
int launch_bwd(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s) {
  if (grid.x == 0) return PV_OK;
  auto kernel = pv_attn_bwd_kernel<T, kBlocks, kDkv>;
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
  return launch_pdl(kernel, grid, kThreads, smem, s, a, m.q, m.k, m.v, m.dout);
}

template <typename T, bool kDkv>
int side(const AttnArgs& a, const AttnMaps& m, dim3 grid, cudaStream_t s) {
  return a.D > 64 ? launch_bwd<T, 2, kDkv>(a, m, grid, s) : launch_bwd<T, 1, kDkv>(a, m, grid, s);
}

}  // namespace

int attn_backward_dq(const AttnArgs& a, int dtype, const AttnMaps& m, dim3 grid, cudaStream_t s) {
  return dtype == PV_BF16 ? side<__nv_bfloat16, false>(a, m, grid, s) : side<__half, false>(a, m, grid, s);
}

int attn_backward_dkv(const AttnArgs& a, int dtype, const AttnMaps& m, dim3 grid, cudaStream_t s) {
  return dtype == PV_BF16 ? side<__nv_bfloat16, true>(a, m, grid, s) : side<__half, true>(a, m, grid, s);
}

}  // namespace pvs
