// Linear attention with a decay for each head: whole frames in chunks, one token at a
// time, and the backward pass (pv_linear_attention, pv_linear_attention_step,
// pv_linear_attention_backward in pv.h).
//
//   S[t] = e^d S[t-1] + k[t] v[t]^T,  o[t] = scale q[t] S[t].
//
// In a chunk of 128 tokens, with i and s places in the order of reading and Z the state that
// the chunk begins with (already decayed for its first token):
//   o[i] = scale (sum_{s <= i} e^(d (i - s)) (q_i.k_s) v_s + e^(d i) q_i Z),
//   Z'   = e^(d n) Z + sum_s e^(d (n - s)) k_s v_s^T.
// One form does all passes.  It is run with (a, b, c) in the places of (q, k, v):
//   o  (q, k, v) forward;  dq (do, v, k) the same way, its state that of o transposed;
//   dk (v, do, q) and dv (k, q, do) the other way, their state the gradient of S.
//
// Three kernels (two where no frame is cut: the first one joins, too).  The first walks the chunks of a frame (or of a segment of it: frames are cut so that there are
// blocks for all multiprocessors) one after another, from b and c alone, and leaves the state that each
// chunk begins with, counted from the segment's beginning and rounded, and what the segment adds to the
// state, in 32 bits.  The second joins these to the state that each segment begins with, and to the last one.  In the
// third no chunk waits for another: both states, the chunk's own and the segment's, stand side by side under q.
//
// Precision: the scores (but in short frames) and the states are rounded to the storage type where the tensor
// cores take them, as attention's probabilities are.  What is added to the state is not: c times its
// decay is cut into three bfloat16 parts, 24 bits, so that states lose nothing from chunk to chunk (two
// parts, 16 bits, where no state leaves and all that is read of it is rounded to 8).
//
// A block takes one head and 64 columns of c: with heads of more than 64 both blocks of a head read all of a and b.
// (As a cluster, with loads for both, they wait for one another: 24,571 tokens of 128 took 89 us instead of 86.)
//
// What bounds it: products of 64 and 128 columns out of shared memory (50 + 0.48 N cycles for N columns, 128
// rows and 16 of the depth, whatever their order: some 1,300 to 2,600 cycles a chunk in each kernel), the
// chain product - decay - product - output beside them, and some 5 us at the beginning of each kernel.
// Measured: 8 ragged frames of up to 6,000 tokens, 8 heads of 64: 57 us (states 24, join 4, outputs 28); 24,571
// tokens, 8 heads of 128: 84 us (36, 5, 42); a training step on 4 frames of up to 4,000, 83.  One kernel that carries the state from
// chunk to chunk beside the outputs: 65, 83 and 91 us; it cannot cut the chains as finely, and is as quick only for the long frame.

#include "pv_attn.cuh"
#include "pv_tc.cuh"

#include <algorithm>
#include <cmath>
#include <initializer_list>

namespace {

using namespace pvs;
using T = __nv_bfloat16;

constexpr int kRows = 128;  // tokens of a chunk
constexpr int kCols = 64;   // columns of c, and of the state, that a block takes
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMostRuns = 3;

struct Run {
  int a, b, c;          // which of the tensor maps
  int a_head, b_head, c_head;  // 0: one head that every head reads
  int reverse;
  View out;
  float scale;          // of the output: on the scores and on the state's rows
  const float* in;      // [frames, H, D, D] or null
  float in_scale;
  int in_turned;        // the state is the transpose of what `in` holds
  int in_step;          // 1: `in` has still to be decayed for the first token
  float* end;           // the state after the last token, times end_scale, or null
  float end_scale;
  int end_step;         // 1: decayed once more
};

struct LinArgs {
  Run run[kMostRuns];
  const float* log_decay;
  float* segs;             // [run, segment, H, halves, 64 / 4, kD, 4]: what a segment adds to the state
  long long seg_run;       // floats of a run's segments
  unsigned char* states;   // [run, chunk, H, halves, kD, 64]: a chunk's state from its segment's beginning, rounded, swizzled
  long long state_run;     // bytes of a run's
  unsigned char* starts;   // [run, segment, H, halves, kD, 64]: the state that a segment begins with, likewise
  int frames, H, D, halves, chunk;  // chunk: chunks of a segment
  int whole;                        // every frame is one segment
  int off[PV_MAX_FRAMES + 1];
  int seg0[PV_MAX_FRAMES + 1];      // first segment of each frame
  int chunk0[PV_MAX_FRAMES + 1];    // first chunk
};

struct Maps {
  CUtensorMap m[4];
};

constexpr int kTile = kRows * 128;  // bytes of 128 rows of 64 elements

// e^(d x), d in units of log2: 1 for x = 0, whatever d is (a state that is not kept has d = -inf).
__device__ __forceinline__ float decay(float d, float x) { return exp2_fast(d * x); }
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// e^(d x) as the sum of two numbers, good to 2^-25.3 (q's three roundings; 2^-26 is the most that was seen.  A state goes
// through one a chunk, and an error of 2^-22 in each would add up).  y = d x = n ln 2 + r with r in two parts; e^r = 1 + r + q, q =
// r^2 / 2 + r^3 / 6 + ..., at most 0.071, by its series; the sum's rounding is kept.
__device__ __forceinline__ float2 decay_exact(float d, float x) {
  constexpr double kLn2 = 0.69314718055994530942;
  constexpr float kHigh = 0.693145751953125f, kLow = static_cast<float>(kLn2 - static_cast<double>(kHigh));  // 16 bits, the rest
  const float y = d * x, y_low = fmaf(d, x, -y);
  const float n = rintf(y * kLog2e);
  const float r0 = fmaf(n, -kHigh, y), r1 = fmaf(n, -kLow, y_low);  // (r0 is exact)
  const float r = r0 + r1, r_low = (r0 - r) + r1;
  float q = 1.0f / 40320.0f;
  q = fmaf(q, r, 1.0f / 5040.0f);
  q = fmaf(q, r, 1.0f / 720.0f);
  q = fmaf(q, r, 1.0f / 120.0f);
  q = fmaf(q, r, 1.0f / 24.0f);
  q = fmaf(q, r, 1.0f / 6.0f);
  q = fmaf(q, r, 0.5f);
  q = q * r * r;
  const float s = 1.0f + r, low = (r - (s - 1.0f)) + (q + r_low);
  if (y < -87.0f) return make_float2(0.0f, 0.0f);
  const float up = y > 88.0f ? INFINITY : __int_as_float((static_cast<int>(n) + 127) << 23);  // 2^n
  return make_float2(s * up, low * up);
}

__device__ __forceinline__ float decay_of(const float* log_decay, int h) { return max_nan(log_decay[h] * kLog2e, -1e4f); }

// bar_wait in as little code as it goes: with some twenty waits in the kernel their code is a
// part of what has to stay in the instruction cache.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* given_up) {
  unsigned long long until = 0;
#pragma unroll 1
  for (int i = 1; !bar_try(bar, parity); ++i) {
    if (i & 63) continue;
    if (*given_up) return false;
    const unsigned long long now = now_ns();
    if (!until) until = now + kBarLimitNs;
    if (now > until) {
      *given_up = 1;
      return false;
    }
  }
  return true;
}
// (A warp whose wait has run out neither writes what others read nor arrives for them: several warps' arrivals end a
// barrier's phase, and those who still read would find another chunk's numbers in the place of their own.)
__device__ __forceinline__ bool warp_wait_for(uint64_t* bar, uint32_t parity, volatile int* given_up) {
  return __all_sync(0xFFFFFFFFu, wait_for(bar, parity, given_up));
}

// Tokens of a frame of n that come before the k-th of its chunks in the order of reading.
__device__ __forceinline__ int before(int k, int n, int chunks, bool reverse) {
  return !reverse ? min(k * kRows, n) : k == 0 ? 0 : n - (chunks - k) * kRows;
}

// What a block works on: a segment of a frame, a head, a half of c's columns.
struct Place {
  int f, seg, here, h, half, rest, n, chunks, k0, count;
  bool last, reverse;
  // Row of the frame at which the i-th chunk of the segment begins, and its rows.
  __device__ __forceinline__ int row_of(int i) const { return (reverse ? chunks - 1 - k0 - i : k0 + i) * kRows; }
  __device__ __forceinline__ int len_of(int i) const { return min(kRows, n - row_of(i)); }
  // Tokens of the frame before the i-th chunk of the segment.
  __device__ __forceinline__ int past(int i) const { return before(k0 + i, n, chunks, reverse); }
};
__device__ __forceinline__ Place place_of(const LinArgs& a, const Run& run) {
  Place p;
  const int per = a.H * a.halves;
  p.seg = blockIdx.x / per;
  p.f = frame_of(a.seg0, a.frames, p.seg);
  p.rest = blockIdx.x - p.seg * per;
  p.h = p.rest / a.halves;
  p.half = p.rest - p.h * a.halves;
  p.n = a.off[p.f + 1] - a.off[p.f];
  p.chunks = (p.n + kRows - 1) / kRows;
  p.here = p.seg - a.seg0[p.f];
  p.k0 = p.here * a.chunk;
  p.count = min(a.chunk, p.chunks - p.k0);
  p.last = p.k0 + p.count == p.chunks;
  p.reverse = run.reverse != 0;
  return p;
}
// The i-th chunk's state, of kD rows of 128 bytes.
template <int kBlocks>
__device__ __forceinline__ unsigned char* state_of(const LinArgs& a, const Place& p, int i) {
  return a.states + blockIdx.y * a.state_run +
         (static_cast<long long>(a.chunk0[p.f] + p.k0 + i) * a.H * a.halves + p.rest) * (kBlocks * kTile / 2);
}

// ------------------------------------------------------------ segments

// Takes four columns of a row of a frame's and head's state (i: which of them) through the frame's segments.
template <int kBlocks>
__device__ __forceinline__ void join_segments(const LinArgs& a, const Run& run, int f, int rest, int i) {
  constexpr int kD = 64 * kBlocks, kBlock = kD * kCols, kAhead = 8;
  const int heads = a.H * a.halves, h = rest / a.halves;
  const int own = i % kD, j = i / kD * 4;  // row; columns j .. j + 3
  const int n = a.off[f + 1] - a.off[f], chunks = (n + kRows - 1) / kRows, s0 = a.seg0[f], segments = a.seg0[f + 1] - s0;
  const bool reverse = run.reverse != 0;
  const float ld = max_nan(a.log_decay[h], -1e4f);
  const int column = (rest - h * a.halves) * kCols + j;
  const bool there = own < a.D && column < a.D;
  const long long state = (static_cast<long long>(f) * a.H + h) * a.D * a.D;
  float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (run.in && there) {
    if (run.in_turned) {
      const float* in = run.in + state + static_cast<long long>(column) * a.D + own;
      z = make_float4(in[0], in[a.D], in[2 * a.D], in[3 * a.D]);
    } else {
      z = *reinterpret_cast<const float4*>(run.in + state + static_cast<long long>(own) * a.D + column);
    }
    // (An empty frame's state leaves as it came.)
    const float2 w = decay_exact(ld, static_cast<float>(run.in_step));
    const float by = n == 0 ? 1.0f : run.in_scale * (w.x + w.y);
    z = make_float4(z.x * by, z.y * by, z.z * by, z.w * by);
  }
  const float* const segs = a.segs + blockIdx.y * a.seg_run + (static_cast<long long>(s0) * heads + rest) * kBlock + own * 4 + j * kD;
  unsigned char* const starts = a.starts + 2 * (blockIdx.y * a.seg_run + (static_cast<long long>(s0) * heads + rest) * kBlock) + own * 128 +
                                (((j >> 3) ^ (own & 7)) << 4) + (j & 4) * 2;
  const long long step = static_cast<long long>(heads) * kBlock;
  const int sums = segments - (run.end && n ? 0 : 1);  // segments that add to something
  for (int s = 0; s < segments; s += kAhead) {
    float4 v[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x)
      if (s + x < sums) v[x] = *reinterpret_cast<const float4*>(segs + (s + x) * step);
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      if (s + x >= segments) break;
      *reinterpret_cast<uint2*>(starts + 2 * (s + x) * step) = make_uint2(Pack<T>::two(z.x, z.y), Pack<T>::two(z.z, z.w));
      if (s + x >= sums) break;
      const bool end = s + x + 1 == segments;
      const int tokens = before(min((s + x + 1) * a.chunk, chunks), n, chunks, reverse) - before((s + x) * a.chunk, n, chunks, reverse);
      const float2 w = decay_exact(ld, static_cast<float>(tokens - (end && !run.end_step ? 1 : 0)));
      z.x = fmaf(z.x, w.x, fmaf(z.x, w.y, v[x].x)), z.y = fmaf(z.y, w.x, fmaf(z.y, w.y, v[x].y));
      z.z = fmaf(z.z, w.x, fmaf(z.z, w.y, v[x].z)), z.w = fmaf(z.w, w.x, fmaf(z.w, w.y, v[x].w));
    }
  }
  if (run.end && there) {
    const float by = n == 0 ? 1.0f : run.end_scale;
    *reinterpret_cast<float4*>(run.end + state + static_cast<long long>(own) * a.D + column) = make_float4(z.x * by, z.y * by, z.z * by, z.w * by);
  }
}

template <int kBlocks>
__global__ void __launch_bounds__(256) pv_linear_join_kernel(const __grid_constant__ LinArgs a) {
  constexpr int kEach = 64 * kBlocks * kCols / 4 / 256;  // blocks of a frame's head
  wait_prior_grid();
  const int who = blockIdx.x / kEach, f = who / (a.H * a.halves);
  join_segments<kBlocks>(a, a.run[blockIdx.y], f, who - f * a.H * a.halves, (blockIdx.x - who * kEach) * 256 + threadIdx.x);
  allow_next_grid();
}

// ------------------------------------------------------------ states

// Warps 0-3 hold the state in registers (a row and 64 columns a thread), 4-19 put the decay on c,
// 20 issues the products, 21 loads.
constexpr int kStateThreads = 768;
// Registers of a thread: 80 at launch (768 x 80 = 61,440); what the helpers give back goes to
// the state's warps (128 + 4 x 64 + 56 = 440 a thread of each warpgroup, of 480).
constexpr int kRegsState = 128, kRegsParts = 64, kRegsIssue = 56;

template <int kBlocks>
struct StateSmem {
  static constexpr int kStages = kBlocks == 1 ? 3 : 2;
  alignas(1024) unsigned char bc[kStages][(kBlocks + 1) * kTile];
  alignas(1024) unsigned char parts[2][3][kTile];  // c, decayed to the chunk's end, in parts
  // (The warps that fill `parts` are up to two chunks ahead: barriers of two places have a phase each.)
  uint64_t full[kStages], empty[kStages], part_ready[2], d_full[2], d_free[2];
  uint32_t tmem;
  int given_up;
};

template <int kBlocks>
__global__ void __launch_bounds__(kStateThreads, 1)
    pv_linear_states_kernel(const __grid_constant__ LinArgs a, const __grid_constant__ Maps maps) {
  using S = StateSmem<kBlocks>;
  constexpr int kD = 64 * kBlocks;
  extern __shared__ __align__(1024) unsigned char raw[];
  S& sm = *reinterpret_cast<S*>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Run& run = a.run[blockIdx.y];
  const Place at = place_of(a, run);
  // Chunks whose sum is needed: the last one's is where another segment or the caller asks for it.
  const bool to_end = at.last && run.end;
  const int sums = at.count - (at.last && !run.end ? 1 : 0), parts = run.end ? 3 : 2;
  if (at.count <= 0) {
    wait_prior_grid();
    if (a.whole)
      for (int i = threadIdx.x; i < kD * kCols / 4; i += kStateThreads) join_segments<kBlocks>(a, run, at.f, at.rest, i);
    allow_next_grid();
    return;
  }
  if (threadIdx.x == 0) {
    sm.given_up = 0;
    for (int i = 0; i < S::kStages; ++i) bar_init(&sm.full[i], 1), bar_init(&sm.empty[i], 1);
    for (int i = 0; i < 2; ++i) bar_init(&sm.part_ready[i], 16), bar_init(&sm.d_full[i], 1), bar_init(&sm.d_free[i], 4);
    fence_bar_init();
  }
  if (warp == 20) tmem_alloc<256>(&sm.tmem);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = sm.tmem;
  volatile int* given_up = &sm.given_up;
  wait_prior_grid();
  bool ok = true;

  if (warp >= 20) {
    regs_down<kRegsIssue>();
    if (warp == 21 && lane == 0) {
      int slot = 0, parity = 1, i = 0;
      for (; i < sums; ++i) {
        if (!wait_for(&sm.empty[slot], parity, given_up)) break;
        const int row = a.off[at.f] + at.row_of(i);
        bar_expect(&sm.full[slot], (kBlocks + 1) * kTile);
        for (int b = 0; b < kBlocks; ++b)
          tma_load4(sm.bc[slot] + b * kTile, &maps.m[run.b], b * 64, 0, run.b_head ? at.h : 0, row, &sm.full[slot]);
        tma_load4(sm.bc[slot] + kBlocks * kTile, &maps.m[run.c], at.half * 64, 0, run.c_head ? at.h : 0, row, &sm.full[slot]);
        if (++slot == S::kStages) slot = 0, parity ^= 1;
      }
      bars_drain(sm.full, S::kStages, i);
    }
    if (warp == 20 && elect_one()) {
      // Sums over tokens: b's rows lie along the depth.  (With heads of up to 64, b's second block of
      // 64 is c: what comes of it is not looked at.)
      const uint32_t word_d = mma_word(true, 128, kCols, true, true), word_dd = mma_word(true, 128, 2 * kCols, true, true);
      const uint32_t b_op = operand(smem_addr(sm.bc[0]), kTile), part_op = operand(smem_addr(sm.parts[0][0]), kTile);
      int slot = 0;
      // (Who puts c in parts has waited for its load, and b's.)
      for (int i = 0; i < sums; ++i) {
        const int buf = i & 1;
        if (!wait_for(&sm.part_ready[buf], (i >> 1) & 1, given_up) || !wait_for(&sm.d_free[buf], ((i >> 1) & 1) ^ 1, given_up)) break;
        tc_after();
        const uint32_t to = tm + 128 * buf, from = part_op + buf * (3 * kTile >> 4), b = b_op + slot * (sizeof(sm.bc[0]) >> 4);
        // Two parts side by side (a product of 128 columns takes 111 cycles, one of 64 80).
#pragma unroll
        for (int x = 0; x < kRows / 16; ++x) mma_ss(to, b + x * (2048 >> 4), from + x * (2048 >> 4), word_dd, x > 0);
        if (parts == 3) {
#pragma unroll
          for (int x = 0; x < kRows / 16; ++x) mma_ss(to, b + x * (2048 >> 4), from + (2 * kTile >> 4) + x * (2048 >> 4), word_d, true);
        }
        mma_commit(&sm.d_full[buf]);
        mma_commit(&sm.empty[slot]);
        if (++slot == S::kStages) slot = 0;
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---- c, decayed to the chunk's end, in parts
    regs_down<kRegsParts>();
    const float d = decay_of(a.log_decay, at.h);
    const int t = threadIdx.x - 128;  // 0 .. 511
    int slot = 0, parity = 0;
    for (int i = 0; i < sums; ++i) {
      const int len = at.len_of(i), buf = i & 1;
      const int step = to_end && i + 1 == at.count && !run.end_step ? 1 : 0;  // steps short of the next token
      ok = ok && warp_wait_for(&sm.full[slot], parity, given_up);
      if (i > 1) ok = ok && warp_wait_for(&sm.d_full[buf], ((i >> 1) - 1) & 1, given_up);
      if (!ok) break;
      unsigned char* const c = sm.bc[slot] + kBlocks * kTile;
#pragma unroll
      for (int x = 0; x < kRows; x += 64) {
        const int row = x + (t >> 3), spot = row * 128 + (t & 7) * 16;
        // (The swizzle moves the pieces of a row about, of c and of its parts alike.)
        float v[8];
        Pack<T>::load(c + spot, v);
        const float w = row < len ? decay(d, static_cast<float>(at.reverse ? row + 1 - step : len - step - row)) : 0.0f;
        uint32_t p[3][4];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          float r0, r1;
          mul2(r0, r1, v[j], v[j + 1], w, w);
          if (row >= len) r0 = r1 = 0.0f;
#pragma unroll
          for (int z = 0; z < 3; ++z) {
            const uint32_t b = Pack<T>::two(r0, r1);
            p[z][j / 2] = b;
            if (z < 2) fma2(r0, r1, __uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u), -1.0f, -1.0f, r0, r1);
          }
        }
#pragma unroll
        for (int z = 0; z < 3; ++z)
          if (z < 2 || parts == 3) *reinterpret_cast<uint4*>(sm.parts[buf][z] + spot) = make_uint4(p[z][0], p[z][1], p[z][2], p[z][3]);
      }
      if (len < kRows) {
        // Rows past the frame's end are another frame's: whatever they hold must not meet the zeros
        // of these places.  (c's own, too: it stands in for a second block of b.)
        for (int y = len * 8 + t; y < kRows * 8; y += 512)
#pragma unroll
          for (int x = 0; x <= kBlocks; ++x) *reinterpret_cast<uint4*>(sm.bc[slot] + x * kTile + y * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_to_async();
      warp_arrive(&sm.part_ready[buf]);
      if (++slot == S::kStages) slot = 0, parity ^= 1;
    }
  } else {
    // ---- the state: row `own` of it, 64 columns
    regs_up<kRegsState>();
    const float ld = max_nan(a.log_decay[at.h], -1e4f);
    const int own = warp * 32 + lane;
    float z[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) z[j] = 0.0f;
    // Of a frame that is not cut: eight columns, from 8 j, of the state that it begins with.
    const float2 w0 = decay_exact(ld, static_cast<float>(run.in_step));
    const float by0 = run.in_scale * (w0.x + w0.y);
    const long long given = (static_cast<long long>(at.f) * a.H + at.h) * a.D * a.D;
    auto initial = [&](int j, float* v) {
      const int column = at.half * kCols + 8 * j;
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = 0.0f;
      if (!run.in || own >= a.D || column >= a.D) return;
      const float* in = run.in + given + (run.in_turned ? static_cast<long long>(column) * a.D + own : static_cast<long long>(own) * a.D + column);
      const int step = run.in_turned ? a.D : 1;
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = in[x * step] * by0;
    };
    if (a.whole && warp * 32 < kD) {
      unsigned char* const to = a.starts + 2 * (blockIdx.y * a.seg_run + (static_cast<long long>(at.seg) * a.H * a.halves + at.rest) * (kD * kCols)) + own * 128;
#pragma unroll 4
      for (int j = 0; j < 8; ++j) {
        float v[8];
        initial(j, v);
        Pack<T>::store(to + ((j ^ (own & 7)) << 4), v);
      }
    }
    const float2 whole = decay_exact(ld, static_cast<float>(kRows));
    for (int i = 0; i < at.count; ++i) {
      if (warp * 32 < kD) {
        unsigned char* const to = state_of<kBlocks>(a, at, i) + own * 128;
#pragma unroll
        for (int j = 0; j < 8; ++j) Pack<T>::store(to + ((j ^ (own & 7)) << 4), z + 8 * j);
      }
      if (i >= sums) break;
      const int steps = at.len_of(i) - (to_end && i + 1 == at.count && !run.end_step ? 1 : 0);
      const float2 by = steps == kRows ? whole : decay_exact(ld, static_cast<float>(steps));
      ok = ok && warp_wait_for(&sm.d_full[i & 1], (i >> 1) & 1, given_up);
      tc_after();
      if (warp * 32 < kD) {
        const uint32_t from = tm + (static_cast<uint32_t>(warp * 32) << 16) + 128 * (i & 1);
        // The second block, the smaller parts, joins the smaller part of the decayed state.
#pragma unroll
        for (int j = 0; j < kCols; j += 16) {
          float u[16], v[16];
          tmem_read2x16(from + j, from + kCols + j, v, u);
#pragma unroll
          for (int x = 0; x < 16; x += 2) {
            fma2(u[x], u[x + 1], z[j + x], z[j + x + 1], by.y, by.y, u[x], u[x + 1]);
            add2(v[x], v[x + 1], v[x], v[x + 1], u[x], u[x + 1]);
            fma2(z[j + x], z[j + x + 1], z[j + x], z[j + x + 1], by.x, by.x, v[x], v[x + 1]);
          }
        }
        if (!ok) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) z[j] = NAN;
        }
      }
      tc_before();
      if (ok) warp_arrive(&sm.d_free[i & 1]);
    }
    if (a.whole && to_end && own < a.D) {
      const float2 w = decay_exact(ld, static_cast<float>(at.n - (run.end_step ? 0 : 1)));
      float* const to = run.end + given + static_cast<long long>(own) * a.D + at.half * kCols;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (at.half * kCols + 8 * j >= a.D) continue;
        float v[8];
        initial(j, v);
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = fmaf(v[x], w.x, fmaf(v[x], w.y, z[8 * j + x])) * run.end_scale;
        *reinterpret_cast<float4*>(to + 8 * j) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(to + 8 * j + 4) = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
    if (!a.whole && sums == at.count && warp * 32 < kD) {
      float* to = a.segs + blockIdx.y * a.seg_run + (static_cast<long long>(at.seg) * a.H * a.halves + at.rest) * (kD * kCols) + own * 4;
#pragma unroll
      for (int j = 0; j < kCols; j += 4) *reinterpret_cast<float4*>(to + j * kD) = make_float4(z[j], z[j + 1], z[j + 2], z[j + 3]);
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  allow_next_grid();
  if (warp == 20) tmem_free<256>(tm);
}

// ------------------------------------------------------------ outputs

// Warps 0-3 and 4-7 put the decay on the scores of every other chunk and hand them over in tensor
// memory, 8-11 and 12-15 write the output, a half of the columns each, 16 issues the products, 17 loads.
constexpr int kOutThreads = 576;

template <int kBlocks>
struct OutSmem {
  static constexpr int kStages = kBlocks == 1 ? 3 : 2;
  static constexpr int kState = kBlocks * kTile / 2;          // [64 kBlocks][64]
  static constexpr int kAB = 2 * kBlocks * kTile;             // then the chunk's state, then c
  alignas(1024) unsigned char in[kStages][kAB + kState + kTile];
  alignas(1024) unsigned char state[kState];                  // the segment's
  uint64_t ab_full[kStages], ab_empty[kStages], c_full[kStages], c_empty[kStages], p_full[2], p_ready[2], s_full, o_full, o_free;
  alignas(16) float powers[2][32];  // the decay of 31 .. 0 tokens, and of 0 .. 31
  uint32_t tmem;
  int given_up;
};

// Columns of tensor memory: two buffers of scores, the output's terms (scores; the chunk's state, the segment's).
constexpr int kP = 0, kO = 256, kZ = 320;

// Scores are taken in two bfloat16 parts in frames of one chunk.  There few terms make a row, and one's
// rounding shows (a single token's output is one score times v); in longer frames two parts turn 1.41 times the output's own
// rounding into 1.2 and take 8 ragged frames of up to 6,000 from 58 to 63 us.  It goes by the frame, so that what a
// frame gives does not depend on the frames beside it; calls whose frames are all alike have a kernel without the question
// (asked in every block, the same 8 frames take 60 us).
enum Scores { kOnePart, kTwoParts, kByFrame };

template <int kBlocks, int kScores>
__global__ void __launch_bounds__(kOutThreads, 1)
    pv_linear_out_kernel(const __grid_constant__ LinArgs a, const __grid_constant__ Maps maps) {
  using S = OutSmem<kBlocks>;
  constexpr int kD = 64 * kBlocks;
  constexpr int kC = S::kAB + S::kState;
  extern __shared__ __align__(1024) unsigned char raw[];
  S& sm = *reinterpret_cast<S*>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Run& run = a.run[blockIdx.y];
  const Place at = place_of(a, run);
  const int count = at.count;
  const bool two = kScores == kTwoParts || (kScores == kByFrame && at.chunks == 1);
  // From the segment's last chunk to its first: what the states' kernel read and wrote last is still in the L2 cache
  // (24,571 tokens, 8 heads of 128: 86 us from the first to the last, 84 like this).
  auto nth = [&](int i) { return count - 1 - i; };
  if (threadIdx.x == 0) {
    sm.given_up = 0;
    for (int i = 0; i < S::kStages; ++i)
      bar_init(&sm.ab_full[i], 1), bar_init(&sm.ab_empty[i], 1), bar_init(&sm.c_full[i], 1), bar_init(&sm.c_empty[i], 1);
    for (int i = 0; i < 2; ++i) bar_init(&sm.p_full[i], 1), bar_init(&sm.p_ready[i], 4);
    bar_init(&sm.s_full, 1), bar_init(&sm.o_full, 1), bar_init(&sm.o_free, 8);
    fence_bar_init();
  }
  if (warp == 16) tmem_alloc<512>(&sm.tmem);
  wait_prior_grid();
  const float d = decay_of(a.log_decay, at.h);
  if (threadIdx.x < 64) sm.powers[threadIdx.x >> 5][lane] = decay(d, static_cast<float>(threadIdx.x < 32 ? 31 - lane : lane));
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = sm.tmem;
  volatile int* given_up = &sm.given_up;
  bool ok = true;

  if (warp == 17) {
    // ---- loads
    if (lane == 0) {
      int slot = 0, parity = 1, ab = 0, c = 0;
      if (count > 0) {
        bar_expect(&sm.s_full, S::kState);
        tma_copy(sm.state, a.starts + 2 * (blockIdx.y * a.seg_run + (static_cast<long long>(at.seg) * a.H * a.halves + at.rest) * (kD * kCols)),
                 S::kState, &sm.s_full);
      }
      for (int i = 0; i < count; ++i) {
        unsigned char* const to = sm.in[slot];
        const int row = a.off[at.f] + at.row_of(nth(i));
        if (!wait_for(&sm.ab_empty[slot], parity, given_up)) break;
        bar_expect(&sm.ab_full[slot], S::kAB + S::kState);
        ++ab;
        for (int b = 0; b < kBlocks; ++b) {
          tma_load4(to + b * kTile, &maps.m[run.a], b * 64, 0, run.a_head ? at.h : 0, row, &sm.ab_full[slot]);
          tma_load4(to + (kBlocks + b) * kTile, &maps.m[run.b], b * 64, 0, run.b_head ? at.h : 0, row, &sm.ab_full[slot]);
        }
        tma_copy(to + S::kAB, state_of<kBlocks>(a, at, nth(i)), S::kState, &sm.ab_full[slot]);
        if (!wait_for(&sm.c_empty[slot], parity, given_up)) break;
        bar_expect(&sm.c_full[slot], kTile);
        ++c;
        tma_load4(to + kC, &maps.m[run.c], at.half * 64, 0, run.c_head ? at.h : 0, row, &sm.c_full[slot]);
        if (++slot == S::kStages) slot = 0, parity ^= 1;
      }
      bars_drain(&sm.s_full, 1, count > 0);
      bars_drain(sm.ab_full, S::kStages, ab);
      bars_drain(sm.c_full, S::kStages, c);
    }
    __syncwarp();
  } else if (warp == 16) {
    // ---- products
    if (elect_one()) {
      const uint32_t word_p = mma_word(true, 128, 128, false, false), word_z = mma_word(true, 128, 2 * kCols, false, true);
      const uint32_t word_o = mma_word(true, 128, kCols, false, true);
      constexpr uint32_t kStep = sizeof(sm.in[0]) >> 4;
      const uint32_t base = smem_addr(sm.in[0]);
      const uint32_t a_op = operand(base, 16), b_op = operand(base + kBlocks * kTile, 16), c_op = operand(base + kC, kTile);
      // Scores go ahead, so that their decay is put on beside other chunks' products: two chunks where there
      // are three stages (into the buffer that the last product has just been done with), one
      // where there are two.  (Every product stands in the code once: this warp's code is walked through
      // once a chunk, and what all roles walk through has to stay in the instruction cache.)
      constexpr int kAhead = S::kStages - 1;
      int slot = 0, parity = 0, next = 0;
      auto scores = [&](int i) {
        if (!wait_for(&sm.ab_full[next], parity, given_up)) return false;
        tc_after();
        const uint32_t to = tm + kP + (i & 1) * 128, from = next * kStep;
#pragma unroll
        for (int x = 0; x < 4 * kBlocks; ++x) {
          const uint32_t off = from + (((x >> 2) * kTile + (x & 3) * 32) >> 4);
          mma_ss(to, a_op + off, b_op + off, word_p, x > 0);
        }
        mma_commit(&sm.p_full[i & 1]);
        if (++next == S::kStages) next = 0, parity ^= 1;
        return true;
      };
      for (int i = -kAhead; ok && i < count; ++i) {
        if (i >= 0) {  // both states under q: the chunk's own and, 64 columns further, the segment's
          if (!(ok = (i > 0 || wait_for(&sm.s_full, 0, given_up)) && wait_for(&sm.o_free, (i & 1) ^ 1, given_up))) break;
          tc_after();
          const uint32_t own = base + slot * sizeof(sm.in[0]) + S::kAB;
          const uint32_t from = a_op + slot * kStep, z = operand(own, smem_addr(sm.state) - own);
#pragma unroll
          for (int x = 0; x < 4 * kBlocks; ++x)
            mma_ss(tm + kZ, from + (((x >> 2) * kTile + (x & 3) * 32) >> 4), z + x * (2048 >> 4), word_z, x > 0);
          mma_commit(&sm.ab_empty[slot]);
        }
        if (kAhead == 1 && i + 1 < count && !(ok = scores(i + 1))) break;
        if (i >= 0) {  // scores times c (which those who hand them over have waited for)
          if (!(ok = wait_for(&sm.p_ready[i & 1], (i >> 1) & 1, given_up))) break;
          tc_after();
          const uint32_t p = tm + kP + (i & 1) * 128, c = c_op + slot * kStep;
#pragma unroll
          for (int x = 0; x < kRows / 16; ++x) {
            const uint32_t at_p = p + (x >> 1) * 32 + (x & 1) * 8, at_c = c + x * (2048 >> 4);
            mma_ts(tm + kO, at_p, at_c, word_o, x > 0);
            if (two) mma_ts(tm + kO, at_p + 16, at_c, word_o, true);
          }
          mma_commit(&sm.o_full);
          mma_commit(&sm.c_empty[slot]);
          if (++slot == S::kStages) slot = 0;
        }
        if (kAhead == 2 && i + 2 < count && !(ok = scores(i + 2))) break;
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---- scores of every other chunk: a row a thread, the decay of the distance put on
    const int diagonal = warp & 3, row = diagonal * 32 + lane, turn = warp >> 2;
    const uint32_t own = tm + (static_cast<uint32_t>(diagonal * 32) << 16) + kP + turn * 128;
    for (int i = turn; i < count; i += 2) {
      const int len = at.len_of(nth(i)), slot = i % S::kStages;
      ok = ok && warp_wait_for(&sm.p_full[turn], (i >> 1) & 1, given_up);
      if (!ok) break;
      tc_after();
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        // (Where the block's 32 scores were: what they are rounded to and, if it is taken, what that leaves.)
        uint32_t out[kScores == kOnePart ? 16 : 32];
        float v[32];
        if (at.reverse ? j < diagonal : j > diagonal) {
#pragma unroll
          for (int x = 0; x < 16; ++x) out[x] = 0, v[2 * x] = v[2 * x + 1] = 0.0f;
        } else {
          tmem_read32(own + 32 * j, v);
          if (j != diagonal && 32 * j + 32 <= len) {
            // Away from the diagonal a distance is the row's from the block's near edge and the
            // column's to it, and so the decay a product (no exponential for each score: 16
            // a cycle would be what these warps wait for).
            const float by = run.scale * decay(d, static_cast<float>(at.reverse ? 32 * j - row : row - 32 * j - 31));
            const float* const powers = sm.powers[at.reverse];
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              float4 w = *reinterpret_cast<const float4*>(powers + x);
              mul2(w.x, w.y, w.x, w.y, by, by);
              mul2(w.z, w.w, w.z, w.w, by, by);
              mul2(v[x], v[x + 1], v[x], v[x + 1], w.x, w.y);
              mul2(v[x + 2], v[x + 3], v[x + 2], v[x + 3], w.z, w.w);
              out[x / 2] = Pack<T>::two(v[x], v[x + 1]);
              out[x / 2 + 1] = Pack<T>::two(v[x + 2], v[x + 3]);
            }
          } else {
            const float gap = static_cast<float>(at.reverse ? 32 * j - row : row - 32 * j), sign = at.reverse ? 1.0f : -1.0f;
            const int left = len - 32 * j;
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              float g0, g1;
              fma2(g0, g1, sign, sign, static_cast<float>(x), static_cast<float>(x + 1), gap, gap);
              float e0, e1;
              mul2(e0, e1, g0, g1, d, d);
              mul2(v[x], v[x + 1], v[x], v[x + 1], run.scale, run.scale);
              mul2(v[x], v[x + 1], v[x], v[x + 1], exp2_fast(e0), exp2_fast(e1));
              if (g0 < 0.0f || x >= left) v[x] = 0.0f;
              if (g1 < 0.0f || x + 1 >= left) v[x + 1] = 0.0f;
              out[x / 2] = Pack<T>::two(v[x], v[x + 1]);
            }
          }
        }
        if constexpr (kScores != kOnePart) {
          if (two) {
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float r0 = __uint_as_float(out[x] << 16), r1 = __uint_as_float(out[x] & 0xFFFF0000u);
              out[16 + x] = Pack<T>::two(v[2 * x] - r0, v[2 * x + 1] - r1);
            }
            tmem_st32(own + 32 * j, out);
          }
        }
        if (!two) tmem_st16(own + 32 * j, out);
      }
      tc_wait_st();
      ok = ok && warp_wait_for(&sm.c_full[slot], (i / S::kStages) & 1, given_up);
      if (!ok) break;
      if (len < kRows) {
        // Rows past the frame's end are another frame's: whatever they hold must not meet the zeros
        // of these places.
        for (int y = len * 8 + diagonal * 32 + lane; y < kRows * 8; y += 128)
          *reinterpret_cast<uint4*>(sm.in[slot] + kC + y * 16) = make_uint4(0, 0, 0, 0);
        fence_to_async();
      }
      tc_before();
      warp_arrive(&sm.p_ready[turn]);
    }
  } else {
    // ---- output: a row and a half of the columns a thread
    const int own = (warp & 3) * 32 + lane;
    const int first = (warp >> 2 & 1) * (kCols / 2);
    const uint32_t mine = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16) + first;
    for (int i = 0; i < count; ++i) {
      const int len = at.len_of(nth(i));
      ok = ok && warp_wait_for(&sm.o_full, i & 1, given_up);
      tc_after();
      const float by = run.scale * decay(d, static_cast<float>(max(0, at.reverse ? len - 1 - own : own)));
      const float far = by * decay(d, static_cast<float>(at.past(nth(i)) - at.past(0)));
      uint4 out[kCols / 16];
#pragma unroll
      for (int j = 0; j < kCols / 2; j += 16) {
        float o[16], u[16], v[16];
        tmem_read3x16(mine + kO + j, mine + kZ + j, mine + kZ + kCols + j, o, u, v);
        if (j + 16 == kCols / 2) {
          tc_before();
          if (ok) warp_arrive(&sm.o_free);
        }
#pragma unroll
        for (int x = 0; x < 16; x += 2) {
          fma2(o[x], o[x + 1], u[x], u[x + 1], by, by, o[x], o[x + 1]);
          fma2(o[x], o[x + 1], v[x], v[x + 1], far, far, o[x], o[x + 1]);
          if (!ok) o[x] = o[x + 1] = NAN;
        }
        Pack<T>::store(out + j / 8, o);
        Pack<T>::store(out + j / 8 + 1, o + 8);
      }
      if (own < len) {
        const int c0 = at.half * kCols + first;
        char* const to = run.out.data + (static_cast<long long>(a.off[at.f]) + at.row_of(nth(i)) + own) * run.out.row + at.h * run.out.head + c0 * 2;
#pragma unroll
        for (int j = 0; j < kCols / 2; j += 8)
          if (c0 + j < a.D) *reinterpret_cast<uint4*>(to + 2 * j) = out[j / 8];
      }
      __syncwarp();
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  allow_next_grid();
  if (warp == 16) tmem_free<512>(tm);
}

// ------------------------------------------------------------ one token

struct StepArgs {
  View q, k, v, out;
  const float* log_decay;
  const float* state;
  float* next;
  int H, D;
  float scale;
};

// A block takes one stream's head; its state is read and written once, which bounds it: D / 4 lanes of
// a warp's worth of float4 hold a row of it, the rows dealt over the block.  32 streams of 8 heads of 128: 12.5 us with
// the states in DRAM, less than the host's part of the call.
template <typename U>
__global__ void __launch_bounds__(256) pv_linear_step_kernel(const __grid_constant__ StepArgs a) {
  __shared__ alignas(16) float q[128], k[128], v[128];  // (v is read in fours)
  __shared__ float4 sums[256];
  wait_prior_grid();
  const int i = blockIdx.x / a.H, h = blockIdx.x - i * a.H, D = a.D;
  const float* from = a.state + static_cast<long long>(blockIdx.x) * D * D;
  float* to = a.next + static_cast<long long>(blockIdx.x) * D * D;
  const int quads = D >> 2, rows = 256 / quads, c = threadIdx.x % quads, r = threadIdx.x / quads;
  // The first rows are under way while the token's vectors come in.
  constexpr int kAhead = 8;
  float4 s[kAhead];
  const bool on = r < rows;
#pragma unroll
  for (int x = 0; x < kAhead; ++x)
    if (on && r + x * rows < D) s[x] = *reinterpret_cast<const float4*>(from + (r + x * rows) * D + 4 * c);
  if (threadIdx.x < D) {
    const long long e = threadIdx.x * sizeof(U);
    auto get = [&](const View& t) {
      return Pack<U>::to(*reinterpret_cast<const U*>(t.data + static_cast<long long>(i) * t.row + h * t.head + e));
    };
    q[threadIdx.x] = get(a.q);
    k[threadIdx.x] = get(a.k);
    v[threadIdx.x] = get(a.v);
  }
  const float by = expf(a.log_decay[h]);
  __syncthreads();
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (on) {
    const float4 w = *reinterpret_cast<const float4*>(v + 4 * c);
    for (int x0 = 0; x0 * rows < D; x0 += kAhead) {
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int row = r + (x0 + x) * rows;
        if (row >= D) continue;
        float4 z = s[x];
        const int further = row + kAhead * rows;
        if (further < D) s[x] = *reinterpret_cast<const float4*>(from + further * D + 4 * c);
        const float b = k[row], y = q[row];
        z.x = fmaf(z.x, by, b * w.x), z.y = fmaf(z.y, by, b * w.y), z.z = fmaf(z.z, by, b * w.z), z.w = fmaf(z.w, by, b * w.w);
        *reinterpret_cast<float4*>(to + row * D + 4 * c) = z;
        o.x = fmaf(y, z.x, o.x), o.y = fmaf(y, z.y, o.y), o.z = fmaf(y, z.z, o.z), o.w = fmaf(y, z.w, o.w);
      }
    }
  }
  sums[threadIdx.x] = o;
  __syncthreads();
  if (threadIdx.x < D) {
    // Element e is part e % 4 of column e / 4 of every row of lanes.
    const float* p = reinterpret_cast<const float*>(sums) + threadIdx.x;
    float t = 0.0f;
    for (int x = 0; x < rows; ++x) t += p[x * D];
    *reinterpret_cast<U*>(a.out.data + static_cast<long long>(i) * a.out.row + h * a.out.head + threadIdx.x * sizeof(U)) = Pack<U>::one(t * a.scale);
  }
  allow_next_grid();
}

// ------------------------------------------------------------ host side

View view_of(const pv_heads* h, int elem) { return View{static_cast<char*>(h->data), h->row_stride * elem, h->head_stride * elem}; }

constexpr float kLeastScale = 5.421010862427522e-20f;  // 2^-64

int check_shape(int heads, int head_dim, float scale, const float* log_decay, int* dev) {
  if (heads < 1 || heads > 4096 || head_dim < 8 || head_dim > 128 || head_dim % 8) return PV_ERR_INVALID;
  // (Backward, gradients of last states are divided by the scale.)
  if (!(scale >= kLeastScale) || !std::isfinite(scale)) return PV_ERR_INVALID;
  if (!log_decay || !aligned(log_decay, 4) || (*dev = device_of(log_decay)) < 0) return PV_ERR_INVALID;
  return PV_OK;
}

int check_params(const pv_linear_params* p, int* dev) {
  if (!p || p->dtype != PV_BF16) return PV_ERR_INVALID;
  const int st = check_offsets(p->offsets, p->frames);
  if (st != PV_OK) return st;
  if (p->offsets[p->frames] > PV_ATTENTION_MAX_ROWS) return PV_ERR_TOO_LARGE;
  return check_shape(p->heads, p->head_dim, p->scale, p->log_decay, dev);
}

int check_tiles(const pv_heads* h, int64_t rows, int heads, int dev) {
  const int st = check_heads(h, rows, heads, 2, dev);
  return st == PV_OK && rows > 1 && h->row_stride == 0 ? PV_ERR_INVALID : st;
}

bool state_on(const float* p, int dev) { return aligned(p, 16) && device_of(p) == dev; }

LinArgs args_of(const pv_linear_params* p) {
  LinArgs a{};
  a.log_decay = p->log_decay;
  a.frames = p->frames;
  a.H = p->heads;
  a.D = p->head_dim;
  a.halves = a.D > kCols ? 2 : 1;
  for (int f = 0; f <= p->frames; ++f) a.off[f] = static_cast<int>(p->offsets[f]);
  return a;
}

// Chunks of a segment: as many as a frame has, or the fewest that go into one to four rounds of blocks, whichever is
// done first.  Every block has some two chunks' time of its own, and joining segments takes some three.
int chunk_of(const LinArgs& a, int runs, int sms) {
  int most = 1;
  for (int f = 0; f < a.frames; ++f) most = std::max(most, a.chunk0[f + 1] - a.chunk0[f]);
  constexpr double kBlock = 2.0, kJoin = 3.0;
  const int64_t heads = static_cast<int64_t>(a.H) * a.halves * runs;
  auto rounds = [&](int chunk) {
    int64_t n = 0;
    for (int f = 0; f < a.frames; ++f) n += std::max(1, (a.chunk0[f + 1] - a.chunk0[f] + chunk - 1) / chunk);
    return (n * heads + sms - 1) / sms;
  };
  double least = rounds(most) * (most + kBlock);
  int best = most;
  for (int64_t r = rounds(most); r <= 4; ++r) {
    int low = 1, high = most;  // the smallest that needs no more than r rounds
    while (low < high) {
      const int mid = (low + high) / 2;
      if (rounds(mid) <= r) high = mid; else low = mid + 1;
    }
    const double cost = rounds(low) * (low + kBlock) + kJoin;
    if (low < most && cost < least) least = cost, best = low;
  }
  return best;
}

template <int kBlocks, int kScores>
int launch_out(const LinArgs& a, const Maps& m, dim3 grid, cudaStream_t s) {
  const int smem = static_cast<int>(sizeof(OutSmem<kBlocks>)) + 1024, st = allow_smem(pv_linear_out_kernel<kBlocks, kScores>, smem);
  return st != PV_OK ? st : launch_pdl(pv_linear_out_kernel<kBlocks, kScores>, grid, kOutThreads, smem, s, a, m);
}

template <int kBlocks>
int launch_runs(const LinArgs& a, const Maps& m, int segments, int runs, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(segments) * a.H * a.halves, runs);
  const int smem = static_cast<int>(sizeof(StateSmem<kBlocks>)) + 1024;
  int st;
  if ((st = allow_smem(pv_linear_states_kernel<kBlocks>, smem)) != PV_OK ||
      (st = launch_pdl(pv_linear_states_kernel<kBlocks>, grid, kStateThreads, smem, s, a, m)) != PV_OK)
    return st;
  if (!a.whole) {
    const dim3 joins(static_cast<unsigned>(a.frames) * a.H * a.halves * (64 * kBlocks * kCols / 4 / 256), runs);
    if ((st = launch_pdl(pv_linear_join_kernel<kBlocks>, joins, 256, 0, s, a)) != PV_OK) return st;
  }
  bool shorts = false, longs = false;  // frames of one chunk, of several
  for (int f = 0; f < a.frames; ++f) {
    const int chunks = a.chunk0[f + 1] - a.chunk0[f];
    shorts = shorts || chunks == 1, longs = longs || chunks > 1;
  }
  if (!shorts && !longs) return PV_OK;  // no rows
  return !shorts ? launch_out<kBlocks, kOnePart>(a, m, grid, s)
                 : longs ? launch_out<kBlocks, kByFrame>(a, m, grid, s) : launch_out<kBlocks, kTwoParts>(a, m, grid, s);
}

int go(LinArgs& a, const Maps& m, int runs, int dev, pv_stream_t stream) {
  const int sms = sm_count(dev);
  if (sms < 1) return PV_ERR_CUDA;
  for (int f = 0; f < a.frames; ++f)
    a.chunk0[f + 1] = a.chunk0[f] + static_cast<int>((static_cast<int64_t>(a.off[f + 1]) - a.off[f] + kRows - 1) / kRows);
  a.chunk = chunk_of(a, runs, sms);
  int64_t segments = 0;
  for (int f = 0; f < a.frames; ++f) {
    segments += std::max(1, (a.chunk0[f + 1] - a.chunk0[f] + a.chunk - 1) / a.chunk);
    if (segments > INT32_MAX) return PV_ERR_TOO_LARGE;
    a.seg0[f + 1] = static_cast<int>(segments);
  }
  a.whole = segments == a.frames;
  const int64_t heads = static_cast<int64_t>(a.H) * a.halves, blocks = segments * heads;
  if (blocks >= (int64_t(1) << 31)) return PV_ERR_TOO_LARGE;
  const int64_t state = (a.D > 64 ? 128 : 64) * kCols;
  a.seg_run = blocks * state;
  a.state_run = a.chunk0[a.frames] * heads * state * 2;
  Scratch scratch;
  const int st = scratch.open(dev, stream, kPlain, static_cast<size_t>(runs) * (6 * a.seg_run + a.state_run));
  if (st != PV_OK) return st;
  a.segs = static_cast<float*>(scratch.body());
  a.starts = reinterpret_cast<unsigned char*>(a.segs + runs * a.seg_run);
  a.states = a.starts + 2 * runs * a.seg_run;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return a.D > 64 ? launch_runs<2>(a, m, static_cast<int>(segments), runs, s)
                  : launch_runs<1>(a, m, static_cast<int>(segments), runs, s);
}

int maps_of(Maps* m, const LinArgs& a, std::initializer_list<const pv_heads*> tensors) {
  int i = 0;
  const int64_t rows = a.off[a.frames];
  if (rows == 0) return PV_OK;  // nothing is loaded
  for (const pv_heads* t : tensors) {
    const int st = make_map(&m->m[i++], view_of(t, 2), PV_BF16, a.D, a.H, 1, rows, kRows);
    if (st != PV_OK) return st;
  }
  return PV_OK;
}

}  // namespace

extern "C" int pv_linear_attention(const pv_linear_params* params, const pv_heads* q, const pv_heads* k, const pv_heads* v,
                                   const float* state, const pv_heads* out, float* last, pv_stream_t stream) try {
  int dev = 0, st = check_params(params, &dev);
  if (st != PV_OK) return st;
  const int64_t rows = params->offsets[params->frames];
  for (const pv_heads* t : {q, k, v})
    if ((st = check_tiles(t, rows, params->heads, dev)) != PV_OK) return st;
  if ((st = check_out_heads(out, rows, params->heads, 2, dev)) != PV_OK) return st;
  if ((state && !state_on(state, dev)) || (last && (!state_on(last, dev) || last == state))) return PV_ERR_INVALID;
  if (rows == 0 && !last) return PV_OK;
  DeviceScope scope(dev);
  if (!scope.ok()) return PV_ERR_CUDA;
  LinArgs a = args_of(params);
  Maps m{};
  if ((st = maps_of(&m, a, {q, k, v})) != PV_OK) return st;
  Run& r = a.run[0];
  r.a = 0, r.b = 1, r.c = 2;
  r.a_head = q->head_stride != 0, r.b_head = k->head_stride != 0, r.c_head = v->head_stride != 0;
  r.reverse = params->reverse != 0;
  r.out = view_of(out, 2);
  r.scale = params->scale;
  r.in = state, r.in_scale = 1.0f, r.in_step = 1;
  r.end = last, r.end_scale = 1.0f;
  return go(a, m, 1, dev, stream);
} catch (...) {
  return caught();
}

extern "C" int pv_linear_attention_backward(const pv_linear_params* params, const pv_heads* dout, const float* dlast,
                                            const pv_heads* q, const pv_heads* k, const pv_heads* v, const float* state,
                                            const pv_heads* dq, const pv_heads* dk, const pv_heads* dv, float* dstate,
                                            pv_stream_t stream) try {
  int dev = 0, st = check_params(params, &dev);
  if (st != PV_OK) return st;
  const int64_t rows = params->offsets[params->frames];
  for (const pv_heads* t : {dout, q, k, v})
    if ((st = check_tiles(t, rows, params->heads, dev)) != PV_OK) return st;
  for (const pv_heads* t : {dq, dk, dv})
    if ((st = check_out_heads(t, rows, params->heads, 2, dev)) != PV_OK) return st;
  for (const float* t : {dlast, state, static_cast<const float*>(dstate)})
    if (t && !state_on(t, dev)) return PV_ERR_INVALID;
  if (dstate && (dstate == dlast || dstate == state)) return PV_ERR_INVALID;
  if (rows == 0 && !dstate) return PV_OK;
  DeviceScope scope(dev);
  if (!scope.ok()) return PV_ERR_CUDA;
  LinArgs a = args_of(params);
  Maps m{};
  if ((st = maps_of(&m, a, {q, k, v, dout})) != PV_OK) return st;
  const pv_heads* from[4] = {q, k, v, dout};
  auto set = [&](int i, int x, int y, int z, bool back, const pv_heads* out, const float* in, bool turned) {
    Run& r = a.run[i];
    r.a = x, r.b = y, r.c = z;
    r.a_head = from[x]->head_stride != 0, r.b_head = from[y]->head_stride != 0, r.c_head = from[z]->head_stride != 0;
    r.reverse = (params->reverse != 0) != back;
    r.out = view_of(out, 2);
    r.scale = params->scale;
    r.in = in, r.in_turned = turned;
    // The gradient of the last state joins the others as it is, neither scaled nor decayed.
    r.in_scale = back ? 1.0f / params->scale : 1.0f;
    r.in_step = !back;
  };
  set(0, 1, 0, 3, true, dv, dlast, false);
  set(1, 2, 3, 0, true, dk, dlast, true);
  set(2, 3, 2, 1, false, dq, state, true);
  a.run[0].end = dstate;
  a.run[0].end_scale = params->scale;
  a.run[0].end_step = 1;
  return go(a, m, kMostRuns, dev, stream);
} catch (...) {
  return caught();
}

extern "C" int pv_linear_attention_step(const pv_linear_step_params* params, const pv_heads* q, const pv_heads* k, const pv_heads* v,
                                        const float* state, const pv_heads* out, float* next_state, pv_stream_t stream) try {
  if (!params || !dtype_size(params->dtype) || params->streams < 0 || params->streams >= (int64_t(1) << 31)) return PV_ERR_INVALID;
  int dev = 0, st = check_shape(params->heads, params->head_dim, params->scale, params->log_decay, &dev);
  if (st != PV_OK) return st;
  const int elem = dtype_size(params->dtype);
  for (const pv_heads* t : {q, k, v})
    if ((st = check_heads(t, params->streams, params->heads, elem, dev)) != PV_OK) return st;
  if ((st = check_out_heads(out, params->streams, params->heads, elem, dev)) != PV_OK) return st;
  if (params->streams == 0) return PV_OK;
  if (!state || !next_state || !state_on(state, dev) || !state_on(next_state, dev)) return PV_ERR_INVALID;
  const int64_t blocks = params->streams * params->heads;
  if (blocks >= (int64_t(1) << 31)) return PV_ERR_TOO_LARGE;
  DeviceScope scope(dev);
  if (!scope.ok()) return PV_ERR_CUDA;
  const StepArgs a{view_of(q, elem), view_of(k, elem), view_of(v, elem), view_of(out, elem), params->log_decay, state, next_state,
                   params->heads, params->head_dim, params->scale};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(blocks));
  switch (params->dtype) {
    case PV_F32: return launch_pdl(pv_linear_step_kernel<float>, grid, 256, 0, s, a);
    case PV_BF16: return launch_pdl(pv_linear_step_kernel<__nv_bfloat16>, grid, 256, 0, s, a);
    default: return launch_pdl(pv_linear_step_kernel<__half>, grid, 256, 0, s, a);
  }
} catch (...) {
  return caught();
}
