// Gated linear recurrence along each frame and its backward pass
// (pv_gated_scan, pv_gated_scan_backward in pv.h):
//   h[t] = a[t] h[t-1] + z[t] x[t],  z = sigmoid(gate), a = 1 - z.
//
// One pass over the data.  A frame is cut into tiles of steps (in reading
// order); a block holds one tile of 64 channels or fewer at a time, each thread
// kSteps steps of its one or two channels.  The map of a stretch of steps,
// h_out = A h_in + B, is composed thread by thread in shared memory, published
// per tile, and the state before the tile found from the published maps; then
// every thread runs its steps from its own start and writes them.
//
// The state before a tile is always worked out in the same order, whatever
// blocks finish first: tiles come in groups of kGroup or fewer, the state before a
// group (its base) is published by the last tile of the group before, and a
// tile composes the maps of the tiles ahead of it in its group, in order, onto
// its group's base.  So a link of the chain along a frame is one group, and
// results do not depend on timing.  A published value is one 64-bit word of
// the value and this launch's epoch: readers poll the words themselves, there
// are no flags to clear or fences to pay for.  The launch is cooperative and a
// block takes every gridDim-th tile of one list in which a tile comes after
// those that it waits for: the earliest tile that is not done always belongs to
// a block that runs and works on it.  The list goes round the frames (their
// first tiles, their second ones, ...), so that with many frames what a tile waits for
// was done a round ago.  While a tile's
// arithmetic and its chain go on, the block's next tile is on its way into
// shared memory, each thread copying what it will read itself.
//
// The backward pass walks the tiles the other way.  With c the gradient that
// step t hands to t - 1, e[t] = dh[t] + c[t+1], c[t] = a[t] e[t]: the same
// kind of recurrence.  The forward pass leaves the state before each tile, so
// h[t-1] is rebuilt inside the tile and x, gate and dh are read once.
//
// Bound by memory: forward 2 reads and 1 write per element, backward 3 and 2.
// Measured at 204,057 steps of 512 channels in 32 frames, bf16: forward 151 us,
// backward 255 us, 4.1 TB/s of these bytes; half of the issue slots, the barriers of
// a tile the largest stall.  Two blocks a multiprocessor: three (forward, 85 registers
// a thread) waited more for one another (425 us for both passes against 408, when a step
// was s - z s + z x, which loses infinite states), as did blocks of 128 threads (420) and
// as many blocks as chains (462).

#include "pv_seq.cuh"

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace {

using namespace pvs;

constexpr int kThreads = 256;
constexpr int kSteps = 16;   // steps of a thread
constexpr int kGroup = 8;    // tiles of a group at most
constexpr int kMaxSlab = 64; // channels of a block: 32 lanes of 2
constexpr unsigned long long kWaitNs = 1000000000ull;  // bounded waits: 1 s

struct ScanArgs {
  const void* x;
  const void* gate;
  const void* dh;
  void* out;    // forward: h; backward: dx
  void* out2;   // backward: dgate
  long long xs, gs, ds, os, os2;  // row strides in elements
  const float* first;   // forward: h0; backward: dlast (may be null)
  float* last;          // forward: the last states; backward: dh0 (may be null)
  float* states;        // forward: written (may be null); backward: read
  unsigned long long* maps;   // published: [tiles][A, B][channels]
  unsigned long long* bases;  // published: [groups][channels]
  unsigned int* ctl;    // finished blocks, epoch
  int channels, slabs, lanes_log2, frames, tiles, reverse, steps, group_log2;
  int row0[PV_MAX_FRAMES + 1];   // row offsets of the frames
  int tile0[PV_MAX_FRAMES + 1];  // first tile of each frame
  int group0[PV_MAX_FRAMES + 1]; // first group of each frame
  unsigned char order[PV_MAX_FRAMES];  // the frames by their number of tiles, most first
};

__device__ __forceinline__ void put(unsigned long long* p, float v, unsigned int epoch) {
  const unsigned long long w = (static_cast<unsigned long long>(epoch) << 32) | __float_as_uint(v);
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(w) : "memory");
}

__device__ __forceinline__ unsigned long long peek(const unsigned long long* p) {
  unsigned long long w;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w) : "l"(p) : "memory");
  return w;
}

// The published value at p, of which `w` was read a while ago; NaN if it does
// not come within the limit.
__device__ __forceinline__ float take(unsigned long long w, const unsigned long long* p, unsigned int epoch) {
  unsigned long long until = 0;
  while (static_cast<unsigned int>(w >> 32) != epoch) {
    const unsigned long long t = now_ns();
    if (!until) until = t + kWaitNs;
    if (t > until) return __int_as_float(0x7FFFFFFF);
    w = peek(p);
  }
  return __uint_as_float(static_cast<unsigned int>(w));
}

// 1 / (1 + exp(-v)): -inf gives 0, +inf 1.  For 16-bit gates the fast
// exponential and division, whose errors (some 1e-6 of z) are far below a
// gate's own rounding.
template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
  float e, z;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(z) : "f"(1.0f + e));
  return z;
}
template <>
__device__ __forceinline__ float sigmoid<float>(float v) {
  return 1.0f / (1.0f + expf(-v));
}

// r = a b + c, r = a + b and r = a b for a thread's one or two channels.
template <int V>
__device__ __forceinline__ void vfma(float* r, const float* a, const float* b, const float* c) {
  if (V == 2)
    fma2(r[0], r[V - 1], a[0], a[V - 1], b[0], b[V - 1], c[0], c[V - 1]);
  else
    r[0] = fmaf(a[0], b[0], c[0]);
}
template <int V>
__device__ __forceinline__ void vadd(float* r, const float* a, const float* b) {
  if (V == 2)
    add2(r[0], r[V - 1], a[0], a[V - 1], b[0], b[V - 1]);
  else
    r[0] = a[0] + b[0];
}
template <int V>
__device__ __forceinline__ void vmul(float* r, const float* a, const float* b) {
  if (V == 2)
    mul2(r[0], r[V - 1], a[0], a[V - 1], b[0], b[V - 1]);
  else
    r[0] = a[0] * b[0];
}

// r = a - b.
template <int V>
__device__ __forceinline__ void vsub(float* r, const float* a, const float* b) {
  const float minus[2] = {-1.0f, -1.0f};
  vfma<V>(r, b, minus, a);
}
// a = 1 - z.
template <int V>
__device__ __forceinline__ void keep(float* a, const float* z) {
  const float one[2] = {1.0f, 1.0f};
  vsub<V>(a, one, z);
}

// The product of two factors that states are kept by, which is 0 only if one of them is:
// an infinite state stays infinite however many steps a map spans.
constexpr float kLeast = 1.401298464e-45f;  // the least number above 0
__device__ __forceinline__ float kept(float a, float b) { return fmaxf(a * b, fminf(fminf(a, b), kLeast)); }

template <typename T, int V>
struct Lane;  // V neighbouring channels of one row
template <>
struct Lane<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ Raw closed() { return __uint_as_float(0xFF800000u); }  // a gate of -inf
  static __device__ __forceinline__ void open(Raw r, float* f) { f[0] = r; }
  static __device__ __forceinline__ Raw close(const float* f) { return f[0]; }
};
template <typename T>
struct Lane<T, 1> {
  using Raw = T;
  static __device__ __forceinline__ Raw closed() { return Pack<T>::one(__uint_as_float(0xFF800000u)); }
  static __device__ __forceinline__ void open(Raw r, float* f) { f[0] = Pack<T>::to(r); }
  static __device__ __forceinline__ Raw close(const float* f) { return Pack<T>::one(f[0]); }
};
template <>
struct Lane<__nv_bfloat16, 2> {
  using Raw = uint32_t;
  static __device__ __forceinline__ Raw closed() { return 0xFF80FF80u; }
  static __device__ __forceinline__ void open(Raw r, float* f) {
    f[0] = __uint_as_float(r << 16);
    f[1] = __uint_as_float(r & 0xFFFF0000u);
  }
  static __device__ __forceinline__ Raw close(const float* f) { return Pack<__nv_bfloat16>::two(f[0], f[1]); }
};
template <>
struct Lane<__half, 2> {
  using Raw = uint32_t;
  static __device__ __forceinline__ Raw closed() { return 0xFC00FC00u; }
  static __device__ __forceinline__ void open(Raw r, float* f) {
    const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&r));
    f[0] = d.x;
    f[1] = d.y;
  }
  static __device__ __forceinline__ Raw close(const float* f) { return Pack<__half>::two(f[0], f[1]); }
};

// Copies one word that only this thread reads back.  16-bit words, which the
// asynchronous copy does not take, go through a register.
template <typename Raw>
__device__ __forceinline__ void stage(Raw* to, const Raw* from) {
  if constexpr (sizeof(Raw) == 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from)
                 : "memory");
  } else {
    *to = __ldcs(from);
  }
}
__device__ __forceinline__ void stage_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All groups but the last one are there.
__device__ __forceinline__ void stage_wait() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// The last block of a launch leaves the counter as it found it, the epoch one on.
__device__ __forceinline__ void leave(const ScanArgs& a) {
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(a.ctl, 1u) == gridDim.x - 1) {
      a.ctl[0] = 0;
      a.ctl[1] += 1u;
    }
  }
}

// Frames without rows: their last state is the first one (backward: dh0 = dlast).
__device__ __forceinline__ void empty_frames(const ScanArgs& a) {
  if (!a.last) return;
  for (int f = blockIdx.x; f < a.frames; f += gridDim.x)
    if (a.row0[f] == a.row0[f + 1])
      for (int c = threadIdx.x; c < a.channels; c += kThreads)
        a.last[static_cast<long long>(f) * a.channels + c] =
            a.first ? a.first[static_cast<long long>(f) * a.channels + c] : 0.0f;
}

template <typename T, int V, bool kBack>
__global__ void __launch_bounds__(kThreads, 2) pv_scan_kernel(const __grid_constant__ ScanArgs a) {
  using L = Lane<T, V>;
  using Raw = typename L::Raw;
  constexpr int kIn = kBack ? 3 : 2;    // tensors read
  constexpr int kRows = kBack ? 3 : 2;  // of a thread's maps: A, B (, the gradient's B)
  // Two stages of every thread's words, [stage][tensor][step][thread], then the
  // threads' maps, [segment][row][channel].
  extern __shared__ __align__(16) unsigned char dyn[];
  Raw* const words = reinterpret_cast<Raw*>(dyn) + threadIdx.x;
  float* const all = reinterpret_cast<float*>(dyn + sizeof(Raw) * 2 * kIn * kSteps * kThreads);
  __shared__ float carry[kMaxSlab];
  __shared__ float fetch[kGroup][2][kMaxSlab];
  wait_prior_grid();
  empty_frames(a);
  const unsigned int epoch = *reinterpret_cast<volatile unsigned int*>(a.ctl + 1) + 1u;
  const int lanes = 1 << a.lanes_log2;
  const int width_log2 = a.lanes_log2 + (V - 1);
  const int width = 1 << width_log2;
  const int cl = threadIdx.x & (lanes - 1);
  const int seg = threadIdx.x >> a.lanes_log2, segs = kThreads >> a.lanes_log2;
  const int C = a.channels;
  const long long dir = a.reverse ? -1 : 1;
  const int total = a.tiles * a.slabs;

  struct Tile {
    int tile, frame, slab, ch, n;  // n: steps of this thread (may be negative)
    long long row;                 // row of its first step
  };
  // Place i of the list, for rising i: round `round` starts at place `before` and
  // has the `count` frames of `order` that have that many tiles.
  int round = 0, before = 0, count = a.frames;
  auto tiles_in = [&](int f) { return a.tile0[f + 1] - a.tile0[f]; };
  auto shrink = [&]() {
    while (count > 0 && tiles_in(a.order[count - 1]) <= round) --count;
  };
  shrink();
  auto tile_at = [&](int i) {
    Tile t;
    const int place = i / a.slabs;
    t.slab = i - place * a.slabs;
    while (place >= before + count) {
      before += count;
      ++round;
      shrink();
    }
    t.frame = a.order[place - before];
    t.tile = kBack ? a.tile0[t.frame + 1] - 1 - round : a.tile0[t.frame] + round;
    const int r0 = a.row0[t.frame], len = a.row0[t.frame + 1] - r0;
    const int i0 = (t.tile - a.tile0[t.frame]) * a.steps + seg * kSteps;
    t.ch = t.slab * width + cl * V;
    t.n = t.ch < C ? min(kSteps, len - i0) : 0;
    t.row = a.reverse ? r0 + len - 1 - i0 : r0 + i0;
    return t;
  };
  auto load = [&](const Tile& t, int at) {
    Raw* to = words + at * (kIn * kSteps * kThreads);
    const Raw* px = reinterpret_cast<const Raw*>(static_cast<const T*>(a.x) + t.row * a.xs + t.ch);
    const Raw* pg = reinterpret_cast<const Raw*>(static_cast<const T*>(a.gate) + t.row * a.gs + t.ch);
    const Raw* pd = reinterpret_cast<const Raw*>(static_cast<const T*>(a.dh) + t.row * a.ds + t.ch);
    const long long sx = dir * a.xs / V, sg = dir * a.gs / V, sd = dir * a.ds / V;
    if (__all_sync(0xFFFFFFFFu, t.n == kSteps)) {
#pragma unroll
      for (int j = 0; j < kSteps; ++j, px += sx, pg += sg, pd += sd) {
        stage(to + j * kThreads, px);
        stage(to + (kSteps + j) * kThreads, pg);
        if (kBack) stage(to + (2 * kSteps + j) * kThreads, pd);
      }
    } else {
      // Steps past the frame's end, and channels past the last, are steps with a
      // closed gate and nothing to read: they leave the state alone.
      const float zero[V] = {};
#pragma unroll 4
      for (int j = 0; j < kSteps; ++j, px += sx, pg += sg, pd += sd) {
        if (j < t.n) {
          stage(to + j * kThreads, px);
          stage(to + (kSteps + j) * kThreads, pg);
          if (kBack) stage(to + (2 * kSteps + j) * kThreads, pd);
        } else {
          to[j * kThreads] = L::close(zero);
          to[(kSteps + j) * kThreads] = L::closed();
          if (kBack) to[(2 * kSteps + j) * kThreads] = L::close(zero);
        }
      }
    }
  };

  int at = 0;
  Tile next{};
  if (static_cast<int>(blockIdx.x) < total) {
    next = tile_at(blockIdx.x);
    load(next, 0);
  }
  stage_close();
  for (int i = blockIdx.x; i < total; i += gridDim.x, at ^= 1) {
    const Tile now = next;
    if (i + static_cast<int>(gridDim.x) < total) {
      next = tile_at(i + gridDim.x);
      load(next, at ^ 1);
    }
    stage_close();
    // Where the tile stands in its frame's chain, and the published words that it
    // will need: read now, looked at (and if need be awaited) after its own maps.
    const int t0 = a.tile0[now.frame], nt = a.tile0[now.frame + 1] - t0;
    const int place = kBack ? nt - 1 - (now.tile - t0) : now.tile - t0;
    const int group = place >> a.group_log2, ahead = place - (group << a.group_log2);
    const bool closes = ahead + 1 == 1 << a.group_log2;  // the last of its group
    const int c0 = now.slab * width, own = c0 + threadIdx.x;
    const bool owner = threadIdx.x < width && own < C;
    auto map_at = [&](int k) {  // of the chain's tile k: A, then B, of channel 0
      return a.maps + static_cast<long long>(kBack ? t0 + nt - 1 - k : t0 + k) * 2 * C;
    };
    // A thread takes channel c of the tiles j0, j0 + j_step, ... ahead.
    constexpr int kTurns = kGroup * 32 * V / kThreads;
    const int c = threadIdx.x & (width - 1), j0 = threadIdx.x >> width_log2, j_step = kThreads >> width_log2;
    const int wanted = c0 + c < C ? ahead : 0;
    const unsigned long long* const ahead_at = map_at((group << a.group_log2) + j0) + c0 + c;
    const long long ahead_step = static_cast<long long>(kBack ? -2 : 2) * C * j_step;
    unsigned long long early[kTurns][2];
#pragma unroll
    for (int q = 0; q < kTurns; ++q) {
      if (j0 + q * j_step < wanted) {
        early[q][0] = peek(ahead_at + q * ahead_step);
        early[q][1] = peek(ahead_at + q * ahead_step + C);
      }
    }
    const unsigned long long* base_at = a.bases + static_cast<long long>(a.group0[now.frame] + group) * C + own;
    unsigned long long base_word = 0;
    float start = 0.0f, state = 0.0f;  // group 0's base; backward: the state before the tile
    if (owner) {
      if (group)
        base_word = peek(base_at);
      else if (a.first)
        start = a.first[static_cast<long long>(now.frame) * C + own];
      if (kBack) state = a.states[static_cast<long long>(now.tile) * C + own];
    }
    stage_wait();
    const Raw* in = words + at * (kIn * kSteps * kThreads);
    auto word = [&](int tensor, int j, float* f) { L::open(in[(tensor * kSteps + j) * kThreads], f); };
    // A step is (1 - z) s + z x as it stands (s + z (x - s) would make no number of an
    // infinite s, as would s - z s), two channels an instruction.
    float z[kSteps][V];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      word(1, j, z[j]);
#pragma unroll
      for (int v = 0; v < V; ++v) z[j][v] = sigmoid<T>(z[j][v]);
    }
    float A[V], B[V], Cb[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f, Cb[v] = 0.0f;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      float x[V], k[V];
      word(0, j, x);
      keep<V>(k, z[j]);
      vmul<V>(x, z[j], x);
      vmul<V>(A, k, A);
      vfma<V>(B, k, B, x);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (A[v] == 0.0f) {  // as in `kept`, all at once: seldom
        float most = 0.0f;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) most = fmaxf(most, z[j][v]);
        if (most < 1.0f) A[v] = kLeast;
      }
    }
    if (kBack) {
#pragma unroll
      for (int j = kSteps - 1; j >= 0; --j) {
        float d[V], k[V];
        word(2, j, d);
        keep<V>(k, z[j]);
        vadd<V>(d, d, Cb);
        vmul<V>(Cb, k, d);
      }
    }
    float* const mine = all + seg * kRows * width + cl * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      mine[v] = A[v];
      mine[width + v] = B[v];
      if (kBack) mine[2 * width + v] = Cb[v];
    }
    __syncthreads();
    // One thread per channel joins the threads' maps; each map is replaced by
    // the map of everything ahead of it in the tile (backward: the state before
    // it, and the map of everything behind it).
    float TA = 1.0f, TB = 0.0f;
    if (owner) {
      float* p = all + threadIdx.x;
      if (!kBack) {
#pragma unroll 8
        for (int s = 0; s < segs; ++s, p += kRows * width) {
          const float sa = p[0], sb = p[width];
          p[0] = TA;
          p[width] = TB;
          TB = fmaf(sa, TB, sb);
          TA = kept(sa, TA);
        }
      } else {
        // Forward along the tile from the state that the forward pass left, and
        // the gradient's map backward.
        float h = state;
        float* pe = p + (segs - 1) * kRows * width;
#pragma unroll 8
        for (int s = 0; s < segs; ++s, p += kRows * width) {
          const float sb = p[width];
          p[width] = h;
          h = fmaf(p[0], h, sb);
        }
#pragma unroll 8
        for (int s = 0; s < segs; ++s, pe -= kRows * width) {
          const float sa = pe[0], sc = pe[2 * width];
          pe[0] = TA;
          pe[2 * width] = TB;
          TB = fmaf(sa, TB, sc);
          TA = kept(sa, TA);
        }
      }
    }
    if (owner && !closes) {
      put(map_at(place) + own, TA, epoch);
      put(map_at(place) + C + own, TB, epoch);
    }
#pragma unroll
    for (int q = 0; q < kTurns; ++q) {
      const int j = j0 + q * j_step;
      if (j < wanted) {
        fetch[j][0][c] = take(early[q][0], ahead_at + q * ahead_step, epoch);
        fetch[j][1][c] = take(early[q][1], ahead_at + q * ahead_step + C, epoch);
      }
    }
    if (ahead) __syncthreads();
    if (owner) {
      // The maps ahead are joined before the base is waited for: a link of the
      // chain is one multiply-add.
      float GA = 1.0f, GB = 0.0f;
#pragma unroll 5
      for (int j = 0; j < ahead; ++j) {
        GB = fmaf(fetch[j][0][threadIdx.x], GB, fetch[j][1][threadIdx.x]);
        GA = kept(fetch[j][0][threadIdx.x], GA);
      }
      if (group) start = take(base_word, base_at, epoch);
      const float s = fmaf(GA, start, GB), after = fmaf(TA, s, TB);
      carry[threadIdx.x] = s;
      if (place == nt - 1) {
        if (a.last) a.last[static_cast<long long>(now.frame) * C + own] = after;
      } else if (closes) {
        put(a.bases + static_cast<long long>(a.group0[now.frame] + group + 1) * C + own, after, epoch);
      }
      if (!kBack && a.states) a.states[static_cast<long long>(now.tile) * C + own] = s;
    }
    __syncthreads();
    float s[V];
    if (!kBack) {
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = fmaf(mine[v], carry[cl * V + v], mine[width + v]);
      Raw* po = reinterpret_cast<Raw*>(static_cast<T*>(a.out) + now.row * a.os + now.ch);
      const long long so = dir * a.os / V;
      auto run = [&](auto whole) {
#pragma unroll
        for (int j = 0; j < kSteps; ++j, po += so) {
          float x[V], k[V];
          word(0, j, x);
          keep<V>(k, z[j]);
          vmul<V>(x, z[j], x);
          vfma<V>(s, k, s, x);
          if (decltype(whole)::value || j < now.n) __stcs(po, L::close(s));
        }
      };
      if (__all_sync(0xFFFFFFFFu, now.n == kSteps))
        run(std::true_type{});
      else
        run(std::false_type{});
    } else {
      float diff[kSteps][V];  // x[t] - h[t-1]
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = mine[width + v];
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        float x[V], k[V];
        word(0, j, x);
        vsub<V>(diff[j], x, s);
        keep<V>(k, z[j]);
        vmul<V>(x, z[j], x);
        vfma<V>(s, k, s, x);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = fmaf(mine[v], carry[cl * V + v], mine[2 * width + v]);
      const long long so = dir * a.os / V, sq = dir * a.os2 / V;
      Raw* po = reinterpret_cast<Raw*>(static_cast<T*>(a.out) + now.row * a.os + now.ch) + (kSteps - 1) * so;
      Raw* pq = reinterpret_cast<Raw*>(static_cast<T*>(a.out2) + now.row * a.os2 + now.ch) + (kSteps - 1) * sq;
      auto run = [&](auto whole) {
#pragma unroll
        for (int j = kSteps - 1; j >= 0; --j, po -= so, pq -= sq) {
          float d[V], k[V], gx[V], gg[V];
          word(2, j, d);
          vadd<V>(d, d, s);
          vmul<V>(gx, d, z[j]);  // e z
          keep<V>(k, z[j]);
          vmul<V>(s, k, d);
          vmul<V>(gg, z[j], diff[j]);
          vmul<V>(gg, gg, s);  // e z (1 - z) (x - h)
          if (decltype(whole)::value || j < now.n) {
            __stcs(po, L::close(gx));
            __stcs(pq, L::close(gg));
          }
        }
      };
      if (__all_sync(0xFFFFFFFFu, now.n == kSteps))
        run(std::true_type{});
      else
        run(std::false_type{});
    }
    // (No barrier here: of what the next tile writes before its first one, the other threads
    // read nothing any more.)
  }
  leave(a);
  allow_next_grid();
}

// ------------------------------------------------------------ host side

struct Shape {
  int vec, lanes_log2, steps, slabs, elem;
  int64_t tiles;
};

// Two 16-bit channels share a 32-bit word where every row begins on one.
bool paired(const void* p, int64_t stride) { return stride % 2 == 0 && aligned(p, 4); }

// How the steps are cut into tiles goes by the offsets, the number of channels and the type
// alone, since the states that a forward call leaves are handed to a backward call whose
// tensors may lie otherwise: an even number of 16-bit channels has the tiles of lanes of
// two channels, also where alignment leaves a lane only one.
int shape_of(const pv_scan_params* p, bool pairs, Shape* s) {
  s->elem = dtype_size(p->dtype);
  const int per_lane = s->elem == 2 && p->channels % 2 == 0 ? 2 : 1;
  s->vec = pairs ? per_lane : 1;
  const int64_t words = (p->channels + per_lane - 1) / per_lane;
  s->lanes_log2 = 0;
  while ((1 << s->lanes_log2) < 32 && (int64_t(1) << s->lanes_log2) < words) ++s->lanes_log2;
  s->steps = (kThreads >> s->lanes_log2) * kSteps;
  const int64_t width = int64_t(s->vec) << s->lanes_log2;
  s->slabs = static_cast<int>((p->channels + width - 1) / width);
  s->tiles = 0;
  for (int b = 0; b < p->frames; ++b) {
    const int64_t t = (p->offsets[b + 1] - p->offsets[b] + s->steps - 1) / s->steps;
    s->tiles += t;
  }
  return s->tiles * s->slabs < (int64_t(1) << 31) ? PV_OK : PV_ERR_TOO_LARGE;
}

int check_params(const pv_scan_params* p) {
  if (!p || !dtype_size(p->dtype)) return PV_ERR_INVALID;
  int st = check_offsets(p->offsets, p->frames);
  if (st != PV_OK) return st;
  if (p->channels < 1 || p->channels > (int64_t(1) << 20)) return PV_ERR_INVALID;
  return PV_OK;
}

// A row stride of 0 is one row seen as many, for what is read.
bool readable(int64_t stride, int64_t channels) { return stride >= channels || stride == 0; }

bool on_device(const void* p, size_t align, int dev) { return p && aligned(p, align) && device_of(p) == dev; }

template <typename T, int V, bool kBack>
int run(ScanArgs& a, const Shape& sh, int dev, int sms, pv_stream_t stream) {
  auto kernel = pv_scan_kernel<T, V, kBack>;
  const size_t smem = sizeof(typename Lane<T, V>::Raw) * 2 * (kBack ? 3 : 2) * kSteps * kThreads +
                      sizeof(float) * (kBack ? 3 : 2) * kThreads * V;
  // Blocks that the device holds at once, asked once per device.
  static std::atomic<int> resident[64];
  int per_sm = resident[dev].load();
  if (!per_sm) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, smem) != cudaSuccess || per_sm < 1) {
      cudaGetLastError();
      return PV_ERR_CUDA;
    }
    resident[dev].store(per_sm);
  }
  const int64_t all = std::max<int64_t>(1, sh.tiles * sh.slabs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(std::min<int64_t>(all, static_cast<int64_t>(per_sm) * sms)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeCooperative;
  at[0].val.cooperative = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return PV_ERR_CUDA;
  }
  return PV_OK;
}

template <bool kBack>
int start(const pv_scan_params* p, const Shape& sh, ScanArgs& a, int dev, pv_stream_t stream) {
  DeviceScope scope(dev);
  if (!scope.ok()) return PV_ERR_CUDA;
  if (dev >= 64) return PV_ERR_UNSUPPORTED;
  a.x = p->x;
  a.gate = p->gate;
  a.xs = p->x_stride;
  a.gs = p->gate_stride;
  a.channels = static_cast<int>(p->channels);
  a.slabs = sh.slabs;
  a.lanes_log2 = sh.lanes_log2;
  a.frames = p->frames;
  a.tiles = static_cast<int>(sh.tiles);
  a.reverse = p->reverse != 0;
  a.steps = sh.steps;
  const int sms = sm_count(dev);
  if (sms < 1) return PV_ERR_CUDA;
  int frames = 0;
  for (int b = 0; b < p->frames; ++b) frames += p->offsets[b + 1] > p->offsets[b];
  // Groups shorten a chain whose tiles are worked on side by side, and cost their maps'
  // publishing and joining: half as many tiles as one chain has in flight.  (As above, forward
  // and backward, bf16, 512 channels, groups of 1 and 8: 32 frames of up to 9,000 steps,
  // 256 chains, 427 and 448 us; one frame of 60,000, 8 chains, 457 and 214 us.)
  const int64_t chains = std::max<int64_t>(1, static_cast<int64_t>(frames) * sh.slabs);
  a.group_log2 = 0;
  while ((1 << a.group_log2) < kGroup && (chains << a.group_log2) * 4 <= 2 * sms) ++a.group_log2;
  for (int b = 0; b < p->frames; ++b) {
    const int64_t t = (p->offsets[b + 1] - p->offsets[b] + sh.steps - 1) / sh.steps;
    a.row0[b + 1] = static_cast<int>(p->offsets[b + 1]);
    a.tile0[b + 1] = a.tile0[b] + static_cast<int>(t);
    a.group0[b + 1] = a.group0[b] + static_cast<int>((t + (1 << a.group_log2) - 1) >> a.group_log2);
    a.order[b] = static_cast<unsigned char>(b);
  }
  std::stable_sort(a.order, a.order + p->frames, [&](unsigned char x, unsigned char y) {
    return a.tile0[x + 1] - a.tile0[x] > a.tile0[y + 1] - a.tile0[y];
  });
  Scratch scratch;
  const size_t words = static_cast<size_t>(2 * sh.tiles + a.group0[p->frames]) * p->channels;
  int st = scratch.open(dev, stream, kTagged, 8 * words);
  if (st != PV_OK) return st;
  a.ctl = static_cast<unsigned int*>(scratch.head());
  a.maps = static_cast<unsigned long long*>(scratch.body());
  a.bases = a.maps + 2 * sh.tiles * p->channels;
  if (p->dtype == PV_F32) return run<float, 1, kBack>(a, sh, dev, sms, stream);
  if (p->dtype == PV_BF16)
    return sh.vec == 2 ? run<__nv_bfloat16, 2, kBack>(a, sh, dev, sms, stream)
                       : run<__nv_bfloat16, 1, kBack>(a, sh, dev, sms, stream);
  return sh.vec == 2 ? run<__half, 2, kBack>(a, sh, dev, sms, stream) : run<__half, 1, kBack>(a, sh, dev, sms, stream);
}

}  // namespace

extern "C" int64_t pv_gated_scan_states(const pv_scan_params* params) {
  int st = check_params(params);
  if (st != PV_OK) return st;
  Shape sh;
  if ((st = shape_of(params, true, &sh)) != PV_OK) return st;
  return sh.tiles;
}

extern "C" int pv_gated_scan(const pv_scan_params* params, const float* h0, void* out_h, int64_t h_stride,
                             float* out_last, float* out_states, pv_stream_t stream) try {
  int st = check_params(params);
  if (st != PV_OK) return st;
  const int64_t rows = params->offsets[params->frames], C = params->channels;
  const int elem = dtype_size(params->dtype);
  const void* any = rows ? out_h : static_cast<void*>(out_last);
  if (!any) return rows ? PV_ERR_INVALID : PV_OK;
  const int dev = device_of(any);
  if (dev < 0) return PV_ERR_INVALID;
  if (rows && (!on_device(params->x, elem, dev) || !on_device(params->gate, elem, dev) ||
               !on_device(out_h, elem, dev) || !readable(params->x_stride, C) || !readable(params->gate_stride, C) || h_stride < C))
    return PV_ERR_INVALID;
  if ((h0 && !on_device(h0, 4, dev)) || (out_last && !on_device(out_last, 4, dev)) ||
      (rows && out_states && !on_device(out_states, 4, dev)))
    return PV_ERR_INVALID;
  const bool pairs = paired(params->x, params->x_stride) && paired(params->gate, params->gate_stride) &&
                     paired(out_h, h_stride);
  Shape sh;
  if ((st = shape_of(params, pairs, &sh)) != PV_OK) return st;
  ScanArgs a{};
  a.out = out_h;
  a.os = h_stride;
  a.first = h0;
  a.last = out_last;
  a.states = out_states;
  return start<false>(params, sh, a, dev, stream);
} catch (...) {
  return caught();
}

extern "C" int pv_gated_scan_backward(const pv_scan_params* params, const void* dh, int64_t dh_stride,
                                      const float* dlast, const float* states, void* dx, int64_t dx_stride,
                                      void* dgate, int64_t dgate_stride, float* dh0, pv_stream_t stream) try {
  int st = check_params(params);
  if (st != PV_OK) return st;
  const int64_t rows = params->offsets[params->frames], C = params->channels;
  const int elem = dtype_size(params->dtype);
  const void* any = rows ? dx : static_cast<void*>(dh0);
  if (!any) return rows ? PV_ERR_INVALID : PV_OK;
  const int dev = device_of(any);
  if (dev < 0) return PV_ERR_INVALID;
  if (rows && (!on_device(params->x, elem, dev) || !on_device(params->gate, elem, dev) || !on_device(dh, elem, dev) ||
               !on_device(dx, elem, dev) || !on_device(dgate, elem, dev) || !on_device(states, 4, dev) ||
               !readable(params->x_stride, C) || !readable(params->gate_stride, C) || !readable(dh_stride, C) ||
               dx_stride < C || dgate_stride < C))
    return PV_ERR_INVALID;
  if ((dlast && !on_device(dlast, 4, dev)) || (dh0 && !on_device(dh0, 4, dev))) return PV_ERR_INVALID;
  const bool pairs = paired(params->x, params->x_stride) && paired(params->gate, params->gate_stride) &&
                     paired(dh, dh_stride) && paired(dx, dx_stride) && paired(dgate, dgate_stride);
  Shape sh;
  if ((st = shape_of(params, pairs, &sh)) != PV_OK) return st;
  ScanArgs a{};
  a.dh = dh;
  a.ds = dh_stride;
  a.out = dx;
  a.os = dx_stride;
  a.out2 = dgate;
  a.os2 = dgate_stride;
  a.first = dlast;
  a.last = dh0;
  a.states = const_cast<float*>(states);
  return start<true>(params, sh, a, dev, stream);
} catch (...) {
  return caught();
}
