// Gated linear recurrence along each frame and its backward pass
// (pv_gated_scan, pv_gated_scan_backward in pv.h):
//   h[t] = a[t] h[t-1] + z[t] x[t],  z = sigmoid(gate), a = 1 - z.
//
// One pass over the data.  A frame is cut into tiles of steps (in reading
// order); a block holds one tile of 32 * kVec channels or fewer, each thread
// kSteps steps of its channels in registers.  The map of a stretch of steps,
// h_out = A h_in + B, is composed thread by thread in shared memory, published
// per tile, and the state before the tile found from the published maps; then
// every thread runs its steps from its own start and writes them.
//
// The state before a tile is always worked out in the same order, whatever
// blocks finish first: tiles come in groups of kGroup, the state before a
// group (its base) is published by the last tile of the group before, and a
// tile composes the maps of the tiles ahead of it in its group, in order, onto
// its group's base.  So a link of the chain along a frame is one group, and
// results do not depend on timing.  A published value is one 64-bit word of
// the value and this launch's epoch: readers poll the words themselves, there
// are no flags to clear or fences to pay for.  Tiles are handed out by a
// ticket in chain order, so a block only ever waits for blocks that run.
//
// The backward pass walks the tiles the other way.  With c the gradient that
// step t hands to t - 1, e[t] = dh[t] + c[t+1], c[t] = a[t] e[t]: the same
// kind of recurrence.  The forward pass leaves the state before each tile, so
// h[t-1] is rebuilt inside the tile and x, gate and dh are read once.
//
// Bound by memory: forward 2 reads and 1 write per element, backward 3 and 2.

#include "pv_seq.cuh"

#include <algorithm>

namespace {

using namespace pvs;

constexpr int kThreads = 256;
constexpr int kSteps = 16;   // steps of a thread
constexpr int kGroup = 16;   // tiles of a group
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
  unsigned int* ctl;    // ticket, finished blocks, epoch
  int channels, slabs, lanes_log2, frames, tiles, reverse, steps;
  int row0[PV_MAX_FRAMES + 1];   // row offsets of the frames
  int tile0[PV_MAX_FRAMES + 1];  // first tile of each frame
  int group0[PV_MAX_FRAMES + 1]; // first group of each frame
};

__device__ __forceinline__ void put(unsigned long long* p, float v, unsigned int epoch) {
  const unsigned long long w = (static_cast<unsigned long long>(epoch) << 32) | __float_as_uint(v);
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(w) : "memory");
}

// A published value; NaN if it does not come within the limit.
__device__ __forceinline__ float take(const unsigned long long* p, unsigned int epoch) {
  unsigned long long w, until = 0;
  for (;;) {
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w) : "l"(p) : "memory");
    if (static_cast<unsigned int>(w >> 32) == epoch) return __uint_as_float(static_cast<unsigned int>(w));
    const unsigned long long t = now_ns();
    if (!until) until = t + kWaitNs;
    if (t > until) return __int_as_float(0x7FFFFFFF);
  }
}

// 1 / (1 + exp(-v)): -inf gives 0, +inf 1.  For 16-bit gates the fast
// exponential and division, whose errors (some 1e-6 of z) are far below a
// gate's own rounding.
template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
  return __fdividef(1.0f, 1.0f + __expf(-v));
}
template <>
__device__ __forceinline__ float sigmoid<float>(float v) {
  return 1.0f / (1.0f + expf(-v));
}

template <typename T, int V>
struct Lane;  // V neighbouring channels of one row
template <>
struct Lane<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ void open(Raw r, float* f) { f[0] = r; }
  static __device__ __forceinline__ Raw close(const float* f) { return f[0]; }
};
template <typename T>
struct Lane<T, 1> {
  using Raw = T;
  static __device__ __forceinline__ void open(Raw r, float* f) { f[0] = Pack<T>::to(r); }
  static __device__ __forceinline__ Raw close(const float* f) { return Pack<T>::one(f[0]); }
};
template <>
struct Lane<__nv_bfloat16, 2> {
  using Raw = uint32_t;
  static __device__ __forceinline__ void open(Raw r, float* f) {
    f[0] = __uint_as_float(r << 16);
    f[1] = __uint_as_float(r & 0xFFFF0000u);
  }
  static __device__ __forceinline__ Raw close(const float* f) { return Pack<__nv_bfloat16>::two(f[0], f[1]); }
};
template <>
struct Lane<__half, 2> {
  using Raw = uint32_t;
  static __device__ __forceinline__ void open(Raw r, float* f) {
    const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&r));
    f[0] = d.x;
    f[1] = d.y;
  }
  static __device__ __forceinline__ Raw close(const float* f) { return Pack<__half>::two(f[0], f[1]); }
};

struct Place {
  int tile, frame, chan, seg, segs, step0, len, row_at;
  long long dir;
};

// The state (or gradient) handed to tile `k` of its chain: base of its group,
// then the maps of the tiles ahead of it in the group, in order.  Called by the
// whole block; the result for channel c of the block is carry[c].
// index(i) = place in `maps` of chain tile i of this frame.
template <bool kBack>
__device__ __forceinline__ void chain(const ScanArgs& a, int tile, int frame, int slab, unsigned int epoch, int width,
                                      float A, float B, bool owner, int c_own, float* carry, float (*fetch)[2][kMaxSlab]) {
  const int t0 = a.tile0[frame], n = a.tile0[frame + 1] - t0;
  const int k = kBack ? n - 1 - (tile - t0) : tile - t0;  // place along the chain
  const int g = k / kGroup, ahead = k - g * kGroup;
  const long long C = a.channels;
  const int c0 = slab * width;
  auto at = [&](int i) { return static_cast<long long>(kBack ? t0 + n - 1 - i : t0 + i); };
  if (owner) {  // this tile's own map
    put(a.maps + (at(k) * 2) * C + c0 + c_own, A, epoch);
    put(a.maps + (at(k) * 2 + 1) * C + c0 + c_own, B, epoch);
  }
  // All polls at once: every thread one (tile, channel) at a time.
  for (int i = threadIdx.x; i < ahead * width; i += kThreads) {
    const int j = i / width, c = i - j * width;
    if (c0 + c < C) {
      fetch[j][0][c] = take(a.maps + (at(g * kGroup + j) * 2) * C + c0 + c, epoch);
      fetch[j][1][c] = take(a.maps + (at(g * kGroup + j) * 2 + 1) * C + c0 + c, epoch);
    }
  }
  __syncthreads();
  if (owner) {
    float s;
    // The maps ahead are joined before the base is waited for: a link of the
    // chain is one multiply-add.
    float GA = 1.0f, GB = 0.0f;
    for (int j = 0; j < ahead; ++j) {
      GB = fmaf(fetch[j][0][c_own], GB, fetch[j][1][c_own]);
      GA *= fetch[j][0][c_own];
    }
    if (g == 0)
      s = a.first ? a.first[frame * C + c0 + c_own] : 0.0f;
    else
      s = take(a.bases + (a.group0[frame] + g) * C + c0 + c_own, epoch);
    s = fmaf(GA, s, GB);
    carry[c_own] = s;
    const float after = fmaf(A, s, B);
    if (k == n - 1) {
      if (a.last) a.last[frame * C + c0 + c_own] = after;
    } else if (ahead == kGroup - 1) {
      put(a.bases + (a.group0[frame] + g + 1) * C + c0 + c_own, after, epoch);
    }
    if (!kBack && a.states) a.states[static_cast<long long>(tile) * C + c0 + c_own] = s;
  }
  __syncthreads();
}

// The next tile of this launch, and the frame it belongs to.
template <bool kBack>
__device__ __forceinline__ void claim(const ScanArgs& a, int* tile, int* slab, int* frame, unsigned int* epoch) {
  __shared__ int s[3];
  __shared__ unsigned int e;
  if (threadIdx.x == 0) {
    const int ticket = static_cast<int>(atomicAdd(a.ctl, 1u));
    const int t = kBack ? a.tiles - 1 - ticket / a.slabs : ticket / a.slabs;
    int lo = 0, hi = a.frames - 1;  // the last frame whose first tile is not past t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.tile0[mid] <= t)
        lo = mid;
      else
        hi = mid - 1;
    }
    s[0] = t;
    s[1] = ticket % a.slabs;
    s[2] = lo;
    e = *reinterpret_cast<volatile unsigned int*>(a.ctl + 2) + 1u;
  }
  __syncthreads();
  *tile = s[0];
  *slab = s[1];
  *frame = s[2];
  *epoch = e;
}

// The last block of a launch leaves the counters as it found them, the epoch one on.
__device__ __forceinline__ void leave(const ScanArgs& a) {
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(a.ctl + 1, 1u) == gridDim.x - 1) {
      a.ctl[0] = 0;
      a.ctl[1] = 0;
      a.ctl[2] += 1u;
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
  extern __shared__ float dyn[];  // maps of the threads: [segs][A, B(, backward B)][width]
  __shared__ float carry[kMaxSlab];
  __shared__ float fetch[kGroup][2][kMaxSlab];
  wait_prior_grid();
  empty_frames(a);
  if (a.tiles == 0) {
    allow_next_grid();
    return;
  }
  int tile, slab, frame;
  unsigned int epoch;
  claim<kBack>(a, &tile, &slab, &frame, &epoch);
  const int lanes = 1 << a.lanes_log2;
  const int width = lanes * V;
  const int cl = threadIdx.x & (lanes - 1);
  const int seg = threadIdx.x >> a.lanes_log2, segs = kThreads >> a.lanes_log2;
  const int C = a.channels;
  const int ch = slab * width + cl * V;
  const int r0 = a.row0[frame], len = a.row0[frame + 1] - r0;
  const int i0 = (tile - a.tile0[frame]) * a.steps + seg * kSteps;  // first step of this thread
  const int n = ch < C ? min(kSteps, len - i0) : 0;                 // its steps (may be negative)
  const long long first_row = a.reverse ? r0 + len - 1 - i0 : r0 + i0;
  const long long dir = a.reverse ? -1 : 1;

  Raw rx[kSteps], rg[kSteps], rd[kSteps];
  {
    const T* px = static_cast<const T*>(a.x) + first_row * a.xs + ch;
    const T* pg = static_cast<const T*>(a.gate) + first_row * a.gs + ch;
    const T* pd = static_cast<const T*>(a.dh) + first_row * a.ds + ch;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      if (j < n) {
        rx[j] = __ldcs(reinterpret_cast<const Raw*>(px + j * dir * a.xs));
        rg[j] = __ldcs(reinterpret_cast<const Raw*>(pg + j * dir * a.gs));
        if (kBack) rd[j] = __ldcs(reinterpret_cast<const Raw*>(pd + j * dir * a.ds));
      }
    }
  }
  float z[kSteps][V];
  float A[V], B[V], Cb[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f, Cb[v] = 0.0f;
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    float g[V], x[V];
    if (j < n) {
      L::open(rg[j], g);
      L::open(rx[j], x);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        z[j][v] = sigmoid<T>(g[v]);
        const float keep = 1.0f - z[j][v];
        A[v] *= keep;
        B[v] = fmaf(keep, B[v], z[j][v] * x[v]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) z[j][v] = 0.0f;
    }
  }
  if (kBack) {
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
      if (j < n) {
        float d[V];
        L::open(rd[j], d);
#pragma unroll
        for (int v = 0; v < V; ++v) Cb[v] = (1.0f - z[j][v]) * (d[v] + Cb[v]);
      }
    }
  }
  constexpr int kRows = kBack ? 3 : 2;
  float* mine = dyn + seg * kRows * width + cl * V;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    mine[v] = A[v];
    mine[width + v] = B[v];
    if (kBack) mine[2 * width + v] = Cb[v];
  }
  __syncthreads();
  // One thread per channel joins the threads' maps; each map is replaced by
  // the map of everything ahead of it in the tile (backward also: behind it).
  const bool owner = threadIdx.x < width && slab * width + threadIdx.x < C;
  float TA = 1.0f, TB = 0.0f;
  if (owner) {
    float* p = dyn + threadIdx.x;
    if (!kBack) {
      for (int s = 0; s < segs; ++s, p += kRows * width) {
        const float sa = p[0], sb = p[width];
        p[0] = TA;
        p[width] = TB;
        TB = fmaf(sa, TB, sb);
        TA *= sa;
      }
    } else {
      // Forward along the tile from the state that the forward pass left, and
      // the gradient's map backward.
      float h = a.states[static_cast<long long>(tile) * C + slab * width + threadIdx.x];
      float* pe = p + (segs - 1) * kRows * width;
      for (int s = 0; s < segs; ++s, p += kRows * width) {
        const float sb = p[width];
        p[width] = h;
        h = fmaf(p[0], h, sb);
      }
      for (int s = 0; s < segs; ++s, pe -= kRows * width) {
        const float sa = pe[0], sc = pe[2 * width];
        pe[0] = TA;
        pe[2 * width] = TB;
        TB = fmaf(sa, TB, sc);
        TA *= sa;
      }
    }
  }
  chain<kBack>(a, tile, frame, slab, epoch, width, TA, TB, owner, threadIdx.x, carry, fetch);
  if (n > 0) {
    float s[V];
    T* po = static_cast<T*>(a.out) + first_row * a.os + ch;
    if (!kBack) {
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = fmaf(mine[v], carry[cl * V + v], mine[width + v]);
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        if (j < n) {
          float x[V];
          L::open(rx[j], x);
#pragma unroll
          for (int v = 0; v < V; ++v) s[v] = fmaf(1.0f - z[j][v], s[v], z[j][v] * x[v]);
          __stcs(reinterpret_cast<Raw*>(po + j * dir * a.os), L::close(s));
        }
      }
    } else {
      T* pq = static_cast<T*>(a.out2) + first_row * a.os2 + ch;
      float diff[kSteps][V];  // x[t] - h[t-1]
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = mine[width + v];
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        if (j < n) {
          float x[V];
          L::open(rx[j], x);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            diff[j][v] = x[v] - s[v];
            s[v] = fmaf(1.0f - z[j][v], s[v], z[j][v] * x[v]);
          }
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = fmaf(mine[v], carry[cl * V + v], mine[2 * width + v]);
#pragma unroll
      for (int j = kSteps - 1; j >= 0; --j) {
        if (j < n) {
          float d[V], gx[V], gg[V];
          L::open(rd[j], d);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float e = d[v] + s[v], keep = 1.0f - z[j][v];
            gx[v] = e * z[j][v];
            gg[v] = gx[v] * keep * diff[j][v];
            s[v] = keep * e;
          }
          __stcs(reinterpret_cast<Raw*>(po + j * dir * a.os), L::close(gx));
          __stcs(reinterpret_cast<Raw*>(pq + j * dir * a.os2), L::close(gg));
        }
      }
    }
  }
  leave(a);
  allow_next_grid();
}

// ------------------------------------------------------------ host side

struct Shape {
  int vec, lanes_log2, steps, slabs, elem;
  int64_t tiles, groups;
};

// Two 16-bit channels share a 32-bit word where every row begins on one.
bool paired(const void* p, int64_t stride) { return stride % 2 == 0 && aligned(p, 4); }

int shape_of(const pv_scan_params* p, bool pairs, Shape* s) {
  s->elem = dtype_size(p->dtype);
  s->vec = s->elem == 2 && pairs ? 2 : 1;
  const int64_t words = (p->channels + s->vec - 1) / s->vec;
  s->lanes_log2 = 0;
  while ((1 << s->lanes_log2) < 32 && (int64_t(1) << s->lanes_log2) < words) ++s->lanes_log2;
  s->steps = (kThreads >> s->lanes_log2) * kSteps;
  s->slabs = static_cast<int>((words + (1 << s->lanes_log2) - 1) >> s->lanes_log2);
  s->tiles = s->groups = 0;
  for (int b = 0; b < p->frames; ++b) {
    const int64_t t = (p->offsets[b + 1] - p->offsets[b] + s->steps - 1) / s->steps;
    s->tiles += t;
    s->groups += (t + kGroup - 1) / kGroup;
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

bool on_device(const void* p, size_t align, int dev) { return p && aligned(p, align) && device_of(p) == dev; }

template <typename T, int V, bool kBack>
int run(ScanArgs& a, const Shape& sh, pv_stream_t stream) {
  const int width = (1 << sh.lanes_log2) * V;
  const size_t smem = sizeof(float) * (kThreads >> sh.lanes_log2) * (kBack ? 3 : 2) * width;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(std::max<int64_t>(1, sh.tiles * sh.slabs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, pv_scan_kernel<T, V, kBack>, a) != cudaSuccess) {
    cudaGetLastError();
    return PV_ERR_CUDA;
  }
  return PV_OK;
}

template <bool kBack>
int start(const pv_scan_params* p, const Shape& sh, ScanArgs& a, int dev, pv_stream_t stream) {
  DeviceScope scope(dev);
  if (!scope.ok()) return PV_ERR_CUDA;
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
  for (int b = 0; b < p->frames; ++b) {
    const int64_t t = (p->offsets[b + 1] - p->offsets[b] + sh.steps - 1) / sh.steps;
    a.row0[b + 1] = static_cast<int>(p->offsets[b + 1]);
    a.tile0[b + 1] = a.tile0[b] + static_cast<int>(t);
    a.group0[b + 1] = a.group0[b] + static_cast<int>((t + kGroup - 1) / kGroup);
  }
  Scratch scratch;
  const size_t words = static_cast<size_t>(2 * sh.tiles + sh.groups) * p->channels;
  int st = scratch.open(dev, stream, kTagged, 8 * words);
  if (st != PV_OK) return st;
  a.ctl = static_cast<unsigned int*>(scratch.head());
  a.maps = static_cast<unsigned long long*>(scratch.body());
  a.bases = a.maps + 2 * sh.tiles * p->channels;
  if (p->dtype == PV_F32) return run<float, 1, kBack>(a, sh, stream);
  if (p->dtype == PV_BF16)
    return sh.vec == 2 ? run<__nv_bfloat16, 2, kBack>(a, sh, stream) : run<__nv_bfloat16, 1, kBack>(a, sh, stream);
  return sh.vec == 2 ? run<__half, 2, kBack>(a, sh, stream) : run<__half, 1, kBack>(a, sh, stream);
}

}  // namespace

extern "C" int64_t pv_gated_scan_states(const pv_scan_params* params) {
  int st = check_params(params);
  if (st != PV_OK) return st;
  // The shortest tile that any of the calls on these sizes takes: one channel
  // a lane.  (Whether two channels share a lane goes by alignment.)
  Shape one, two;
  if ((st = shape_of(params, false, &one)) != PV_OK || (st = shape_of(params, true, &two)) != PV_OK) return st;
  return std::max(one.tiles, two.tiles);
}

extern "C" int pv_gated_scan(const pv_scan_params* params, const float* h0, void* out_h, int64_t h_stride,
                             float* out_last, float* out_states, pv_stream_t stream) {
  int st = check_params(params);
  if (st != PV_OK) return st;
  const int64_t rows = params->offsets[params->frames], C = params->channels;
  const int elem = dtype_size(params->dtype);
  const void* any = rows ? out_h : static_cast<void*>(out_last);
  if (!any) return rows ? PV_ERR_INVALID : PV_OK;
  const int dev = device_of(any);
  if (dev < 0) return PV_ERR_INVALID;
  if (rows && (!on_device(params->x, elem, dev) || !on_device(params->gate, elem, dev) ||
               !on_device(out_h, elem, dev) || params->x_stride < C || params->gate_stride < C || h_stride < C))
    return PV_ERR_INVALID;
  if ((h0 && !on_device(h0, 4, dev)) || (out_last && !on_device(out_last, 4, dev)) ||
      (rows && out_states && !on_device(out_states, 4, dev)))
    return PV_ERR_INVALID;
  // The states' layout is part of what is handed to the backward call, so with
  // states the tiles go by the shape alone: channels in pairs if C is even.
  const bool pairs = C % 2 == 0 && paired(params->x, params->x_stride) && paired(params->gate, params->gate_stride) &&
                     paired(out_h, h_stride);
  if (out_states && C % 2 == 0 && elem == 2 && !pairs) return PV_ERR_INVALID;
  Shape sh;
  if ((st = shape_of(params, pairs, &sh)) != PV_OK) return st;
  ScanArgs a{};
  a.out = out_h;
  a.os = h_stride;
  a.first = h0;
  a.last = out_last;
  a.states = out_states;
  return start<false>(params, sh, a, dev, stream);
}

extern "C" int pv_gated_scan_backward(const pv_scan_params* params, const void* dh, int64_t dh_stride,
                                      const float* dlast, const float* states, void* dx, int64_t dx_stride,
                                      void* dgate, int64_t dgate_stride, float* dh0, pv_stream_t stream) {
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
               params->x_stride < C || params->gate_stride < C || dh_stride < C || dx_stride < C || dgate_stride < C))
    return PV_ERR_INVALID;
  if ((dlast && !on_device(dlast, 4, dev)) || (dh0 && !on_device(dh0, 4, dev))) return PV_ERR_INVALID;
  const bool pairs = C % 2 == 0 && paired(params->x, params->x_stride) && paired(params->gate, params->gate_stride) &&
                     paired(dh, dh_stride) && paired(dx, dx_stride) && paired(dgate, dgate_stride);
  if (C % 2 == 0 && elem == 2 && !pairs) return PV_ERR_INVALID;
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
}
