// What the voxel-token operators (pv_rope.cu, pv_scan.cu, pv_attn*.cu) share:
// their per-(device, stream) workspace, argument checks, and conversions
// between the storage types and 32-bit arithmetic.

#pragma once

#include "pv.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

namespace pvs {

// ------------------------------------------------------------ host side (pv_seq.cu)

// Device that owns a pointer, or -1 if it is not device (or managed) memory.
int device_of(const void* ptr);
int sm_count(int dev);

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline size_t round_up(size_t v, size_t m) { return (v + m - 1) / m * m; }
inline int dtype_size(int dtype) { return dtype == PV_F32 ? 4 : dtype == PV_BF16 || dtype == PV_F16 ? 2 : 0; }

// PV_OK if `off` holds n + 1 row offsets: 0, never decreasing, below 2^31.
int check_offsets(const int64_t* off, int n);

// PV_OK if `h` can be read (or written) in 16-byte pieces on device `dev`; with
// no rows or no heads the data pointer is not looked at.
int check_heads(const pv_heads* h, int64_t rows, int heads, int elem, int dev);

// The same for what a call writes: its rows and heads do not share memory by a stride of 0.
int check_out_heads(const pv_heads* h, int64_t rows, int heads, int elem, int dev);

// The status of the exception that is being handled.  The entries are called from C: each
// ends in a handler that returns this (maps, lists and locks may throw).
int caught() noexcept;

// Makes `dev` current for a scope.
class DeviceScope {
 public:
  explicit DeviceScope(int dev) {
    if (cudaGetDevice(&prev_) != cudaSuccess) return;
    ok_ = prev_ == dev || cudaSetDevice(dev) == cudaSuccess;
    changed_ = prev_ != dev;
  }
  ~DeviceScope() {
    if (changed_) cudaSetDevice(prev_);
  }
  bool ok() const { return ok_; }

 private:
  int prev_ = 0;
  bool ok_ = false, changed_ = false;
};

// The operators' scratch on one (device, stream).  Locked while a call
// enqueues its work, so the launches of two threads on one stream do not mix.
// A head that is zero at first (counters that each launch leaves as it found
// them, epochs that only grow) and a body of `bytes`, zero at first too.
//
// A call that is being captured into a graph takes one of the capture's own instead (per
// stream, so that it is not shared by branches): the graph holds its address, and may run
// at any time beside calls and graphs that came from the same stream.  The graph, and
// what is instantiated from it, owns that one; the last of them to go gives it back, for
// later captures to take.
enum ScratchKind {
  kPlain = 0,  // the body holds nothing between calls
  kTagged = 1  // the body holds (value, epoch) pairs of the recurrence only
};
constexpr int kHeadFrames = 64;
static_assert(4 * (kHeadFrames + PV_MAX_FRAMES) <= 4096, "the head holds the frames' counters");
struct SeqSpace;
class Scratch {
 public:
  static constexpr size_t kHead = 4096;  // words from kHeadFrames on: a counter a frame
  int open(int dev, pv_stream_t stream, ScratchKind kind, size_t bytes);
  ~Scratch();
  void* head() const;
  void* body() const { return static_cast<char*>(head()) + kHead; }

 private:
  int open_captured(int dev, pv_stream_t stream, ScratchKind kind, size_t need, unsigned long long capture,
                    cudaGraph_t graph);
  SeqSpace* sp_ = nullptr;
};

int release_scratch();  // frees every Scratch that no graph owns (pv_release_workspace)

// ------------------------------------------------------------ device side

__device__ __forceinline__ void wait_prior_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next_grid() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// Two 32-bit operations in one instruction.
__device__ __forceinline__ void fma2(float& x0, float& x1, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(x0), "=f"(x1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float& x0, float& x1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(x0), "=f"(x1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

__device__ __forceinline__ void mul2(float& x0, float& x1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(x0), "=f"(x1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

template <typename T>
struct Pack;  // 16 bytes of T as floats

template <>
struct Pack<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void open(uint4 v, float* f) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ void load(const void* p, float* f) { open(*static_cast<const uint4*>(p), f); }
  static __device__ __forceinline__ void store(void* p, const float* f) {
    *static_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
  static __device__ __forceinline__ float one(float v) { return v; }
  static __device__ __forceinline__ float to(float v) { return v; }
};

template <>
struct Pack<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void load(const void* p, float* f) { open(*static_cast<const uint4*>(p), f); }
  static __device__ __forceinline__ void open(uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint32_t two(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void store(void* p, const float* f) {
    *static_cast<uint4*>(p) = make_uint4(two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7]));
  }
  static __device__ __forceinline__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 one(float v) { return __float2bfloat16_rn(v); }
};

template <>
struct Pack<__half> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void load(const void* p, float* f) { open(*static_cast<const uint4*>(p), f); }
  static __device__ __forceinline__ void open(uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = d.x;
      f[2 * i + 1] = d.y;
    }
  }
  static __device__ __forceinline__ uint32_t two(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void store(void* p, const float* f) {
    *static_cast<uint4*>(p) = make_uint4(two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7]));
  }
  static __device__ __forceinline__ float to(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half one(float v) { return __float2half_rn(v); }
};

}  // namespace pvs
