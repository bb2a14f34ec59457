// Attention inside frames and its backward pass (pv_attention,
// pv_attention_backward in pv.h).
//
//   s = scale q.k;  t = cap tanh(s / cap) (or s);  u = t - slope * distance;
//   p = exp(u - lse), lse = log sum of exp(u) over the visible keys;  o = p v.
//   dv = p^T do;  du = p (do.v - delta), delta = do.o;
//   ds = du (1 - (t / cap)^2) scale;  dq = ds k;  dk = ds^T q.
//
// Tiles of 16 rows against tiles of 32, in 32-bit arithmetic on the CUDA
// cores; the running maximum and sum of a row stay in registers.

#include "pv_attn.cuh"

#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <initializer_list>

namespace {

using namespace pvs;

constexpr int kThreads = 128;
constexpr int kOwn = 16;    // rows of a block
constexpr int kOther = 32;  // rows of a step
constexpr int kPad = 129;

// The score of a pair and, for the backward pass, d(score)/d(scale q.k).
__device__ __forceinline__ float score(const AttnArgs& a, float dot, float slope, const int* qp, const int* kp, float* grad) {
  float s = dot * a.scale;
  *grad = 1.0f;
  if (a.cap > 0.0f) {
    const float t = tanhf(s / a.cap);
    *grad = 1.0f - t * t;
    s = a.cap * t;
  }
  if (a.slopes) {
    float d = 0.0f;
    for (int x = 0; x < a.axes; ++x) d += fabsf(static_cast<float>(qp[x]) - static_cast<float>(kp[x]));
    s = fmaf(-slope, d, s);
  }
  return s;
}

__device__ __forceinline__ bool visible(const AttnArgs& a, int f, int i, int j, int nq, int nk) {
  return i < nq && j < nk && (!a.causal || j <= i + nk - nq || j < a.prefix[f]);
}

template <typename T>
__device__ __forceinline__ void load_rows(const View& v, int head, int row0, int rows, int most, int D, float (*to)[kPad]) {
  for (int i = threadIdx.x; i < most * D; i += kThreads) {
    const int r = i / D, d = i - r * D;
    to[r][d] = r < rows ? Pack<T>::to(*(reinterpret_cast<const T*>(v.data + (row0 + r) * v.row + head * v.head) + d)) : 0.0f;
  }
}

__device__ __forceinline__ float dot_of(const float* a, const float* b, int D) {
  float s = 0.0f;
  for (int d = 0; d < D; ++d) s = fmaf(a[d], b[d], s);
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) pv_attn_delta_kernel(const __grid_constant__ AttnArgs a) {
  wait_prior_grid();
  const long long w = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w < static_cast<long long>(a.queries) * a.H) {
    const int row = static_cast<int>(w / a.H), h = static_cast<int>(w % a.H);
    const T* o = reinterpret_cast<const T*>(a.o.data + row * a.o.row + h * a.o.head);
    const T* g = reinterpret_cast<const T*>(a.dout.data + row * a.dout.row + h * a.dout.head);
    float s = 0.0f;
    for (int d = lane; d < a.D; d += 32) s = fmaf(Pack<T>::to(o[d]), Pack<T>::to(g[d]), s);
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    if (lane == 0) a.delta[static_cast<long long>(h) * a.queries + row] = s;
  }
  allow_next_grid();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) pv_attn_dq_kernel(const __grid_constant__ AttnArgs a) {
  extern __shared__ float dyn[];
  auto rows = [&](int at) { return reinterpret_cast<float(*)[kPad]>(dyn + at * kPad); };
  float(*qs)[kPad] = rows(0), (*gs)[kPad] = rows(kOwn), (*ks)[kPad] = rows(2 * kOwn), (*vs)[kPad] = rows(2 * kOwn + kOther);
  __shared__ float ps[kOwn][kOther + 1];
  wait_prior_grid();
  const int f = frame_of(a.tile0, a.frames, blockIdx.x), h = blockIdx.y, g = h / a.G;
  const int nq = a.q0[f + 1] - a.q0[f], nk = a.k0[f + 1] - a.k0[f];
  const int i0 = (blockIdx.x - a.tile0[f]) * kOwn;
  const int r = threadIdx.x >> 3, c = threadIdx.x & 7, i = i0 + r, qrow = a.q0[f] + i;
  load_rows<T>(a.q, h, a.q0[f] + i0, nq - i0, kOwn, a.D, qs);
  load_rows<T>(a.dout, h, a.q0[f] + i0, nq - i0, kOwn, a.D, gs);
  float acc[16];
  for (int d = 0; d < 16; ++d) acc[d] = 0.0f;
  const float slope = a.slopes ? a.slopes[h] : 0.0f;
  const float lse = i < nq ? a.lse[static_cast<long long>(h) * a.queries + qrow] : 0.0f;
  const float delta = i < nq ? a.delta[static_cast<long long>(h) * a.queries + qrow] : 0.0f;
  for (int j0 = 0; j0 < nk; j0 += kOther) {
    __syncthreads();
    load_rows<T>(a.k, g, a.k0[f] + j0, nk - j0, kOther, a.D, ks);
    load_rows<T>(a.v, g, a.k0[f] + j0, nk - j0, kOther, a.D, vs);
    __syncthreads();
    for (int x = 0; x < 4; ++x) {
      const int j = j0 + c + 8 * x;
      float ds = 0.0f, grad;
      if (visible(a, f, i, j, nq, nk)) {
        const float s = score(a, dot_of(qs[r], ks[c + 8 * x], a.D), slope, a.qpos + qrow * a.qpos_stride,
                              a.kpos + (a.k0[f] + j) * a.kpos_stride, &grad);
        ds = expf(s - lse) * (dot_of(gs[r], vs[c + 8 * x], a.D) - delta) * grad;
      }
      ps[r][c + 8 * x] = ds;
    }
    __syncwarp();
    for (int j = 0; j < kOther; ++j)
      for (int d = 0; d < 16; ++d)
        if (c + 8 * d < a.D) acc[d] = fmaf(ps[r][j], ks[j][c + 8 * d], acc[d]);
  }
  if (i < nq) {
    T* o = reinterpret_cast<T*>(a.dq.data + qrow * a.dq.row + h * a.dq.head);
    for (int d = 0; d < 16; ++d)
      if (c + 8 * d < a.D) o[c + 8 * d] = Pack<T>::one(acc[d] * a.scale);
  }
  allow_next_grid();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) pv_attn_dkv_kernel(const __grid_constant__ AttnArgs a) {
  extern __shared__ float dyn[];
  auto rows = [&](int at) { return reinterpret_cast<float(*)[kPad]>(dyn + at * kPad); };
  float(*ks)[kPad] = rows(0), (*vs)[kPad] = rows(kOwn), (*qs)[kPad] = rows(2 * kOwn), (*gs)[kPad] = rows(2 * kOwn + kOther);
  __shared__ float ps[kOwn][kOther + 1], dss[kOwn][kOther + 1];
  wait_prior_grid();
  const int f = frame_of(a.tile0, a.frames, blockIdx.x), g = blockIdx.y;
  const int nq = a.q0[f + 1] - a.q0[f], nk = a.k0[f + 1] - a.k0[f];
  const int j0 = (blockIdx.x - a.tile0[f]) * kOwn;
  const int r = threadIdx.x >> 3, c = threadIdx.x & 7, j = j0 + r, krow = a.k0[f] + j;
  load_rows<T>(a.k, g, a.k0[f] + j0, nk - j0, kOwn, a.D, ks);
  load_rows<T>(a.v, g, a.k0[f] + j0, nk - j0, kOwn, a.D, vs);
  float dk[16], dv[16];
  for (int d = 0; d < 16; ++d) dk[d] = dv[d] = 0.0f;
  for (int h = g * a.G; h < (g + 1) * a.G; ++h) {
    const float slope = a.slopes ? a.slopes[h] : 0.0f;
    for (int i0 = 0; i0 < nq; i0 += kOther) {
      __syncthreads();
      load_rows<T>(a.q, h, a.q0[f] + i0, nq - i0, kOther, a.D, qs);
      load_rows<T>(a.dout, h, a.q0[f] + i0, nq - i0, kOther, a.D, gs);
      __syncthreads();
      for (int x = 0; x < 4; ++x) {
        const int i = i0 + c + 8 * x, qrow = a.q0[f] + i;
        float p = 0.0f, ds = 0.0f, grad;
        if (visible(a, f, i, j, nq, nk)) {
          const long long at = static_cast<long long>(h) * a.queries + qrow;
          const float s = score(a, dot_of(ks[r], qs[c + 8 * x], a.D), slope, a.qpos + qrow * a.qpos_stride,
                                a.kpos + krow * a.kpos_stride, &grad);
          p = expf(s - a.lse[at]);
          ds = p * (dot_of(vs[r], gs[c + 8 * x], a.D) - a.delta[at]) * grad;
        }
        ps[r][c + 8 * x] = p;
        dss[r][c + 8 * x] = ds;
      }
      __syncwarp();
      for (int i = 0; i < kOther; ++i)
        for (int d = 0; d < 16; ++d)
          if (c + 8 * d < a.D) {
            dv[d] = fmaf(ps[r][i], gs[i][c + 8 * d], dv[d]);
            dk[d] = fmaf(dss[r][i], qs[i][c + 8 * d], dk[d]);
          }
    }
  }
  if (j < nk) {
    T* ok = reinterpret_cast<T*>(a.dk.data + krow * a.dk.row + g * a.dk.head);
    T* ov = reinterpret_cast<T*>(a.dv.data + krow * a.dv.row + g * a.dv.head);
    for (int d = 0; d < 16; ++d)
      if (c + 8 * d < a.D) {
        ok[c + 8 * d] = Pack<T>::one(dk[d] * a.scale);
        ov[c + 8 * d] = Pack<T>::one(dv[d]);
      }
  }
  allow_next_grid();
}

// ------------------------------------------------------------ host side

View view_of(const pv_heads* h) { return View{static_cast<char*>(h->data), h->row_stride * 2, h->head_stride * 2}; }

int check_params(const pv_attention_params* p, int* dev, const void* some) {
  if (!p || (p->dtype != PV_BF16 && p->dtype != PV_F16)) return PV_ERR_INVALID;
  int st;
  if ((st = check_offsets(p->q_offsets, p->frames)) != PV_OK || (st = check_offsets(p->k_offsets, p->frames)) != PV_OK)
    return st;
  if (p->q_heads < 1 || p->k_heads < 1 || p->q_heads > 4096 || p->q_heads % p->k_heads) return PV_ERR_INVALID;
  if (p->head_dim < 8 || p->head_dim > 128 || p->head_dim % 8) return PV_ERR_INVALID;
  if (!(p->scale > 0.0f) || !std::isfinite(p->scale) || !(p->cap >= 0.0f) || !std::isfinite(p->cap)) return PV_ERR_INVALID;
  if (p->prefix)
    for (int b = 0; b < p->frames; ++b)
      if (p->prefix[b] < 0) return PV_ERR_INVALID;
  const int64_t nq = p->q_offsets[p->frames], nk = p->k_offsets[p->frames];
  *dev = some ? device_of(some) : -1;
  if (*dev < 0) return PV_ERR_INVALID;
  if (p->slopes) {
    if (p->axes < 1 || p->axes > 3 || p->q_position_stride < p->axes || p->k_position_stride < p->axes)
      return PV_ERR_INVALID;
    if (!aligned(p->slopes, 4) || device_of(p->slopes) != *dev) return PV_ERR_INVALID;
    if (nq && (!p->q_positions || !aligned(p->q_positions, 4) || device_of(p->q_positions) != *dev)) return PV_ERR_INVALID;
    if (nk && (!p->k_positions || !aligned(p->k_positions, 4) || device_of(p->k_positions) != *dev)) return PV_ERR_INVALID;
  }
  return PV_OK;
}

AttnArgs args_of(const pv_attention_params* p) {
  AttnArgs a{};
  a.slopes = p->slopes;
  a.qpos = p->q_positions;
  a.kpos = p->k_positions;
  a.qpos_stride = p->q_position_stride;
  a.kpos_stride = p->k_position_stride;
  a.scale = p->scale;
  a.cap = p->cap;
  a.axes = p->slopes ? p->axes : 0;
  a.causal = p->causal != 0;
  a.H = p->q_heads;
  a.Hk = p->k_heads;
  a.G = p->q_heads / p->k_heads;
  a.D = p->head_dim;
  a.Dn = (a.D + 15) / 16 * 16;
  a.frames = p->frames;
  a.queries = static_cast<int>(p->q_offsets[p->frames]);
  a.keys = static_cast<int>(p->k_offsets[p->frames]);
  for (int b = 0; b < p->frames; ++b) {
    a.q0[b + 1] = static_cast<int>(p->q_offsets[b + 1]);
    a.k0[b + 1] = static_cast<int>(p->k_offsets[b + 1]);
    a.prefix[b] = p->prefix ? static_cast<int>(std::min<int64_t>(p->prefix[b], a.k0[b + 1] - a.k0[b])) : 0;
  }
  return a;
}

// Heads that share a tile of rows: the largest power of two of those that share
// a key head.
int pack_of(int G) {
  int p = 0;
  while (p < 7 && G % (2 << p) == 0) ++p;
  return p;
}

// How many key tiles a block takes.  A block's time goes by its key tiles, and
// the blocks run in rounds of one a multiprocessor: of the counts that leave
// some `kLeast` tiles a block, the one with the shortest rounds, where a join
// and its second launch are worth `kJoin` tiles.
int chunk_of(const AttnArgs& a, int heads, int sms) {
  constexpr int kLeast = 2, kJoin = 4;
  int most = 1;
  for (int f = 0; f < a.frames; ++f) most = std::max(most, (a.k0[f + 1] - a.k0[f] + 127) / 128);
  auto cost = [&](int chunk) {
    int64_t blocks = 0;
    for (int f = 0; f < a.frames; ++f) {
      const int64_t rows = static_cast<int64_t>(a.q0[f + 1] - a.q0[f]) << a.pack_log2;
      const int tiles = (a.k0[f + 1] - a.k0[f] + 127) / 128;
      blocks += (rows + 255) / 256 * std::max(1, (tiles + chunk - 1) / chunk);
    }
    return (blocks * heads + sms - 1) / sms * (chunk + 1) + (chunk < most ? kJoin : 0);
  };
  int best = most;
  int64_t least = cost(most);
  for (int parts = 2; parts <= 64 && (most + parts - 1) / parts >= kLeast; ++parts) {
    const int chunk = (most + parts - 1) / parts;
    const int64_t c = cost(chunk);
    if (c < least) {
      least = c;
      best = chunk;
    }
  }
  return best;
}

// Tiles of `own` rows along frames with row offsets `off`; how many there are.
int tiles_of(AttnArgs& a, const int* off, int own) {
  for (int b = 0; b < a.frames; ++b) a.tile0[b + 1] = a.tile0[b] + (off[b + 1] - off[b] + own - 1) / own;
  return a.tile0[a.frames];
}

template <typename K>
int launch(K kernel, dim3 grid, size_t smem, const AttnArgs& a, pv_stream_t stream) {
  if (grid.x == 0 || grid.y == 0) return PV_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess) {
    cudaGetLastError();
    return PV_ERR_CUDA;
  }
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return PV_ERR_CUDA;
  }
  return PV_OK;
}

template <typename T>
int backward(AttnArgs& a, pv_stream_t stream) {
  const size_t smem = sizeof(float) * kPad * 2 * (kOwn + kOther);
  const long long rows = static_cast<long long>(a.queries) * a.H;
  int st = launch(pv_attn_delta_kernel<T>, dim3(static_cast<unsigned int>((rows * 32 + kThreads - 1) / kThreads)), 0, a, stream);
  if (st != PV_OK) return st;
  int n = tiles_of(a, a.q0, kOwn);
  if ((st = launch(pv_attn_dq_kernel<T>, dim3(n, a.H), smem, a, stream)) != PV_OK) return st;
  n = tiles_of(a, a.k0, kOwn);
  return launch(pv_attn_dkv_kernel<T>, dim3(n, a.Hk), smem, a, stream);
}

}  // namespace

int pvs::make_map(CUtensorMap* map, const View& v, int dtype, int D, int heads, int pack, int64_t total, int rows) {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> encode{nullptr};
  auto fn = encode.load();
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult got;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &got) != cudaSuccess ||
        got != cudaDriverEntryPointSuccess || !p) {
      cudaGetLastError();
      return PV_ERR_CUDA;
    }
    fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    encode.store(fn);
  }
  // A head stride of zero is one head that every head reads.
  const cuuint64_t head = v.head ? v.head : 16;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(v.head ? pack : 1),
                              static_cast<cuuint64_t>(v.head ? heads / pack : 1), static_cast<cuuint64_t>(total)};
  const cuuint64_t strides[3] = {head, head * pack, static_cast<cuuint64_t>(v.row ? v.row : 16)};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(pack), 1, static_cast<cuuint32_t>(rows)};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, dtype == PV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, v.data,
                        dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PV_OK : PV_ERR_INVALID;
}

extern "C" int pv_attention(const pv_attention_params* params, const pv_heads* q, const pv_heads* k, const pv_heads* v,
                            const pv_heads* out, float* lse, pv_stream_t stream) {
  if (!params || !params->q_offsets || !out || !q) return PV_ERR_INVALID;
  int dev = 0, st;
  if ((st = check_offsets(params->q_offsets, params->frames)) != PV_OK) return st;
  const int64_t nq = params->q_offsets[params->frames];
  if (nq == 0 && !out->data) return PV_OK;
  if ((st = check_params(params, &dev, out->data)) != PV_OK) return st;
  const int64_t nk = params->k_offsets[params->frames];
  for (const pv_heads* h : {q, out})
    if ((st = check_heads(h, nq, params->q_heads, 2, dev)) != PV_OK) return st;
  for (const pv_heads* h : {k, v})
    if ((st = check_heads(h, nk, params->k_heads, 2, dev)) != PV_OK) return st;
  if (lse && (!aligned(lse, 4) || device_of(lse) != dev)) return PV_ERR_INVALID;
  if (nq == 0) return PV_OK;
  DeviceScope scope(dev);
  if (!scope.ok()) return PV_ERR_CUDA;
  AttnArgs a = args_of(params);
  a.q = view_of(q);
  a.k = view_of(k);
  a.v = view_of(v);
  a.o = view_of(out);
  a.lse = lse;
  a.pack_log2 = a.q.head ? pack_of(a.G) : 0;
  const int heads = a.H >> a.pack_log2;
  const int sms = sm_count(dev);
  if (sms < 1) return PV_ERR_CUDA;
  a.chunk = chunk_of(a, heads, sms);
  int parts = 1;
  for (int f = 0; f < a.frames; ++f) {
    const int rows = static_cast<int>(((static_cast<int64_t>(a.q0[f + 1] - a.q0[f]) << a.pack_log2) + 255) / 256);
    const int splits = std::max(1, ((a.k0[f + 1] - a.k0[f] + 127) / 128 + a.chunk - 1) / a.chunk);
    a.tile0[f + 1] = a.tile0[f] + rows * splits;
    parts = std::max(parts, splits);
  }
  Scratch scratch;
  if (parts > 1) {
    const size_t rows = static_cast<size_t>(parts) * nq * a.H;
    if ((st = scratch.open(dev, stream, kPlain, rows * (sizeof(float) * a.D + sizeof(float2)))) != PV_OK) return st;
    a.part_o = static_cast<float*>(scratch.body());
    a.part_ml = reinterpret_cast<float2*>(a.part_o + rows * a.D);
  }
  AttnMaps m;
  if ((st = make_map(&m.q, a.q, params->dtype, a.D, a.H, 1 << a.pack_log2, nq, 128 >> a.pack_log2)) != PV_OK) return st;
  if (nk == 0) {
    m.k = m.v = m.q;  // no key is loaded
  } else if ((st = make_map(&m.k, a.k, params->dtype, a.D, a.Hk, 1, nk, 128)) != PV_OK ||
             (st = make_map(&m.v, a.v, params->dtype, a.D, a.Hk, 1, nk, 128)) != PV_OK) {
    return st;
  }
  return attn_forward(a, params->dtype, m, dim3(a.tile0[a.frames], heads), reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int pv_attention_backward(const pv_attention_params* params, const pv_heads* dout, const pv_heads* q,
                                     const pv_heads* k, const pv_heads* v, const pv_heads* out, const float* lse,
                                     const pv_heads* dq, const pv_heads* dk, const pv_heads* dv, pv_stream_t stream) {
  if (!params || !params->q_offsets || !params->k_offsets || !dq || !dk || !dv) return PV_ERR_INVALID;
  int dev = 0, st;
  if ((st = check_offsets(params->q_offsets, params->frames)) != PV_OK ||
      (st = check_offsets(params->k_offsets, params->frames)) != PV_OK)
    return st;
  const int64_t nq = params->q_offsets[params->frames], nk = params->k_offsets[params->frames];
  if (nq == 0 && nk == 0) return PV_OK;
  if ((st = check_params(params, &dev, nq ? dq->data : dk->data)) != PV_OK) return st;
  for (const pv_heads* h : {dout, q, out, dq})
    if ((st = check_heads(h, nq, params->q_heads, 2, dev)) != PV_OK) return st;
  for (const pv_heads* h : {k, v, dk, dv})
    if ((st = check_heads(h, nk, params->k_heads, 2, dev)) != PV_OK) return st;
  if (nq && (!lse || !aligned(lse, 4) || device_of(lse) != dev)) return PV_ERR_INVALID;
  DeviceScope scope(dev);
  if (!scope.ok()) return PV_ERR_CUDA;
  AttnArgs a = args_of(params);
  a.dout = view_of(dout);
  a.q = view_of(q);
  a.k = view_of(k);
  a.v = view_of(v);
  a.o = view_of(out);
  a.lse = const_cast<float*>(lse);
  a.dq = view_of(dq);
  a.dk = view_of(dk);
  a.dv = view_of(dv);
  Scratch scratch;
  if ((st = scratch.open(dev, stream, kPlain, sizeof(float) * static_cast<size_t>(nq) * a.H)) != PV_OK) return st;
  a.delta = static_cast<float*>(scratch.body());
  return params->dtype == PV_BF16 ? backward<__nv_bfloat16>(a, stream) : backward<__half>(a, stream);
}
