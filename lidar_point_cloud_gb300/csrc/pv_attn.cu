// Attention inside frames and its backward pass (pv_attention,
// pv_attention_backward in pv.h).
//
//   s = scale q.k;  t = cap tanh(s / cap) (or s);  u = t - slope * distance;
//   p = exp(u - lse), lse = log sum of exp(u) over the visible keys;  o = p v.
//   dv = p^T do;  du = p (do.v - delta), delta = do.o;
//   ds = du (1 - (t / cap)^2) scale;  dq = ds k;  dk = ds^T q.
//
// This file: argument checks, tensor maps, how the work is cut.  The kernels are
// in pv_attn_fwd.cu and pv_attn_bwd.cu.

#include "pv_attn.cuh"

#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <initializer_list>
#include <utility>
#include <vector>

namespace {

using namespace pvs;

View view_of(const pv_heads* h) { return View{static_cast<char*>(h->data), h->row_stride * 2, h->head_stride * 2}; }

int check_params(const pv_attention_params* p, int* dev, const void* some) {
  if (!p || (p->dtype != PV_BF16 && p->dtype != PV_F16)) return PV_ERR_INVALID;
  int st;
  if ((st = check_offsets(p->q_offsets, p->frames)) != PV_OK || (st = check_offsets(p->k_offsets, p->frames)) != PV_OK)
    return st;
  if (p->q_offsets[p->frames] > PV_ATTENTION_MAX_ROWS || p->k_offsets[p->frames] > PV_ATTENTION_MAX_ROWS)
    return PV_ERR_TOO_LARGE;
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

// Tiles of rows are loaded by a tensor map, whose rows lie apart: a row stride of 0 (one
// row seen as many) is for a single row only.
int check_tiles(const pv_heads* h, int64_t rows, int heads, int dev) {
  const int st = check_heads(h, rows, heads, 2, dev);
  return st == PV_OK && rows > 1 && h->row_stride == 0 ? PV_ERR_INVALID : st;
}

AttnArgs args_of(const pv_attention_params* p) {
  AttnArgs a{};
  a.slopes = p->slopes;
  a.qpos = p->q_positions;
  a.kpos = p->k_positions;
  a.qpos_stride = p->q_position_stride;
  a.kpos_stride = p->k_position_stride;
  a.scale = p->scale;
  // Caps past 1e34 or below 1e-30 cap like these (and their products with the scale and
  // with log2(e) stay finite).
  a.cap = p->cap > 0.0f ? std::min(std::max(p->cap, 1e-30f), 1e34f) : 0.0f;
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

constexpr double kBlock = 2.0;  // what a block needs to begin and end, in key tiles

struct Jobs {
  int length;  // key tiles
  int64_t count;
};

// When the last of the blocks ends, one a multiprocessor, longest first.  Multiprocessors
// of equal load are one entry of a heap, so that a call of one frame costs a few steps.
double makespan(std::vector<Jobs>& jobs, std::vector<std::pair<double, int64_t>>& loads, int sms) {
  const auto later = [](const auto& x, const auto& y) { return x.first > y.first; };
  if (jobs.size() > 1)
    std::sort(jobs.begin(), jobs.end(), [](const Jobs& x, const Jobs& y) { return x.length > y.length; });
  loads.assign(1, {0.0, sms});
  double end = 0.0;
  for (const Jobs& job : jobs) {
    const double length = job.length + kBlock;
    int64_t left = job.count;
    const int64_t whole = left / sms;  // rounds that load every multiprocessor alike
    if (whole > 1) {
      for (auto& l : loads) end = std::max(end, l.first += (whole - 1) * length);
      left -= (whole - 1) * sms;
    }
    while (left > 0) {
      std::pop_heap(loads.begin(), loads.end(), later);
      auto& least = loads.back();
      const int64_t n = std::min(left, least.second);
      const std::pair<double, int64_t> now(least.first + length, n);
      if ((least.second -= n) == 0)
        loads.pop_back();
      else
        std::push_heap(loads.begin(), loads.end(), later);
      loads.push_back(now);
      std::push_heap(loads.begin(), loads.end(), later);
      end = std::max(end, now.first);
      left -= n;
    }
  }
  return end;
}

// How many key tiles a block takes: the count with the earliest end, in units of a key
// tile's time (some 1.7 us).  Keys cut into parts cost the parts' outputs (32-bit,
// written and read again, some 4 TB/s) and kJoin for one more launch.  A schedule is played
// through only while its least possible end (all multiprocessors busy throughout, or the
// longest block alone) is below the best found, the likeliest first: a few of the list.
int chunk_of(const AttnArgs& a, int heads, int sms) {
  constexpr double kJoin = 2.0, kBytes = 6.8e6;
  constexpr int kParts[] = {1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 12, 14, 16, 18, 20, 24, 28, 32, 40, 48, 64};
  constexpr int kTries = sizeof(kParts) / sizeof(kParts[0]);
  int rows[PV_MAX_FRAMES], tiles[PV_MAX_FRAMES];  // blocks' rows of all heads, key tiles
  int most = 1, frames = 0;
  int64_t work = 0, blocks = 0;
  for (int f = 0; f < a.frames; ++f) {
    const int64_t r = ((static_cast<int64_t>(a.q0[f + 1] - a.q0[f]) << a.pack_log2) + 255) / 256 * heads;
    const int t = (a.k0[f + 1] - a.k0[f] + 127) / 128;
    most = std::max(most, t);
    work += r * t;
    blocks += r;
    // With many blocks the rounds blur; with much work nothing is left to be won.
    if (blocks >= 4 * static_cast<int64_t>(sms)) continue;
    if (r && t) rows[frames] = static_cast<int>(r), tiles[frames++] = t;
  }
  if (blocks >= 4 * static_cast<int64_t>(sms) || !frames) return most;
  struct Try {
    double least;
    int chunk;
  } tries[kTries];
  int n = 0;
  auto extra = [&](int chunk) {
    const int parts = (most + chunk - 1) / chunk;
    return parts > 1 ? kJoin + 8.0 * parts * a.queries * a.H * a.D / kBytes : 0.0;
  };
  for (int parts : kParts) {
    if (parts > most) break;
    const int chunk = (most + parts - 1) / parts;
    if (n && tries[n - 1].chunk == chunk) continue;
    int64_t count = 0;
    for (int f = 0; f < frames; ++f) count += static_cast<int64_t>(rows[f]) * ((tiles[f] + chunk - 1) / chunk);
    const double even = (static_cast<double>(work) + count * kBlock) / sms;
    tries[n++] = {std::max(even, chunk + kBlock) + extra(chunk), chunk};
  }
  std::stable_sort(tries, tries + n, [](const Try& x, const Try& y) { return x.least < y.least; });
  std::vector<Jobs> jobs;
  std::vector<std::pair<double, int64_t>> loads;
  jobs.reserve(2 * frames);
  loads.reserve(32);
  int best = most;
  double least = INFINITY;
  for (int i = 0; i < n && tries[i].least < least; ++i) {
    const int chunk = tries[i].chunk;
    jobs.clear();
    for (int f = 0; f < frames; ++f) {
      if (tiles[f] / chunk) jobs.push_back({chunk, static_cast<int64_t>(rows[f]) * (tiles[f] / chunk)});
      if (tiles[f] % chunk) jobs.push_back({tiles[f] % chunk, rows[f]});
    }
    const double cost = makespan(jobs, loads, sms) + extra(chunk);
    if (cost < least) least = cost, best = chunk;
  }
  return best;
}

// The blocks' list: count(f) tiles of each frame, the frames in the order of the rows
// that their tiles walk (`walk`: the other side's row offsets), most first, so that
// the last blocks to start are short ones.  Returns how many tiles there are.
template <typename F>
int list_tiles(AttnArgs& a, const int* walk, F count) {
  for (int b = 0; b < a.frames; ++b) a.order[b] = static_cast<unsigned char>(b);
  std::stable_sort(a.order, a.order + a.frames, [&](unsigned char x, unsigned char y) {
    return walk[x + 1] - walk[x] > walk[y + 1] - walk[y];
  });
  int64_t n = 0;
  for (int i = 0; i < a.frames; ++i) {
    n += count(a.order[i]);
    a.tile0[i + 1] = static_cast<int>(n);
  }
  return n * a.heads < (int64_t(1) << 31) ? static_cast<int>(n) : -1;
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
  // A head stride of zero is one head that every head reads; a row stride of zero has one
  // row (check_tiles).
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
                            const pv_heads* out, float* lse, pv_stream_t stream) try {
  if (!params || !params->q_offsets || !out || !q) return PV_ERR_INVALID;
  int dev = 0, st;
  if ((st = check_offsets(params->q_offsets, params->frames)) != PV_OK) return st;
  const int64_t nq = params->q_offsets[params->frames];
  if (nq == 0 && !out->data) return PV_OK;
  if ((st = check_params(params, &dev, out->data)) != PV_OK) return st;
  const int64_t nk = params->k_offsets[params->frames];
  if ((st = check_tiles(q, nq, params->q_heads, dev)) != PV_OK ||
      (st = check_out_heads(out, nq, params->q_heads, 2, dev)) != PV_OK)
    return st;
  for (const pv_heads* h : {k, v})
    if ((st = check_tiles(h, nk, params->k_heads, dev)) != PV_OK) return st;
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
  a.heads = heads;
  const int tiles = list_tiles(a, a.k0, [&](int f) {
    const int64_t rows = ((static_cast<int64_t>(a.q0[f + 1] - a.q0[f]) << a.pack_log2) + 255) / 256;
    const int splits = std::max(1, ((a.k0[f + 1] - a.k0[f] + 127) / 128 + a.chunk - 1) / a.chunk);
    parts = std::max(parts, splits);
    return rows * splits;
  });
  if (tiles < 0) return PV_ERR_TOO_LARGE;
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
  const bool bf16 = params->dtype == PV_BF16;
  return (bf16 ? attn_forward_bf16 : attn_forward_half)(a, m, dim3(tiles * heads), reinterpret_cast<cudaStream_t>(stream));
} catch (...) {
  return caught();
}

extern "C" int pv_attention_backward(const pv_attention_params* params, const pv_heads* dout, const pv_heads* q,
                                     const pv_heads* k, const pv_heads* v, const pv_heads* out, const float* lse,
                                     const pv_heads* dq, const pv_heads* dk, const pv_heads* dv, pv_stream_t stream) try {
  if (!params || !params->q_offsets || !params->k_offsets || !dq || !dk || !dv) return PV_ERR_INVALID;
  int dev = 0, st;
  if ((st = check_offsets(params->q_offsets, params->frames)) != PV_OK ||
      (st = check_offsets(params->k_offsets, params->frames)) != PV_OK)
    return st;
  const int64_t nq = params->q_offsets[params->frames], nk = params->k_offsets[params->frames];
  if (nq == 0 && nk == 0) return PV_OK;
  if ((st = check_params(params, &dev, nq ? dq->data : dk->data)) != PV_OK) return st;
  for (const pv_heads* h : {dout, q})
    if ((st = check_tiles(h, nq, params->q_heads, dev)) != PV_OK) return st;
  for (const pv_heads* h : {k, v})
    if ((st = check_tiles(h, nk, params->k_heads, dev)) != PV_OK) return st;
  if ((st = check_heads(out, nq, params->q_heads, 2, dev)) != PV_OK ||
      (st = check_out_heads(dq, nq, params->q_heads, 2, dev)) != PV_OK)
    return st;
  for (const pv_heads* h : {dk, dv})
    if ((st = check_out_heads(h, nk, params->k_heads, 2, dev)) != PV_OK) return st;
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
  const int sms = sm_count(dev);
  if (sms < 1) return PV_ERR_CUDA;
  int64_t key_tiles = 0;
  for (int f = 0; f < a.frames; ++f) key_tiles += (a.k0[f + 1] - a.k0[f] + 127) / 128;
  // A key head's block walks the queries of all heads that share it: with few
  // blocks for the multiprocessors (under a causal mask of unequal length too) the
  // heads are cut into parts, joined by one more kernel.
  a.head_parts = 1;
  while (a.G % (2 * a.head_parts) == 0 && key_tiles * a.Hk * a.head_parts < 4 * sms) a.head_parts *= 2;
  Scratch scratch;
  // (One tile more than the rows: the last copy of a row of sides is a whole one too.)
  int64_t side_rows = 0;
  for (int f = 0; f < a.frames; ++f) {
    a.side0[f] = static_cast<int>(side_rows);
    side_rows += (a.q0[f + 1] - a.q0[f] + 3) / 4 * 4;
  }
  a.sides_row = side_rows + 128;
  const size_t sides = static_cast<size_t>(a.sides_row) * (2 * a.H + 3);
  const size_t parts = a.head_parts > 1 ? static_cast<size_t>(2) * a.head_parts * nk * a.Hk * a.D : 0;
  // Float16: the blocks that look for a frame's largest gradients and values, and what they leave.
  const bool bf16 = params->dtype == PV_BF16, range = !bf16 && nq && nk;
  if (range) {
    int64_t most = 0;
    for (int f = 0; f < a.frames; ++f)
      most = std::max<int64_t>(most, static_cast<int64_t>(a.q0[f + 1] - a.q0[f]) * a.H + static_cast<int64_t>(a.k0[f + 1] - a.k0[f]) * a.Hk);
    a.norm_parts = static_cast<int>(std::min<int64_t>(std::max(1, std::min(256, 4 * sms / a.frames)), (most + 63) / 64));
  }
  const size_t ups = range ? static_cast<size_t>(a.frames) * 2 * (a.norm_parts + 1) : 0;
  if ((st = scratch.open(dev, stream, kPlain, sizeof(float) * (sides + parts + ups))) != PV_OK) return st;
  a.sides = static_cast<float*>(scratch.body());
  a.part_o = a.sides + sides;
  if (range) {
    a.norms = reinterpret_cast<float2*>(a.part_o + parts);
    a.up = a.norms + static_cast<size_t>(a.frames) * a.norm_parts;
    a.norms_done = static_cast<unsigned int*>(scratch.head()) + kHeadFrames;
  }
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  AttnMaps m{};
  if (nq && ((st = make_map(&m.q, a.q, params->dtype, a.D, a.H, 1, nq, 128)) != PV_OK ||
             (st = make_map(&m.dout, a.dout, params->dtype, a.D, a.H, 1, nq, 128)) != PV_OK))
    return st;
  if (nk && ((st = make_map(&m.k, a.k, params->dtype, a.D, a.Hk, 1, nk, 128)) != PV_OK ||
             (st = make_map(&m.v, a.v, params->dtype, a.D, a.Hk, 1, nk, 128)) != PV_OK))
    return st;
  if (!nk) m.k = m.v = m.q;  // nothing is loaded through these
  if (!nq) m.q = m.dout = m.k;
  AttnArgs b = a;
  a.heads = a.H;
  b.heads = a.Hk * a.head_parts;
  const int q_tiles = list_tiles(a, a.k0, [&](int f) { return (a.q0[f + 1] - a.q0[f] + 127) / 128; });
  const int k_tiles = list_tiles(b, a.q0, [&](int f) { return (a.k0[f + 1] - a.k0[f] + 127) / 128; });
  if (q_tiles < 0 || k_tiles < 0) return PV_ERR_TOO_LARGE;
  if (range && (st = attn_backward_up_half(a, cs)) != PV_OK) return st;
  if ((st = (bf16 ? attn_backward_dq_bf16 : attn_backward_dq_half)(a, m, dim3(q_tiles * a.heads), cs)) != PV_OK) return st;
  return (bf16 ? attn_backward_dkv_bf16 : attn_backward_dkv_half)(b, m, dim3(k_tiles * b.heads), cs);
} catch (...) {
  return caught();
}
