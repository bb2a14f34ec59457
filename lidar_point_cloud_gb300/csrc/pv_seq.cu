// Host side shared by the voxel-token operators: argument checks and their
// per-(device, stream) scratch (see pv_seq.cuh).

#include "pv_seq.cuh"

#include <atomic>
#include <list>
#include <map>
#include <memory>
#include <new>
#include <tuple>

namespace pvs {

struct SeqSpace {
  std::mutex mu;
  int device = 0;
  unsigned char* mem = nullptr;
  size_t cap = 0;
  // Of a captured call: which capture's, and whether its graph still is.
  ScratchKind kind = kPlain;
  unsigned long long capture = 0;
  pv_stream_t stream = nullptr;
  std::atomic<bool> owned{false};
};

namespace {
std::mutex g_seq_mu;
std::map<std::tuple<int, pv_stream_t, int>, SeqSpace*> g_seq;
std::list<SeqSpace*> g_captured;

// Runs when the last graph that owns the space is gone (no CUDA calls are allowed here).
void CUDART_CB give_back(void* space) { static_cast<SeqSpace*>(space)->owned.store(false); }

// Lets this thread allocate while one of its streams is captured.
class RelaxedCapture {
 public:
  RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode_); }
  ~RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode_); }

 private:
  cudaStreamCaptureMode mode_ = cudaStreamCaptureModeRelaxed;
};

// Zeroed memory, now: by a stream that no capture sees.
int zeroed_now(void** mem, size_t bytes) {
  if (cudaMalloc(mem, bytes) != cudaSuccess) {
    cudaGetLastError();
    return PV_ERR_ALLOC;
  }
  cudaStream_t s = nullptr;
  bool ok = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) == cudaSuccess;
  ok = ok && cudaMemsetAsync(*mem, 0, bytes, s) == cudaSuccess && cudaStreamSynchronize(s) == cudaSuccess;
  if (s) cudaStreamDestroy(s);
  if (!ok) {
    cudaGetLastError();
    cudaFree(*mem);
    return PV_ERR_CUDA;
  }
  return PV_OK;
}
std::mutex g_sms_mu;
int g_sms[64];
}  // namespace

int device_of(const void* ptr) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, ptr) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged ? at.device : -1;
}

int sm_count(int dev) {
  if (dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lk(g_sms_mu);
  if (!g_sms[dev] && cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    g_sms[dev] = 0;
  }
  return g_sms[dev];
}

int caught() noexcept {
  try {
    throw;
  } catch (const std::bad_alloc&) {
    return PV_ERR_ALLOC;
  } catch (...) {
    return PV_ERR_CUDA;
  }
}

int check_offsets(const int64_t* off, int n) {
  if (!off || n < 1 || n > PV_MAX_FRAMES || off[0] != 0) return PV_ERR_INVALID;
  for (int i = 0; i < n; ++i)
    if (off[i + 1] < off[i]) return PV_ERR_INVALID;
  return off[n] < (int64_t(1) << 31) ? PV_OK : PV_ERR_INVALID;
}

int check_heads(const pv_heads* h, int64_t rows, int heads, int elem, int dev) {
  if (!h) return PV_ERR_INVALID;
  if (rows == 0 || heads == 0) return PV_OK;
  if (!h->data || !aligned(h->data, 16) || h->row_stride < 0 || h->head_stride < 0) return PV_ERR_INVALID;
  if (h->row_stride * elem % 16 || h->head_stride * elem % 16) return PV_ERR_INVALID;
  return device_of(h->data) == dev ? PV_OK : PV_ERR_INVALID;
}

int check_out_heads(const pv_heads* h, int64_t rows, int heads, int elem, int dev) {
  const int st = check_heads(h, rows, heads, elem, dev);
  if (st != PV_OK || rows == 0) return st;
  return (rows > 1 && h->row_stride == 0) || (heads > 1 && h->head_stride == 0) ? PV_ERR_INVALID : PV_OK;
}

int Scratch::open(int dev, pv_stream_t stream, ScratchKind kind, size_t bytes) {
  const size_t need = round_up(kHead + bytes, size_t(1) << 16);
  cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
  unsigned long long capture = 0;
  cudaGraph_t graph = nullptr;
  // (Refused for the legacy stream beside a capture: the launch will be, too.)
  if (cudaStreamGetCaptureInfo(reinterpret_cast<cudaStream_t>(stream), &capturing, &capture, &graph, nullptr, nullptr,
                               nullptr) != cudaSuccess)
    cudaGetLastError();
  else if (capturing == cudaStreamCaptureStatusActive)
    return open_captured(dev, stream, kind, need, capture, graph);
  {
    std::lock_guard<std::mutex> lk(g_seq_mu);
    SeqSpace*& sp = g_seq[std::make_tuple(dev, stream, static_cast<int>(kind))];
    if (!sp) sp = new SeqSpace();
    sp->device = dev;
    sp->mu.lock();
    sp_ = sp;
  }
  if (sp_->cap >= need) return PV_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (sp_->mem && cudaStreamSynchronize(s) != cudaSuccess) return PV_ERR_CUDA;
  if (sp_->mem) cudaFree(sp_->mem);
  sp_->mem = nullptr;
  sp_->cap = 0;
  void* mem = nullptr;
  if (cudaMalloc(&mem, need) != cudaSuccess) {
    cudaGetLastError();
    return PV_ERR_ALLOC;
  }
  if (cudaMemsetAsync(mem, 0, need, s) != cudaSuccess) {
    cudaGetLastError();
    cudaFree(mem);
    return PV_ERR_CUDA;
  }
  sp_->mem = static_cast<unsigned char*>(mem);
  sp_->cap = need;
  return PV_OK;
}

int Scratch::open_captured(int dev, pv_stream_t stream, ScratchKind kind, size_t need, unsigned long long capture,
                           cudaGraph_t graph) {
  std::lock_guard<std::mutex> lk(g_seq_mu);
  SeqSpace* idle = nullptr;
  for (SeqSpace* sp : g_captured) {
    if (sp->device != dev || sp->kind != kind || sp->cap < need) continue;
    if (!sp->owned.load()) {
      if (!idle || sp->cap < idle->cap) idle = sp;
    } else if (sp->capture == capture && sp->stream == stream) {
      sp->mu.lock();
      sp_ = sp;
      return PV_OK;
    }
  }
  RelaxedCapture relaxed;
  if (!idle) {
    auto space = std::make_unique<SeqSpace>();
    g_captured.push_back(space.get());
    void* mem = nullptr;
    const int st = zeroed_now(&mem, need);
    if (st != PV_OK) {
      g_captured.pop_back();
      return st;
    }
    idle = space.release();
    idle->device = dev;
    idle->mem = static_cast<unsigned char*>(mem);
    idle->cap = need;
    idle->kind = kind;
  }
  cudaUserObject_t owner = nullptr;
  if (cudaUserObjectCreate(&owner, idle, give_back, 1, cudaUserObjectNoDestructorSync) != cudaSuccess) {
    cudaGetLastError();
    return PV_ERR_CUDA;
  }
  idle->owned.store(true);
  if (cudaGraphRetainUserObject(graph, owner, 1, cudaGraphUserObjectMove) != cudaSuccess) {
    cudaGetLastError();
    cudaUserObjectRelease(owner, 1);  // gives it back
    return PV_ERR_CUDA;
  }
  idle->capture = capture;
  idle->stream = stream;
  idle->mu.lock();
  sp_ = idle;
  return PV_OK;
}

Scratch::~Scratch() {
  if (sp_) sp_->mu.unlock();
}

void* Scratch::head() const { return sp_->mem; }

int release_scratch() {
  std::lock_guard<std::mutex> lk(g_seq_mu);
  int st = PV_OK;
  for (auto& kv : g_seq) {
    SeqSpace* sp = kv.second;
    if (!sp) continue;  // the host had no memory for it
    DeviceScope scope(sp->device);
    if (!scope.ok() || cudaDeviceSynchronize() != cudaSuccess) st = PV_ERR_CUDA;
    sp->mu.lock();  // wait for a call that is still enqueueing
    sp->mu.unlock();
    cudaFree(sp->mem);
    delete sp;
  }
  g_seq.clear();
  // (What a graph owns stays with it.  A captured call enqueues while it owns its space.)
  g_captured.remove_if([&](SeqSpace* sp) {
    if (sp->owned.load()) return false;
    DeviceScope scope(sp->device);
    if (!scope.ok() || cudaDeviceSynchronize() != cudaSuccess) st = PV_ERR_CUDA;
    cudaFree(sp->mem);
    delete sp;
    return true;
  });
  return st;
}

}  // namespace pvs
