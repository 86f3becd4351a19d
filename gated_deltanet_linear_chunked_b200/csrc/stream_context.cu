// stream_context.cu -- what the library keeps per (device, stream): an error word
// and the scratch that calls pass between their kernels.  Host code only.
//
// The first call on a stream allocates its error word and scratch, later calls
// reuse them, and a larger problem replaces the scratch with a larger one.  Calls on
// one stream are ordered, so they can share the scratch; calls on different streams
// never share anything.
//
// Two scratches, by who may still name one that a larger call replaces:
//   * the scan's and its gradients'.  A call that is being captured uses it where it
//     is large enough, so a replaced one may live on in a graph and is kept until
//     gdn_workspace_release.  One model has one shape of them.
//   * the operators'.  Their captured calls take an allocation of the graph's own, so
//     a replaced one is named by work already on the stream and by nothing else: it is
//     freed in stream order.  Their sizes follow prompts and batches; kept, every
//     length of a run would leave its buffer behind.
//
// A call made while its stream is being captured, on a stream with no context yet or
// with too small a scratch, cannot allocate outside the graph: it gets none here and
// allocates stream-ordered (captured as graph memory nodes), and reports to the
// device-wide error word.
#include <cuda_runtime.h>

#include <cstdint>
#include <functional>
#include <mutex>
#include <new>
#include <thread>
#include <vector>

#include "gdn_internal.h"

namespace gdn {
namespace {

struct Buffer {
  void* p = nullptr;
  size_t bytes = 0;
};

struct StreamCtx {
  int dev;
  cudaStream_t stream;
  size_t thread;  // owning host thread for the per-thread default stream, else 0
  // Guards what follows, and is held over the launches of a call that passes scratch
  // between them: two threads that call on one stream share its scratch, so their
  // launches must not interleave.  Calls on other streams have their own.
  std::mutex mu;
  unsigned int* err = nullptr;  // error word of this stream's calls
  Buffer scan, op;
};

// Entries stay for the life of the process (a thread may be waiting for one's lock);
// gdn_workspace_release empties them.  Lock order: an entry's, then this one.
std::mutex g_ctx_mu;
std::vector<StreamCtx*> g_ctx;
struct Retired {
  int dev;
  void* p;
};
std::vector<Retired> g_retired;  // the scan's scratch buffers replaced by larger ones

size_t thread_key(cudaStream_t s) {
  if (s != cudaStreamPerThread) return 0;
  return std::hash<std::thread::id>()(std::this_thread::get_id()) | 1u;
}

bool capturing(cudaStream_t s) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing(s, &cs);
  if (e != cudaSuccess) {  // e.g. the legacy stream while another stream captures
    cudaGetLastError();
    return true;
  }
  return cs != cudaStreamCaptureStatusNone;
}

// The entry of (dev, s), made if there is none (unless only looked for); nullptr if there
// is none or the host has no memory.
StreamCtx* entry(int dev, cudaStream_t s, bool make = true) {
  const size_t tk = thread_key(s);
  std::lock_guard<std::mutex> lock(g_ctx_mu);
  for (StreamCtx* x : g_ctx)
    if (x->dev == dev && x->stream == s && x->thread == tk) return x;
  StreamCtx* c = make ? new (std::nothrow) StreamCtx{dev, s, tk} : nullptr;
  if (c) g_ctx.push_back(c);
  return c;
}

gdn_status failed() {
  cudaGetLastError();
  return GDN_ERR_CUDA;
}

// A buffer of at least `bytes` in place of a smaller one.
gdn_status grow_scan(StreamCtx* c, size_t bytes) {
  const size_t grain = size_t(2) << 20;
  const size_t n = (bytes + grain - 1) / grain * grain;
  void* p = nullptr;
  if (cudaMalloc(&p, n) != cudaSuccess) return failed();
  if (c->scan.p) {
    std::lock_guard<std::mutex> lock(g_ctx_mu);
    g_retired.push_back({c->dev, c->scan.p});
  }
  c->scan = {p, n};
  return GDN_OK;
}
gdn_status grow_op(StreamCtx* c, size_t bytes) {
  // a quarter more than asked for, so that lengths that creep up do not allocate
  // every time
  const size_t grain = size_t(2) << 20;
  const size_t n = (bytes + bytes / 4 + grain - 1) / grain * grain;
  if (c->op.p && cudaFreeAsync(c->op.p, c->stream) != cudaSuccess) return failed();
  c->op = {};
  void* p = nullptr;
  if (cudaMallocAsync(&p, n, c->stream) != cudaSuccess) return failed();
  c->op = {p, n};
  return GDN_OK;
}

// The error word and one scratch of an entry whose lock is held, allocated or grown to
// at least `bytes` as needed.  Sets them to nullptr (and returns GDN_OK) when the
// stream is being captured and the entry cannot serve the call as it is.
gdn_status provide(StreamCtx* c, size_t bytes, Buffer StreamCtx::*which, unsigned int** err, void** ws) {
  *err = nullptr;
  *ws = nullptr;
  if (!(c->err && (c->*which).bytes >= bytes)) {
    if (capturing(c->stream)) return GDN_OK;
    if (!c->err) {
      void* p = nullptr;
      if (cudaMalloc(&p, 256) != cudaSuccess) return failed();
      if (cudaMemsetAsync(p, 0, 256, c->stream) != cudaSuccess) {
        cudaFree(p);
        return failed();
      }
      c->err = static_cast<unsigned int*>(p);
    }
    if (bytes > (c->*which).bytes) {
      const gdn_status st = which == &StreamCtx::op ? grow_op(c, bytes) : grow_scan(c, bytes);
      if (st != GDN_OK) return st;
    }
  }
  *err = c->err;
  *ws = (c->*which).p;
  return GDN_OK;
}

// The device-wide error word where the stream has none.
gdn_status some_error_word(unsigned int** err) {
  return *err || current_error_word(err) == cudaSuccess ? GDN_OK : failed();
}

}  // namespace

gdn_status scan_scratch(int dev, cudaStream_t s, size_t bytes, unsigned int** err, void** ws,
                        std::unique_lock<std::mutex>* launching) {
  StreamCtx* c = entry(dev, s);
  if (!c) return GDN_ERR_CUDA;
  *launching = std::unique_lock<std::mutex>(c->mu);
  const gdn_status st = provide(c, bytes, &StreamCtx::scan, err, ws);
  return st != GDN_OK ? st : some_error_word(err);
}

gdn_status op_scratch(int dev, cudaStream_t s, size_t bytes, unsigned int** err, OpScratch* sc) {
  StreamCtx* c = entry(dev, s);
  if (!c) return GDN_ERR_CUDA;
  sc->stream = s;
  sc->launching = std::unique_lock<std::mutex>(c->mu);
  sc->captured = bytes > 0 && capturing(s);
  gdn_status st = provide(c, sc->captured ? 0 : bytes, &StreamCtx::op, err, &sc->p);
  if (st == GDN_OK) st = some_error_word(err);
  if (st != GDN_OK || !sc->captured) return st;
  return cudaMallocAsync(&sc->p, bytes, s) == cudaSuccess ? GDN_OK : failed();
}

cudaError_t op_scratch_done(OpScratch* sc) {
  const cudaError_t e = sc->captured ? cudaFreeAsync(sc->p, sc->stream) : cudaSuccess;
  if (sc->launching.owns_lock()) sc->launching.unlock();
  return e;
}

unsigned int* own_error_word(int dev, cudaStream_t s) {
  StreamCtx* c = entry(dev, s, false);
  if (!c) return nullptr;
  std::lock_guard<std::mutex> lock(c->mu);
  return c->err;
}

gdn_status release_contexts(int dev, cudaError_t (*finish_work)()) {
  // every entry's lock, so that no call is between taking its scratch and its last
  // launch; entries made meanwhile are not this release's
  std::vector<StreamCtx*> mine;
  {
    std::lock_guard<std::mutex> lock(g_ctx_mu);
    for (StreamCtx* c : g_ctx)
      if (c->dev == dev) mine.push_back(c);
  }
  std::vector<std::unique_lock<std::mutex>> held;
  for (StreamCtx* c : mine) held.emplace_back(c->mu);
  std::vector<Retired> old;  // what is here now was named by launches that finish_work waits for
  {
    std::lock_guard<std::mutex> lock(g_ctx_mu);
    old.swap(g_retired);
  }
  gdn_status st = finish_work() == cudaSuccess ? GDN_OK : failed();
  std::vector<Retired> left;
  for (const Retired& r : old) {
    if (st != GDN_OK || r.dev != dev)
      left.push_back(r);
    else if (cudaFree(r.p) != cudaSuccess)
      st = failed();
  }
  {
    std::lock_guard<std::mutex> lock(g_ctx_mu);
    g_retired.insert(g_retired.end(), left.begin(), left.end());
  }
  if (st != GDN_OK) return st;
  for (StreamCtx* c : mine) {
    for (void* p : {c->scan.p, c->op.p, static_cast<void*>(c->err)})
      if (p && cudaFree(p) != cudaSuccess) st = GDN_ERR_CUDA;
    c->scan = c->op = {};
    c->err = nullptr;
  }
  if (st != GDN_OK) cudaGetLastError();
  return st;
}

}  // namespace gdn
