// Drives the library's per-stream scratch (csrc/stream_context.cu, compiled as plain
// C++) against stand-ins for the CUDA runtime calls it makes, which keep a ledger of
// what is allocated and by which stream it is freed.  One check per run, named by the
// argument; exit code 0, or 1 with the failing condition on stderr.
#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <set>
#include <string>
#include <thread>

#include "gdn_internal.h"

#define CHECK(c)                                                      \
  do {                                                                \
    if (!(c)) {                                                       \
      std::fprintf(stderr, "line %d: %s\n", __LINE__, #c);            \
      std::exit(1);                                                   \
    }                                                                 \
  } while (0)

namespace {
std::mutex mu;
struct Block {
  size_t bytes;
  cudaStream_t stream;  // of a stream-ordered allocation, else nullptr
};
std::map<void*, Block> live;
std::set<cudaStream_t> captured;
size_t bytes_live = 0, most_live = 0;
int allocations = 0, fail_after = -1;
unsigned device_word;

cudaError_t allocate(void** p, size_t n, cudaStream_t s) {
  std::lock_guard<std::mutex> l(mu);
  if (fail_after >= 0 && fail_after-- == 0) return cudaErrorMemoryAllocation;
  *p = std::malloc(16);
  live[*p] = {n, s};
  ++allocations;
  bytes_live += n;
  if (bytes_live > most_live) most_live = bytes_live;
  return cudaSuccess;
}
cudaError_t drop(void* p) {
  std::lock_guard<std::mutex> l(mu);
  CHECK(live.count(p));
  bytes_live -= live[p].bytes;
  live.erase(p);
  std::free(p);
  return cudaSuccess;
}
cudaStream_t stream(size_t i) { return reinterpret_cast<cudaStream_t>(i * 64); }
}  // namespace

extern "C" {
cudaError_t cudaMalloc(void** p, size_t n) { return allocate(p, n, nullptr); }
cudaError_t cudaFree(void* p) { return drop(p); }
cudaError_t cudaMallocAsync(void** p, size_t n, cudaStream_t s) { return allocate(p, n, s); }
cudaError_t cudaFreeAsync(void* p, cudaStream_t s) {
  {
    std::lock_guard<std::mutex> l(mu);
    CHECK(live.count(p) && live[p].stream == s);  // freed behind the work that names it
  }
  return drop(p);
}
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t s, cudaStreamCaptureStatus* st) {
  *st = captured.count(s) ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
}

namespace gdn {
cudaError_t current_error_word(unsigned int** out) {
  *out = &device_word;
  return cudaSuccess;
}
}  // namespace gdn

using namespace gdn;

namespace {
constexpr size_t MB = size_t(1) << 20;

cudaError_t done() { return cudaSuccess; }

void* op(int dev, cudaStream_t s, size_t bytes, gdn_status want = GDN_OK) {
  OpScratch sc;
  unsigned* err = nullptr;
  CHECK(op_scratch(dev, s, bytes, &err, &sc) == want);
  if (want != GDN_OK) return nullptr;
  CHECK(err);
  void* p = sc.p;
  CHECK(op_scratch_done(&sc) == cudaSuccess);
  return p;
}
void* scan(int dev, cudaStream_t s, size_t bytes) {
  std::unique_lock<std::mutex> launching;
  unsigned* err = nullptr;
  void* ws = nullptr;
  CHECK(scan_scratch(dev, s, bytes, &err, &ws, &launching) == GDN_OK && err && launching.owns_lock());
  return ws;
}

// Lengths that creep up leave no buffers behind and seldom allocate.
void creeping() {
  size_t bytes = 10 * MB;
  for (int i = 0; i < 400; ++i, bytes += bytes / 100) {
    CHECK(op(0, stream(1), bytes));
    CHECK(bytes_live <= 2 * bytes + 4 * MB);
  }
  CHECK(bytes > 400 * MB && allocations < 40);
  CHECK(most_live <= 2 * bytes + 4 * MB);
  void* p = op(0, stream(1), bytes);
  CHECK(op(0, stream(1), 5 * MB) == p);  // smaller calls keep it
}

// A captured scan may hold the stream's scratch, so a replaced one stays.
void graphs() {
  void* first = scan(0, stream(1), 8 * MB);
  captured.insert(stream(1));
  CHECK(scan(0, stream(1), 8 * MB) == first);
  CHECK(scan(0, stream(1), 9 * MB) == nullptr);  // to be allocated in the graph
  captured.clear();
  CHECK(scan(0, stream(1), 80 * MB) != first);
  CHECK(live.count(first));
  // a captured operator takes its own, and the stream's is left alone
  void* mine = op(0, stream(1), 3 * MB);
  captured.insert(stream(1));
  {
    OpScratch sc;
    unsigned* err = nullptr;
    CHECK(op_scratch(0, stream(1), 2 * MB, &err, &sc) == GDN_OK);
    CHECK(sc.p && sc.p != mine && live[sc.p].stream == stream(1));
    void* p = sc.p;
    CHECK(op_scratch_done(&sc) == cudaSuccess && !live.count(p));
  }
  CHECK(live.count(mine));
  captured.clear();
  CHECK(op(0, stream(1), 3 * MB) == mine);
}

void release() {
  CHECK(scan(0, stream(1), 8 * MB) && scan(0, stream(1), 20 * MB) && op(0, stream(1), 3 * MB) && op(0, stream(2), MB));
  void* other = op(1, stream(1), MB);
  CHECK(release_contexts(0, done) == GDN_OK);
  CHECK(live.count(other) && live.size() == 2);  // and its error word
  CHECK(!own_error_word(0, stream(1)) && own_error_word(1, stream(1)));
  CHECK(op(0, stream(1), MB) && scan(0, stream(1), MB));
  CHECK(release_contexts(0, done) == GDN_OK && release_contexts(1, done) == GDN_OK && live.empty());
}

// An allocation that fails is reported, and the next call is served.
void failures() {
  for (int n = 0; n < 2; ++n) {
    fail_after = n;
    op(0, stream(1), 4 * MB, GDN_ERR_CUDA);
    fail_after = -1;
    CHECK(op(0, stream(1), 4 * MB));
    release_contexts(0, done);
  }
  CHECK(op(0, stream(1), 4 * MB));
  fail_after = 0;
  op(0, stream(1), 400 * MB, GDN_ERR_CUDA);
  fail_after = -1;
  CHECK(op(0, stream(1), 4 * MB) && release_contexts(0, done) == GDN_OK && live.empty());
}

// Whether a thread that does `call` has come through, given a little time.
template <typename F>
bool comes_through(F call, std::thread* t, std::atomic<bool>* through) {
  *through = false;
  *t = std::thread([=] {
    call();
    *through = true;
  });
  for (int i = 0; i < 200 && !*through; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(10));
  return *through;
}

// A call that holds its stream's scratch keeps others off that stream, and off no other
// stream or device; a release waits for it.
void threads() {
  op(0, stream(1), MB);
  OpScratch held;
  unsigned* err = nullptr;
  CHECK(op_scratch(0, stream(1), MB, &err, &held) == GDN_OK);
  std::thread t[6];
  std::atomic<bool> through[6];
  CHECK(comes_through([] { op(0, stream(2), MB); }, &t[0], &through[0]));
  CHECK(comes_through([] { scan(0, stream(3), MB); }, &t[1], &through[1]));
  CHECK(comes_through([] { op(1, stream(1), MB); }, &t[2], &through[2]));
  CHECK(!comes_through([] { op(0, stream(1), MB); }, &t[3], &through[3]));
  CHECK(!comes_through([] { scan(0, stream(1), MB); }, &t[4], &through[4]));
  CHECK(!comes_through([] { release_contexts(0, done); }, &t[5], &through[5]));
  CHECK(live.count(held.p));
  CHECK(op_scratch_done(&held) == cudaSuccess);
  for (auto& x : t) x.join();
  CHECK(release_contexts(0, done) == GDN_OK && release_contexts(1, done) == GDN_OK && live.empty());
}

}  // namespace

int main(int argc, char** argv) {
  const std::map<std::string, void (*)()> checks = {
      {"creeping", creeping}, {"graphs", graphs}, {"release", release}, {"failures", failures},
      {"threads", threads}};
  CHECK(argc == 2 && checks.count(argv[1]));
  checks.at(argv[1])();
  return 0;
}
