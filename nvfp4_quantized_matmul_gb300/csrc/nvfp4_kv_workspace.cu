// Scratch of the cache attention's kernels. Host code alone: no kernel, and of
// CUDA only the runtime's functions.
#include <atomic>
#include <exception>
#include <iterator>
#include <map>
#include <memory>
#include <mutex>
#include <tuple>
#include <vector>

#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr size_t kDoneBytes = 4 * kKvMaxCtas;

// Partial results and arrival counts: two calls that may run at the same time never share them. A stream's calls have one
// allocation, made on the first call that needs it, grown on demand and kept until release_kv_workspaces(). Calls captured
// into a graph run wherever the graph is launched, so each capture has its own, which its graph keeps hold of; when the last
// graph made from the capture is gone, the next capture may have it. The counts are zero between calls.
struct Workspace {
  char* p = nullptr;
  size_t bytes = 0;
  int dev = 0;
  std::atomic<bool> idle{false};  // of a capture whose graphs are gone
};
using WorkspaceRef = std::shared_ptr<Workspace>;
// device, capture (0: none), stream: the handle, or a number of the calling thread's own
using WorkspaceKey = std::tuple<int, unsigned long long, unsigned long long>;
std::mutex g_ws_mu;
std::map<WorkspaceKey, WorkspaceRef> g_ws;
std::vector<WorkspaceRef> g_ws_retired;   // outgrown ones, which queued calls may still use
std::vector<WorkspaceRef> g_ws_captured;  // all that captures have or had

// Called when nothing holds a captured graph any more, on a thread of the driver's: no CUDA calls, no locks.
void CUDART_CB release_captured(void* ref) {
  const std::unique_ptr<WorkspaceRef> p(static_cast<WorkspaceRef*>(ref));
  (*p)->idle.store(true, std::memory_order_release);
}

// A cleared allocation. Cleared here and now, not by the stream: while that is captured, its graph would do it.
cudaError_t make_workspace(int dev, size_t bytes, WorkspaceRef* out) {
  const WorkspaceRef w = std::make_shared<Workspace>();
  cudaStream_t own = nullptr;
  cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&w->p), bytes);
  if (e != cudaSuccess) return e;
  e = cudaStreamCreateWithFlags(&own, cudaStreamNonBlocking);
  if (e == cudaSuccess) e = cudaMemsetAsync(w->p, 0, kDoneBytes, own);
  if (e == cudaSuccess) e = cudaStreamSynchronize(own);
  if (own) cudaStreamDestroy(own);
  if (e != cudaSuccess) {
    cudaFree(w->p);
    return e;
  }
  w->bytes = bytes;
  w->dev = dev;
  *out = w;
  return cudaSuccess;
}

// For a capture: one whose graphs are gone, or a new one; `graph` then holds it.
cudaError_t captured_workspace(int dev, size_t bytes, cudaGraph_t graph, WorkspaceRef* out) {
  for (auto it = g_ws.begin(); it != g_ws.end();)
    it = std::get<1>(it->first) && it->second && it->second->idle ? g_ws.erase(it) : std::next(it);
  g_ws_captured.reserve(g_ws_captured.size() + 1);
  auto ref = std::make_unique<WorkspaceRef>();
  for (const WorkspaceRef& w : g_ws_captured)
    if (w->dev == dev && w->bytes >= bytes && w->idle.exchange(false, std::memory_order_acquire)) {
      *ref = w;
      break;
    }
  cudaError_t e;
  if (!*ref) {
    if ((e = make_workspace(dev, bytes, ref.get())) != cudaSuccess) return e;
    g_ws_captured.push_back(*ref);
  }
  const WorkspaceRef w = *ref;
  cudaUserObject_t holder;
  if ((e = cudaUserObjectCreate(&holder, ref.get(), release_captured, 1, cudaUserObjectNoDestructorSync)) != cudaSuccess) {
    w->idle.store(true, std::memory_order_release);
    return e;
  }
  ref.release();  // the holder's now
  if ((e = cudaGraphRetainUserObject(graph, holder, 1, cudaGraphUserObjectMove)) != cudaSuccess) {
    cudaUserObjectRelease(holder, 1);
    return e;
  }
  *out = w;
  return cudaSuccess;
}

// The thread's capture mode relaxed while it lasts, so that an allocation does not end a capture.
struct Relaxed {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
  ~Relaxed() {
    if (e == cudaSuccess) cudaThreadExchangeStreamCaptureMode(&mode);
  }
};

cudaError_t find_workspace(int dev, cudaStream_t st, size_t bytes, unsigned** done, float** parts) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  unsigned long long capture = 0, stream = reinterpret_cast<uintptr_t>(st);
  cudaGraph_t graph = nullptr;
  cudaError_t e;
  if (st != nullptr && st != cudaStreamLegacy) {  // which cannot be captured, and may not be asked during other captures
    if ((e = cudaStreamGetCaptureInfo(st, &status, &capture, &graph)) != cudaSuccess) return e;
    if (status != cudaStreamCaptureStatusActive) capture = 0;
    if (st == cudaStreamPerThread) {  // one handle, a stream of each thread
      if ((e = cudaStreamGetId(st, &stream)) != cudaSuccess) return e;
      stream |= 1ull << 63;
    }
  }
  bytes += kDoneBytes;
  std::lock_guard<std::mutex> lock(g_ws_mu);
  WorkspaceRef& w = g_ws[WorkspaceKey{dev, capture, stream}];
  if (!w || w->bytes < bytes) {
    const Relaxed relaxed;
    if (relaxed.e != cudaSuccess) return relaxed.e;
    g_ws_retired.reserve(g_ws_retired.size() + 1);
    WorkspaceRef made;
    if ((e = capture ? captured_workspace(dev, bytes, graph, &made) : make_workspace(dev, bytes, &made)) != cudaSuccess) return e;
    if (w && !capture) g_ws_retired.push_back(w);
    w = made;
  }
  *done = reinterpret_cast<unsigned*>(w->p);
  *parts = reinterpret_cast<float*>(w->p + kDoneBytes);
  return cudaSuccess;
}

}  // namespace

cudaError_t kv_workspace(int dev, cudaStream_t st, size_t bytes, unsigned** done, float** parts) {
  cudaError_t e;
  try {
    e = find_workspace(dev, st, bytes, done, parts);
  } catch (const std::exception&) {  // no memory for the host's own records: callers are C
    e = cudaErrorMemoryAllocation;
  }
  if (e != cudaSuccess) cudaGetLastError();  // said here; else the next launch would seem to have failed with it
  return e;
}

void release_kv_workspaces() {
  std::lock_guard<std::mutex> lock(g_ws_mu);
  for (auto& kv : g_ws)
    if (kv.second && !std::get<1>(kv.first)) cudaFree(kv.second->p);
  for (auto& w : g_ws_retired) cudaFree(w->p);
  for (auto& w : g_ws_captured) cudaFree(w->p);  // (what graphs still hold is the description alone)
  g_ws.clear();
  g_ws_retired.clear();
  g_ws_captured.clear();
}

}  // namespace nvfp4
