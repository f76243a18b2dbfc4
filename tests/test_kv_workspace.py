"""The cache attention's scratch on the host alone (no GPU): its source compiled with a small fake of the CUDA runtime,
whose allocations, captures and graphs the checks control."""
import pathlib
import subprocess

import pytest

ROOT = pathlib.Path(__file__).resolve().parent.parent
CSRC = ROOT / "nvfp4_quantized_matmul_gb300" / "csrc"

FAKE = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <new>
#include <set>
#include <thread>
#include <vector>
#include "nvfp4_internal.h"

// ---- host allocations that can be made to fail
static long g_new_left = -1;  // the allocation after so many fails; -1: none
void* operator new(size_t n) {
  if (g_new_left >= 0 && g_new_left-- == 0) throw std::bad_alloc();
  return malloc(n);
}
void operator delete(void* p) noexcept { free(p); }
void operator delete(void* p, size_t) noexcept { free(p); }

// ---- the runtime
struct Holder { void* p; cudaHostFn_t destroy; };
static std::set<void*> g_live;              // device allocations
static int g_fail = 0;                      // 1: cudaMalloc, 2: memset, 3: user objects, 4: retaining them
static cudaError_t g_last = cudaSuccess;
static std::map<cudaStream_t, unsigned long long> g_capturing;
static std::map<void*, std::vector<Holder*>> g_graphs;
static cudaStreamCaptureMode g_mode = cudaStreamCaptureModeGlobal;
static thread_local unsigned long long g_thread_stream = 7;
static cudaError_t set(cudaError_t e) { if (e != cudaSuccess) g_last = e; return e; }
static void let_go(Holder* h) { h->destroy(h->p); delete h; }

extern "C" {
cudaError_t cudaMalloc(void** p, size_t n) {
  if (g_fail == 1 || g_mode != cudaStreamCaptureModeRelaxed) return set(cudaErrorMemoryAllocation);
  *p = malloc(n < 65536 ? 65536 : n);
  g_live.insert(*p);
  return cudaSuccess;
}
cudaError_t cudaFree(void* p) { if (p && !g_live.erase(p)) abort(); free(p); return cudaSuccess; }
cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned) { *s = (cudaStream_t)0x999; return cudaSuccess; }
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return set(g_fail == 2 ? cudaErrorInvalidValue : cudaSuccess); }
cudaError_t cudaGetLastError() { cudaError_t e = g_last; g_last = cudaSuccess; return e; }
cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode* m) { std::swap(*m, g_mode); return cudaSuccess; }
cudaError_t cudaStreamGetId(cudaStream_t, unsigned long long* id) { *id = g_thread_stream; return cudaSuccess; }
cudaError_t cudaStreamGetCaptureInfo(cudaStream_t s, cudaStreamCaptureStatus* status, unsigned long long* id, cudaGraph_t* graph,
                                     const cudaGraphNode_t**, const cudaGraphEdgeData**, size_t*) {
  const auto it = g_capturing.find(s);
  *status = it == g_capturing.end() ? cudaStreamCaptureStatusNone : cudaStreamCaptureStatusActive;
  *id = it == g_capturing.end() ? 12345 : it->second;
  *graph = it == g_capturing.end() ? nullptr : (cudaGraph_t)it->second;
  return cudaSuccess;
}
cudaError_t cudaUserObjectCreate(cudaUserObject_t* out, void* p, cudaHostFn_t destroy, unsigned, unsigned) {
  if (g_fail == 3) return set(cudaErrorInvalidValue);
  Holder* h = (Holder*)malloc(sizeof(Holder));
  *h = Holder{p, destroy};
  *out = (cudaUserObject_t)h;
  return cudaSuccess;
}
cudaError_t cudaUserObjectRelease(cudaUserObject_t o, unsigned) { let_go((Holder*)o); return cudaSuccess; }
cudaError_t cudaGraphRetainUserObject(cudaGraph_t graph, cudaUserObject_t o, unsigned, unsigned) {
  if (g_fail == 4) return set(cudaErrorInvalidValue);
  const long left = g_new_left;  // the fake's own allocations do not count
  g_new_left = -1;
  g_graphs[graph].push_back((Holder*)o);
  g_new_left = left;
  return cudaSuccess;
}
}
static void destroy_graph(unsigned long long id) {
  for (Holder* h : g_graphs[(void*)id]) let_go(h);
  g_graphs.erase((void*)id);
}

#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); exit(1); } } while (0)
static unsigned* at(cudaStream_t s, size_t bytes, cudaError_t want = cudaSuccess) {
  unsigned* done = nullptr;
  float* parts = nullptr;
  const cudaError_t e = nvfp4::kv_workspace(0, s, bytes, &done, &parts);
  CHECK(e == want && g_last == cudaSuccess && g_mode == cudaStreamCaptureModeGlobal);
  CHECK(want != cudaSuccess || (done && (char*)parts == (char*)done + 4 * nvfp4::kKvMaxCtas));
  return done;
}
static cudaStream_t stream(uintptr_t i) { return (cudaStream_t)(0x1000 * i); }

int main() {
  // a stream's own, the same for every call, another when it has to grow
  unsigned* a = at(stream(1), 1000);
  CHECK(at(stream(1), 500) == a && at(stream(2), 1000) != a && at(nullptr, 1000) != a);
  unsigned* grown = at(stream(1), 5000);
  CHECK(grown != a && at(stream(1), 1000) == grown && g_live.count(a));

  // each thread's default stream is one of its own
  unsigned* mine = at(cudaStreamPerThread, 1000);
  unsigned* other = nullptr;
  std::thread([&] { g_thread_stream = 8; other = at(cudaStreamPerThread, 1000); }).join();
  CHECK(mine != other && at(cudaStreamPerThread, 1000) == mine);

  // captures on one stream have one each, not the stream's; two streams of one capture too
  g_capturing[stream(1)] = 21;
  unsigned* first = at(stream(1), 1000);
  CHECK(first != grown && at(stream(1), 1000) == first);
  g_capturing[stream(2)] = 21;
  unsigned* branch = at(stream(2), 1000);
  CHECK(branch != first);
  g_capturing[stream(1)] = 22;
  unsigned* second = at(stream(1), 1000);
  CHECK(second != first && second != branch && second != grown);
  unsigned* second_grown = at(stream(1), 3000);  // both stay with the graph
  CHECK(second_grown != second && g_live.count(second) && g_graphs[(void*)22].size() == 2);
  // the next capture takes over what a graph that is gone had, and nothing else
  destroy_graph(22);
  g_capturing[stream(1)] = 23;
  unsigned* third = at(stream(1), 2000);
  CHECK(third == second_grown);
  g_capturing[stream(1)] = 24;
  unsigned* fourth = at(stream(1), 2000);
  CHECK(fourth != third && fourth != first && fourth != branch);
  size_t live = g_live.size();
  for (unsigned long long id = 100; id < 200; ++id) {  // no growth from capture to capture
    g_capturing[stream(3)] = id;
    at(stream(3), 2000);
    destroy_graph(id);
  }
  CHECK(g_live.size() <= live + 1);

  // failures of the runtime: reported once, nothing lost, and the next call is as if they had not been
  for (int f = 1; f <= 4; ++f) {
    g_capturing[stream(4)] = 300 + f;
    live = g_live.size();
    g_fail = f;
    at(stream(4), 100000 * f, f == 1 ? cudaErrorMemoryAllocation : cudaErrorInvalidValue);
    if (f <= 2) at(stream(5 + f), 1000, f == 1 ? cudaErrorMemoryAllocation : cudaErrorInvalidValue);
    g_fail = 0;
    CHECK(g_live.size() <= live + (f > 2));
    unsigned* w = at(stream(4), 100000 * f);
    CHECK(w && at(stream(4), 1000) == w && g_live.size() <= live + 1);
  }
  // no memory on the host, at each allocation in turn
  for (uintptr_t i = 0; i < 2; ++i)
    for (long n = 0;; ++n) {
      const cudaStream_t s = stream(100 + 50 * i + n);
      if (i) g_capturing[s] = 1000 + n;
      live = g_live.size();
      unsigned* done = nullptr;
      float* parts = nullptr;
      g_new_left = n;
      const cudaError_t e = nvfp4::kv_workspace(0, s, 200000, &done, &parts);
      const bool failed = g_new_left < 0;
      g_new_left = -1;
      CHECK(g_mode == cudaStreamCaptureModeGlobal && g_last == cudaSuccess);
      CHECK(e == (failed ? cudaErrorMemoryAllocation : cudaSuccess));
      if (!failed) break;
      CHECK(g_live.size() == live && n < 40);
      at(s, 1000);
    }

  nvfp4::release_kv_workspaces();
  CHECK(g_live.empty());
  for (auto& g : std::map<void*, std::vector<Holder*>>(g_graphs)) destroy_graph((unsigned long long)g.first);
  g_capturing.clear();
  CHECK(at(stream(1), 1000));
  nvfp4::release_kv_workspaces();
  CHECK(g_live.empty());
  puts("ok");
}
"""


def cuda_include():
    for d in ("/usr/local/cuda/include",):
        if (pathlib.Path(d) / "cuda_runtime.h").exists():
            return d
    pytest.skip("no CUDA headers")


def test_workspaces(tmp_path):
    main, exe = tmp_path / "main.cpp", tmp_path / "workspaces"
    main.write_text(FAKE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wno-attributes", "-pthread", f"-I{CSRC}", f"-I{cuda_include()}", "-x", "c++",
                    str(CSRC / "nvfp4_kv_workspace.cu"), str(main), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and run.stdout == "ok\n", (run.returncode, run.stdout, run.stderr)
