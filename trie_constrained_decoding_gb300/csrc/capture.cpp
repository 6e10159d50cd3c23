// Buffers of calls that are captured into a graph: a graph may be launched on
// any stream, beside others, and for as long as it exists, so what its calls use
// can neither belong to a stream nor end with the object that made the calls.
#include <cuda_runtime.h>

#include <atomic>
#include <new>

#include "tcd_cache.h"
#include "tcd_internal.h"

namespace {

// (`what` ends in ": ")
tc_status fail(const char* what, cudaError_t e) {
  cudaGetLastError();
  return tcd::fail_with(TC_ERR_CUDA, what, cudaGetErrorString(e));
}

// Called by the graph's destruction, on any thread; no CUDA call is allowed.
void CUDART_CB mark(void* word) { static_cast<std::atomic<int32_t>*>(word)->store(1, std::memory_order_release); }
static_assert(sizeof(std::atomic<int32_t>) == sizeof(int32_t), "the word is read as an int32_t");

// This thread's calls are not held to the rules of captures that it is not part of.
struct Relaxed {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  Relaxed() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~Relaxed() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

}  // namespace

extern "C" tc_status tc_capture_id(void* stream, uint64_t* id) {
  if (!id) return TC_ERR_INVALID_ARG;
  *id = 0;
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  unsigned long long n = 0;
  const cudaError_t e = cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &st, &n);
  if (e == cudaErrorStreamCaptureImplicit) {  // (the legacy stream, which cannot be captured, beside a capture)
    cudaGetLastError();
    return TC_OK;
  }
  if (e != cudaSuccess) return fail("tc_capture_id: ", e);
  if (st != cudaStreamCaptureStatusNone) *id = n;
  return TC_OK;
}

extern "C" tc_status tc_capture_watch(void* stream, int32_t** gone) {
  if (!gone) return TC_ERR_INVALID_ARG;
  *gone = nullptr;
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  unsigned long long n = 0;
  cudaGraph_t graph = nullptr;
  cudaError_t e = cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &st, &n, &graph);
  if (e != cudaSuccess) return fail("tc_capture_watch: ", e);
  if (st != cudaStreamCaptureStatusActive || !graph) return TC_ERR_INVALID_ARG;
  auto* word = new (std::nothrow) std::atomic<int32_t>(0);
  if (!word) return TC_ERR_OOM;
  cudaUserObject_t obj = nullptr;
  e = cudaUserObjectCreate(&obj, word, mark, 1, cudaUserObjectNoDestructorSync);
  if (e != cudaSuccess) {
    delete word;
    return fail("tc_capture_watch: ", e);
  }
  e = cudaGraphRetainUserObject(graph, obj, 1, cudaGraphUserObjectMove);
  if (e != cudaSuccess) {  // (the word is marked when the release is done, and stays)
    cudaUserObjectRelease(obj, 1);
    return fail("tc_capture_watch: ", e);
  }
  *gone = reinterpret_cast<int32_t*>(word);
  return TC_OK;
}

extern "C" void tc_capture_unwatch(int32_t* gone) { delete reinterpret_cast<std::atomic<int32_t>*>(gone); }

extern "C" tc_status tc_capture_mode(int32_t* mode) {
  if (!mode || *mode < 0 || *mode > 2) return TC_ERR_INVALID_ARG;
  static const cudaStreamCaptureMode modes[3] = {cudaStreamCaptureModeGlobal, cudaStreamCaptureModeThreadLocal,
                                                 cudaStreamCaptureModeRelaxed};
  cudaStreamCaptureMode m = modes[*mode];
  const cudaError_t e = cudaThreadExchangeStreamCaptureMode(&m);
  if (e != cudaSuccess) return fail("tc_capture_mode: ", e);
  *mode = m == modes[0] ? 0 : m == modes[1] ? 1 : 2;
  return TC_OK;
}

extern "C" tc_status tc_clear_now(void* ptr, int64_t bytes, void* stream) {
  if (!ptr || bytes < 0) return TC_ERR_INVALID_ARG;
  Relaxed relaxed;
  cudaError_t e = cudaMemsetAsync(ptr, 0, (size_t)bytes, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TC_OK : fail("tc_clear_now: ", e);
}
