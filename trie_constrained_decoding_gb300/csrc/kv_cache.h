// Definitions shared by the kernels of the paged cache and of its attention.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "tcd_cache.h"
#include "tcd_internal.h"

namespace tcd {

// One layer of a cache as the kernels see it.
struct KvView {
  uint8_t* base;      // the layer's first page
  int32_t pages;
  int32_t kv_heads;
  int32_t page_size;  // a power of two
  int32_t page_shift; // its logarithm
  int32_t keep;       // only errors are written to the status, and only over TC_OK
};

__device__ __forceinline__ void set_status(int32_t* status, int64_t i, int32_t code, int32_t keep) {
  if (!keep || (code != TC_OK && status[i] == TC_OK)) status[i] = code;
}

// The tokens of a call (tc_tokens_t by value).
struct TokensView {
  const int32_t* cu;
  const int32_t* ctx;
  const int32_t* table;
  int32_t batch, n_tokens, width;
};

// 16-bit element types: pairs to and from 32-bit floats.  kShift is log2 of a
// factor that the attention's weights carry (attend.cu says why).
struct Bf16 {
  // acc + 0 * v for each half: zero as long as every v is finite, else NaN.
  static __device__ __forceinline__ uint32_t trace(uint32_t v, uint32_t acc) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0u), "r"(acc));
    return r;
  }
  static constexpr uint32_t kMma = 1;       // operand type of a tensor-core instruction
  static constexpr uint32_t kExp = 0x7f80;  // exponent bits
  static constexpr float kShift = 0.f;
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
struct F16 {
  static __device__ __forceinline__ uint32_t trace(uint32_t v, uint32_t acc) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0u), "r"(acc));
    return r;
  }
  static constexpr uint32_t kMma = 0;
  static constexpr uint32_t kExp = 0x7c00;
  static constexpr float kShift = 7.f;
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// Slots of a sequence (their numbers, rounded up to tiles, fit 31 bits).
constexpr int64_t kMaxSlots = 0x7fff0000;

// Rows, context and slots of sequence b.  False where they are out of range:
// rows outside the packed arrays, or more slots than the page table has.
struct SeqSpan {
  int32_t row0, n, ctx;
};
__device__ __forceinline__ bool seq_span(const TokensView& t, int page_size, int b, SeqSpan* s) {
  const int32_t lo = __ldg(t.cu + b), hi = __ldg(t.cu + b + 1), c = __ldg(t.ctx + b);
  s->row0 = lo;
  s->n = hi - lo;
  s->ctx = c;
  const int64_t room = (int64_t)t.width * page_size;
  return lo >= 0 && hi >= lo && hi <= t.n_tokens && c >= 0 &&
         (int64_t)c + (hi - lo) <= (room < kMaxSlots ? room : kMaxSlots);
}

// ------------------------------------------------------------ host helpers

inline tc_status kv_fail(tc_status code, const char* who, const char* what = "") noexcept {
  return fail_with(code, who, what);
}

// (`what` ends in ": ")
inline tc_status kv_cuda_fail(cudaError_t e, const char* what) noexcept {
  cudaGetLastError();
  return fail_with(e == cudaErrorMemoryAllocation ? TC_ERR_OOM : TC_ERR_CUDA, what, cudaGetErrorString(e));
}

inline bool kv_misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Makes the cache's device current for the length of a call.
struct KvDevice {
  int prev = -1;
  bool ok = false;
  explicit KvDevice(int dev) {
    ok = cudaGetDevice(&prev) == cudaSuccess && (prev == dev || cudaSetDevice(dev) == cudaSuccess);
    if (prev == dev) prev = -1;
    if (!ok) cudaGetLastError();
  }
  ~KvDevice() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

tc_status kv_check(const char* who, const tc_kv_t* kv);
tc_status kv_check_tokens(const char* who, const tc_tokens_t* t, bool rows);
KvView kv_view(const tc_kv_t* kv, int32_t layer);
inline TokensView tokens_view(const tc_tokens_t* t) {
  return TokensView{t->cu_tokens, t->ctx_lens, t->page_table, t->batch, t->n_tokens, t->table_width};
}

}  // namespace tcd
