// Definitions shared by the projection's kernels: what they are given, the
// instructions they are made of, and what they do with a finished sum.
#pragma once

#include <cuda.h>

#include "kv_cache.h"
#include "tcd_linear.h"

namespace tcd {

// Where a finished sum goes (tc_linear_t and tc_linear_call_t by value).
struct LinearOut {
  const uint16_t* bias;
  const uint16_t* gate_bias;
  const uint16_t* residual;
  uint16_t* out;
  int64_t residual_stride, out_stride;
  int32_t n_tokens, features;
  int32_t act;
  int32_t wide;  // elements that an access of rows may have: four where all rows are aligned and whole fours, else one
};

struct LinearParams {
  LinearOut o;
  int32_t k_tiles;     // 64-element steps of a sum
  int32_t gated;
  int32_t* status;
  int32_t wait_limit;  // polls of one wait before it gives up
  int32_t withhold;    // test switch: the first load is left out
  int32_t tile;        // tokens of a tile; linear_pair.cu: rows of the weights that a CTA loads
  int32_t tok_tiles;
  // few tokens (linear.cu)
  int32_t split;       // CTAs of a cluster, which share out a sum
  int32_t stages;
  int32_t tmem_cols;
};

constexpr int kLinearDevices = 64;
constexpr uint32_t kRowBytes = 128;         // 64 elements of a step: one row of the 128-byte swizzle
// Default polls of one wait, and the fewest of those at a CTA's end for what it has in flight, which must not outlive it.
constexpr int kLinearWaitLimit = 1 << 22;

// ------------------------------------------------------------- instructions

__device__ __forceinline__ uint32_t smem_at(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// One poll of a phase (it waits a while in hardware).
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
// Waits for a phase, at most `limit` polls; false if it gave up or another wait of the CTA has.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, int limit, volatile int32_t* abort) {
  if (bar_try(bar, parity)) return true;
  int i = 1;
#pragma unroll 1
  do {
    if (bar_try(bar, parity)) return true;
    ++i;
  } while (i < limit && !*abort);
  *abort = 1;
  return false;
}
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_tile(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();  // (whole warps meet)
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t tile_desc(uint32_t a) {
  return (uint64_t)((a & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// Instruction descriptor of kind::f16: 32-bit accumulator, both operands K-major and of one type.
template <typename T>
__device__ __forceinline__ uint32_t product_desc(int m, int n) {
  return (1u << 4) | (T::kMma << 7) | (T::kMma << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// -------------------------------------------------------- a finished sum

template <typename T>
__device__ __forceinline__ float one(const uint16_t* p) {
  return T::unpack(__ldg(p)).x;
}

__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float one_over(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case TC_ACT_RELU:
      return z < 0.f ? 0.f : z;  // (NaN stays)
    case TC_ACT_SILU:
      return z * one_over(1.f + exp2_of(z * -1.4426950409f));
    case TC_ACT_GELU: {
      // max(z, 0) - a / 2 erfc(a / sqrt 2), a = |z|, with erfc(x) = t exp(-x^2) P(t), t = 1 / (1 + 0.45 x): P is a
      // least-squares fit whose relative error was levelled out over x = 0 ... 14 (3.6e-7, 3 units of 2^-23).
      const float a = fminf(fabsf(z), 30.f), t = one_over(fmaf(a, 0.3181980515f, 1.f));
      float p = fmaf(t, 0.06890339404f, -0.24888466299f);
      p = fmaf(t, p, 0.22390307486f);
      p = fmaf(t, p, 0.02623970434f);
      p = fmaf(t, p, 0.19616602361f);
      p = fmaf(t, p, 0.22578363121f);
      p = fmaf(t, p, 0.25400400162f);
      p = fmaf(t, p, 0.25388520956f);
      return (z < 0.f ? 0.f : z) - 0.5f * a * (t * p) * exp2_of(a * a * -0.7213475204f);
    }
    case TC_ACT_GELU_TANH: {
      // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
      const float u = z * fmaf(0.044715f * z, z, 1.f) * -2.3022081985f;  // -2 sqrt(2 / pi) log2(e)
      return z * one_over(1.f + exp2_of(u));
    }
    default:
      return z;
  }
}

// Calls f with the activation as a constant.  (Around a loop of finished sums: inside of it each turn of an unrolled
// loop would have code for every activation, and small calls are bound by the fetch of their instructions.)
template <int A>
struct Act {
  static constexpr int kAct = A;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case TC_ACT_RELU: return f(Act<TC_ACT_RELU>());
    case TC_ACT_SILU: return f(Act<TC_ACT_SILU>());
    case TC_ACT_GELU: return f(Act<TC_ACT_GELU>());
    case TC_ACT_GELU_TANH: return f(Act<TC_ACT_GELU_TANH>());
    default: return f(Act<TC_ACT_NONE>());
  }
}

// Many tokens, on pairs of SMs (linear_pair.cu).
cudaError_t launch_linear_pair(const LinearParams& p, int device, int dtype, int pairs, const CUtensorMap& w,
                               const CUtensorMap& g, const CUtensorMap& x, cudaStream_t s);

}  // namespace tcd
