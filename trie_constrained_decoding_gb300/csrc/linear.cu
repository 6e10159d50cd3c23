// Projections: y = act(x W^T + b) [* (x V^T + c)] + r, on the tensor cores.
//
// The weights are the M side of the product and the tokens its N side: a tile
// is 128 features (with a gate: 64 of it and the same 64 of the weights) by up
// to 256 tokens, so a decode step reads every weight once and pads tokens to a
// multiple of 16 only.
//
// Where a product has few tiles its sums are cut: the CTAs of a cluster take a
// part of in_features each, leave their sums in shared memory, and every one of
// them adds up a share of the outputs over the cluster (distributed shared
// memory) in the order of the parts: no workspace, no second launch, the same
// bits each time.
//
// One CTA, four warps: warp 0 loads by TMA (128-byte swizzle; rows and columns
// past the ends are zeros), warp 1 issues the products, all four read the
// accumulator.
#include <cudaTypedefs.h>

#include "linear.h"

namespace tcd {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxStages = 8;
constexpr uint32_t kWeightBytes = 128 * kRowBytes;

struct Hdr {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t done;
  uint32_t tmem;
  int32_t abort;
};

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// Four floats of CTA `rank`'s shared memory, at the place that `a` is in this one's.
__device__ __forceinline__ float4 peer_float4(uint32_t a, uint32_t rank) {
  uint32_t at;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

template <typename T>
__device__ __forceinline__ void finish4(const LinearParams& p, int64_t token, int f, float4 z4, float4 g4) {
  const LinearOut& o = p.o;
  float z[4] = {z4.x, z4.y, z4.z, z4.w}, g[4] = {g4.x, g4.y, g4.z, g4.w};
  const int n = min(4, o.features - f);
  const uint16_t* res = o.residual ? o.residual + token * o.residual_stride + f : nullptr;
  uint16_t* out = o.out + token * o.out_stride + f;
  const bool wide = o.wide >= 4 && n == 4;
  float r[4] = {0.f, 0.f, 0.f, 0.f};
  if (res && wide) {
    const uint2 v = *reinterpret_cast<const uint2*>(res);
    const float2 a = T::unpack(v.x), b = T::unpack(v.y);
    r[0] = a.x, r[1] = a.y, r[2] = b.x, r[3] = b.y;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= n) continue;
    if (res && !wide) r[i] = T::unpack(res[i]).x;
    if (o.bias) z[i] += one<T>(o.bias + f + i);
    if (p.gated) {
      if (o.gate_bias) g[i] += one<T>(o.gate_bias + f + i);
      z[i] *= activate(g[i], o.act);
    } else {
      z[i] = activate(z[i], o.act);
    }
    z[i] += r[i];
  }
  if (wide) {
    *reinterpret_cast<uint2*>(out) = make_uint2(T::pack(z[0], z[1]), T::pack(z[2], z[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) out[i] = (uint16_t)T::pack(z[i], 0.f);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    linear_kernel(const LinearParams p, const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ CUtensorMap map_g, const __grid_constant__ CUtensorMap map_x) {
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ Hdr hdr;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = p.split, rank = blockIdx.x % split, tile = blockIdx.x / split;
  const int tok0 = tile % p.tok_tiles * p.tile, rows = p.gated ? 64 : 128;
  const int f0 = tile / p.tok_tiles * rows;
  const int kt0 = p.k_tiles * rank / split, n = p.k_tiles * (rank + 1) / split - kt0;
  const int live = min(p.tile, p.o.n_tokens - tok0);
  const uint32_t stage_bytes = kWeightBytes + (uint32_t)p.tile * kRowBytes;
  // Tiles lie on 1024-byte boundaries.
  const uint32_t at = (smem_at(smem) + 1023u) & ~1023u;
  volatile int32_t* abort = &hdr.abort;
  const int wl = p.wait_limit, stages = p.stages;
  const bool held = p.withhold != 0 && blockIdx.x == 0;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      bar_init(smem_at(&hdr.full[s]), 1);
      bar_init(smem_at(&hdr.empty[s]), 1);
    }
    bar_init(smem_at(&hdr.done), 1);
    hdr.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(&hdr.tmem)),
                 "r"(p.tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // The setup above touches only this CTA; everything read or written from here on may belong to the kernel before.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = hdr.tmem;

  int armed = 0;
  if (warp == 0 && lane == 0) {
    for (; armed < n; ++armed) {
      const int s = armed % stages, turn = armed / stages;
      if (turn > 0 && !bar_wait(smem_at(&hdr.empty[s]), (turn - 1) & 1, wl, abort)) break;
      const uint32_t bar = smem_at(&hdr.full[s]), dst = at + s * stage_bytes;
      if (held && armed == 0) continue;
      bar_expect(bar, stage_bytes);
      const int k = (kt0 + armed) * 64;
      // (64 rows a copy: with a gate, its rows and then the weights')
      load_tile(dst, p.gated ? &map_g : &map_w, k, f0, bar);
      load_tile(dst + kWeightBytes / 2, &map_w, k, p.gated ? f0 : f0 + 64, bar);
      load_tile(dst + kWeightBytes, &map_x, k, tok0, bar);
    }
  } else if (warp == 1 && lane == 0) {
    const uint32_t id = product_desc<T>(128, p.tile);
    for (int i = 0; i < n; ++i) {
      const int s = i % stages;
      if (!bar_wait(smem_at(&hdr.full[s]), (i / stages) & 1, wl, abort)) break;
      tmem_fence_after();
      const uint64_t a = tile_desc(at + s * stage_bytes), b = tile_desc(at + s * stage_bytes + kWeightBytes);
#pragma unroll
      for (int e = 0; e < 4; ++e) product(tmem, a + 2 * e, b + 2 * e, id, i > 0 || e > 0);
      commit(smem_at(&hdr.empty[s]));
    }
    commit(smem_at(&hdr.done));
  }
  __syncwarp();
  // (after a wait that gave up as well: the issuer commits what it has issued)
  bool ok = bar_wait(smem_at(&hdr.done), 0, wl, abort);
  ok = __syncthreads_and(ok && !*abort);
  if (!ok && warp == 0 && lane == 0) {
    // What was issued has to end before this CTA goes on (waits bounded again): the products, and loads that no
    // product has waited for.
    int32_t none = 0;
    bar_wait(smem_at(&hdr.done), 0, wl, &none);
    for (int i = max(0, armed - stages); i < armed; ++i)
      if (!(held && i == 0)) bar_wait(smem_at(&hdr.full[i % stages]), (i / stages) & 1, wl, &none);
    *p.status = TC_ERR_DEVICE_TIMEOUT;
  }
  __syncthreads();
  tmem_fence_after();
  // This CTA's sums, [token][128 features], where the tiles were.
  const uint32_t mine = at + (uint32_t)(warp * 32 + lane) * 4;
#pragma unroll 1
  for (int c = 0; c < live; c += 16) {
    uint32_t v[16];
    tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + c, v);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (c + j < live) asm volatile("st.shared.b32 [%0], %1;" ::"r"(mine + (c + j) * 512), "r"(v[j]) : "memory");
  }
  tmem_fence_before();
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
  }
  // Four features of a token at a time, shared out over the cluster.
  const int shift = p.gated ? 4 : 5;
  for (int u = rank * kThreads + tid; u < live << shift; u += split * kThreads) {
    const int t = u >> shift, q = u & ((1 << shift) - 1);
    if (f0 + 4 * q >= p.o.features) continue;
    const uint32_t src = at + t * 512 + q * 16;
    float4 z = make_float4(0.f, 0.f, 0.f, 0.f), g = z;
    for (int r = 0; r < split; ++r) {
      const float4 v = peer_float4(p.gated ? src + 256 : src, r);
      z.x += v.x, z.y += v.y, z.z += v.z, z.w += v.w;
      if (p.gated) {
        const float4 w = peer_float4(src, r);
        g.x += w.x, g.y += w.y, g.z += w.z, g.w += w.w;
      }
    }
    finish4<T>(p, tok0 + t, f0 + 4 * q, z, g);
  }
  if (split > 1) cluster_sync();  // (the others have read this CTA's sums)
}

// --------------------------------------------------------------------- host

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// A matrix of `rows` rows of `cols` elements, in boxes of `box` rows by 64 elements.
bool encode(CUtensorMap* m, int dtype, const void* base, int64_t cols, int64_t rows, int64_t stride, int box) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t boxes[2] = {64, (cuuint32_t)box}, ones[2] = {1, 1};
  return fn && fn(m, dtype == TC_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                  const_cast<void*>(base), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;
constexpr size_t kSmemHalf = 112 * 1024, kSmemWhole = 224 * 1024;  // two CTAs an SM, or one

int sm_count(int device) {
  static int known[kMaxDevices];  // (a race writes the same value)
  if (!known[device]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    known[device] = n;
  }
  return known[device];
}

template <typename T>
cudaError_t launch(const LinearParams& p, int device, unsigned grid, size_t smem, const CUtensorMap& w,
                   const CUtensorMap& g, const CUtensorMap& x, cudaStream_t s) {
  static bool ready[kMaxDevices];
  if (!ready[device]) {
    const cudaError_t e =
        cudaFuncSetAttribute(linear_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemWhole);
    if (e != cudaSuccess) return e;
    ready[device] = true;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, linear_kernel<T>, p, w, g, x);
}

}  // namespace
}  // namespace tcd

using namespace tcd;

extern "C" tc_status tc_linear(const tc_linear_t* l, const tc_linear_call_t* c, int32_t* status, void* stream) {
  if (!l || !c || !status) return fail_with(TC_ERR_INVALID_ARG, "tc_linear: an argument is NULL");
  if (l->device < 0 || l->device >= kMaxDevices || l->in_features < 1 || l->out_features < 1 || c->n_tokens < 0 ||
      l->act < TC_ACT_NONE || l->act > TC_ACT_GELU_TANH)
    return fail_with(TC_ERR_INVALID_ARG, "tc_linear: a size, the device or the activation is out of range");
  if (l->dtype != TC_DT_BF16 && l->dtype != TC_DT_F16)
    return fail_with(TC_ERR_UNSUPPORTED, "tc_linear: the elements must be bf16 or f16");
  if (l->in_features > TC_LINEAR_MAX_FEATURES || l->out_features > TC_LINEAR_MAX_FEATURES ||
      c->n_tokens > TC_LINEAR_MAX_TOKENS)
    return fail_with(TC_ERR_CAPACITY, "tc_linear: more than 2^20 features or 2^24 tokens");
  if (!l->weight || kv_misaligned(l->weight, 16) || l->weight_stride % 8 != 0 || l->weight_stride < l->in_features ||
      (l->gate && (kv_misaligned(l->gate, 16) || l->gate_stride % 8 != 0 || l->gate_stride < l->in_features)))
    return fail_with(TC_ERR_INVALID_ARG,
                     "tc_linear: weights must be 16-byte aligned, with row strides that are multiples of 8 and hold a "
                     "row");
  if (kv_misaligned(l->bias, 2) || kv_misaligned(l->gate_bias, 2) || (l->gate_bias && !l->gate))
    return fail_with(TC_ERR_INVALID_ARG, "tc_linear: a bias is misaligned, or is a gate's where there is none");
  if (c->n_tokens == 0) return TC_OK;
  if (!c->x || kv_misaligned(c->x, 16) || c->x_stride % 8 != 0 || c->x_stride < l->in_features)
    return fail_with(TC_ERR_INVALID_ARG,
                     "tc_linear: x must be 16-byte aligned, with a row stride that is a multiple of 8 and holds a row");
  if (!c->out || kv_misaligned(c->out, 2) || c->out_stride < l->out_features || kv_misaligned(c->residual, 2) ||
      (c->residual && c->residual_stride < l->out_features))
    return fail_with(TC_ERR_INVALID_ARG, "tc_linear: out and residual must hold rows of out_features elements");
  KvDevice dev(l->device);
  if (!dev.ok) return fail_with(TC_ERR_CUDA, "tc_linear: cannot use the weights' device");
  const int sms = sm_count(l->device);
  if (sms < 1) return fail_with(TC_ERR_CUDA, "tc_linear: cannot use the weights' device");

  LinearParams p{};
  p.o.bias = static_cast<const uint16_t*>(l->bias);
  p.o.gate_bias = static_cast<const uint16_t*>(l->gate_bias);
  p.o.residual = static_cast<const uint16_t*>(c->residual);
  p.o.out = static_cast<uint16_t*>(c->out);
  p.o.residual_stride = c->residual_stride;
  p.o.out_stride = c->out_stride;
  p.o.n_tokens = c->n_tokens;
  p.o.features = l->out_features;
  p.o.act = l->act;
  const auto aligned = [&](int elements) {
    return !kv_misaligned(c->out, 2 * elements) && c->out_stride % elements == 0 &&
           (!c->residual || (!kv_misaligned(c->residual, 2 * elements) && c->residual_stride % elements == 0));
  };
  p.o.wide = aligned(16) ? 16 : aligned(4) ? 4 : 1;
  p.k_tiles = (l->in_features + 63) / 64;
  p.gated = l->gate != nullptr;
  p.status = status;
  p.wait_limit = c->wait_polls > 0 ? (int32_t)(c->wait_polls < 1 << 30 ? c->wait_polls : 1 << 30) : kLinearWaitLimit;
  p.withhold = c->withhold;

  p.tile = c->n_tokens >= 256 ? 256 : (c->n_tokens + 15) / 16 * 16;
  p.tok_tiles = (c->n_tokens + p.tile - 1) / p.tile;
  p.tmem_cols = 32;
  while (p.tmem_cols < p.tile) p.tmem_cols *= 2;
  const int rows = p.gated ? 64 : 128;
  const int64_t tiles = (int64_t)((l->out_features + rows - 1) / rows) * p.tok_tiles;
  const size_t stage = kWeightBytes + (size_t)p.tile * kRowBytes;
  const size_t room = p.tile > 128 ? kSmemWhole : kSmemHalf;
  p.split = 1;
  while (p.split < 8 && tiles * p.split * 2 <= (p.tile > 128 ? sms : 2 * sms) && p.k_tiles >= p.split * 2 * 2) p.split *= 2;
  p.stages = (int)((room - 1024) / stage);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  const int64_t grid = tiles * p.split;
  if (grid > INT32_MAX) return fail_with(TC_ERR_CAPACITY, "tc_linear: the output has too many tiles");

  CUtensorMap w, g, x;
  if (!encode(&w, l->dtype, l->weight, l->in_features, l->out_features, l->weight_stride, 64) ||
      (l->gate && !encode(&g, l->dtype, l->gate, l->in_features, l->out_features, l->gate_stride, 64)) ||
      !encode(&x, l->dtype, c->x, l->in_features, c->n_tokens, c->x_stride, p.tile))
    return fail_with(TC_ERR_UNSUPPORTED, "tc_linear: the sizes or strides do not fit a tensor map");
  if (!l->gate) g = w;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = 1024 + p.stages * stage;
  const cudaError_t e = l->dtype == TC_DT_BF16 ? launch<Bf16>(p, l->device, (unsigned)grid, smem, w, g, x, s)
                                               : launch<F16>(p, l->device, (unsigned)grid, smem, w, g, x, s);
  return e == cudaSuccess ? TC_OK : kv_cuda_fail(e, "tc_linear: ");
}
