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
// One CTA, eight warps: warp 0 loads by TMA (128-byte swizzle; rows and columns
// past the ends are zeros), warp 1 issues the products, all eight finish the
// outputs: from tensor memory, where a thread has one feature, to shared memory,
// and from there with neighbouring features in neighbouring threads.
//
// Bound: the weights' bytes, and in small calls latencies (setup, the first load,
// the cluster's meeting, the epilogue).  In continuous runs, us: one token of 2048 x 2048
// 4.3 to 4.5, or 4.65 to 4.9 where the weights of 40 layers pass in turn (340 MB, more than L2); 64 of 4096 x 6144
// 13.5 (3.7 TB/s); one gated of 2048 x 8192 13.2 (5.1 TB/s); 64 gated of 4096 x 14336 38.8 to
// 40.6 (6.1 to 5.8 TB/s; alone with cold caches 44 to 45.4, 5.2 to 5.4 TB/s).  24 steps of weights asked for at
// the start instead of the ring's: 3 to 9 % slower.  Weights told to leave L2 first: 1 to 2 %
// slower where 40 layers' pass in turn, one token 8 %.  (With four layers, some of whose weights
// then stay in L2, it looks up to 9 % faster.)
#include <cudaTypedefs.h>

#include "linear.h"

namespace tcd {
namespace {

constexpr int kThreads = 256;
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
// V floats of the shared memory of a CTA of the cluster.
template <bool PEER>
__device__ __forceinline__ void sums(uint32_t at, float (&v)[4]) {
  if (PEER)
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(at)
                 : "memory");
  else
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(at)
                 : "memory");
}
template <bool PEER>
__device__ __forceinline__ void sums(uint32_t at, float (&v)[1]) {
  if (PEER)
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[0]) : "r"(at) : "memory");
  else
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[0]) : "r"(at) : "memory");
}
template <typename T>
__device__ __forceinline__ void load_row(const uint16_t* p, float (&v)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const float2 a = T::unpack(w.x), b = T::unpack(w.y);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}
template <typename T>
__device__ __forceinline__ void load_row(const uint16_t* p, float (&v)[1]) {
  v[0] = T::unpack(*p).x;
}
template <typename T>
__device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(T::pack(v[0], v[1]), T::pack(v[2], v[3]));
}
template <typename T>
__device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[1]) {
  *p = (uint16_t)T::pack(v[0], 0.f);
}

// V: features of a thread of the epilogue: four where rows are aligned, else one, so that a warp still writes whole pieces
// of rows.
template <typename T, int SPLIT, bool GATED, int V>
__global__ void __launch_bounds__(kThreads, 2)
    linear_kernel(const LinearParams p, const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ CUtensorMap map_g, const __grid_constant__ CUtensorMap map_x) {
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ Hdr hdr;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % SPLIT, tile = blockIdx.x / SPLIT;
  constexpr int rows = GATED ? 64 : 128;
  const int tok0 = tile % p.tok_tiles * p.tile;
  const int f0 = tile / p.tok_tiles * rows;
  const int kt0 = p.k_tiles * rank / SPLIT, n = p.k_tiles * (rank + 1) / SPLIT - kt0;
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
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  // The next kernel's CTAs may take the places of those that end: tensor memory is allocated, so that none of this
  // kernel's CTAs can wait for it behind them.  The setup above touches only this CTA; everything read or written from
  // here on may belong to the kernel before.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 0 && lane == 0)
    // The first weights are on their way to L2 while the kernel before ends (L2 has what that one may still write).
    for (int i = 0; i < min(n, stages); ++i) {
      prefetch_tile(GATED ? &map_g : &map_w, (kt0 + i) * 64, f0);
      prefetch_tile(&map_w, (kt0 + i) * 64, GATED ? f0 : f0 + 64);
    }
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
      load_tile(dst, GATED ? &map_g : &map_w, k, f0, bar);
      load_tile(dst + kWeightBytes / 2, &map_w, k, GATED ? f0 : f0 + 64, bar);
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
  // What a thread finishes: V features of every dt-th token.  Biases and the first residuals are fetched while the
  // products run.
  constexpr int kParts = rows / V, dt = SPLIT * kThreads / kParts;
  constexpr int U = 16 / V / SPLIT ? 16 / V / SPLIT : 1;  // tokens at a time
  const LinearOut& o = p.o;
  const int part = tid % kParts, f = f0 + V * part;
  const bool mine_is_out = f < o.features;  // (four features are all there, or none)
  int t = rank * (kThreads / kParts) + tid / kParts;
  float bias[V], gate_bias[V], res[U][V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    bias[j] = o.bias && mine_is_out ? one<T>(o.bias + f + j) : 0.f;
    gate_bias[j] = GATED && o.gate_bias && mine_is_out ? one<T>(o.gate_bias + f + j) : 0.f;
  }
  const auto fetch = [&]() {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < V; ++j) res[u][j] = 0.f;
      if (o.residual && mine_is_out && t + u * dt < live)
        load_row<T>(o.residual + (int64_t)(tok0 + t + u * dt) * o.residual_stride + f, res[u]);
    }
  };
  fetch();
  // (after a wait that gave up as well: the issuer commits what it has issued)
  bool ok = bar_wait(smem_at(&hdr.done), 0, wl, abort);
  ok = __syncthreads_and(ok && !*abort);
  if (!ok && warp == 0 && lane == 0) {
    // What was issued has to end before this CTA goes on (waits bounded again): the products, and loads that no
    // product has waited for.
    const int wl = max(p.wait_limit, kLinearWaitLimit);
    int32_t none = 0;
    bar_wait(smem_at(&hdr.done), 0, wl, &none);
    for (int i = max(0, armed - stages); i < armed; ++i)
      if (!(held && i == 0)) bar_wait(smem_at(&hdr.full[i % stages]), (i / stages) & 1, wl, &none);
    *p.status = TC_ERR_DEVICE_TIMEOUT;
  }
  __syncthreads();
  tmem_fence_after();
  // This CTA's sums, [token][128 features], where the tiles were: a warp has a quarter of the features and half of the
  // tokens.
  const int quarter = warp & 3;
  const uint32_t mine = at + (uint32_t)(quarter * 32 + lane) * 4;
  const int cut = (live + 31) / 32 * 16, c1 = warp < 4 ? min(cut, live) : live;
#pragma unroll 1
  for (int c = warp < 4 ? 0 : cut; c < c1; c += 16) {
    uint32_t v[16];
    tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + c, v);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (c + j < c1) asm volatile("st.shared.b32 [%0], %1;" ::"r"(mine + (c + j) * 512), "r"(v[j]) : "memory");
  }
  tmem_fence_before();
  if (SPLIT > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
  }
  uint32_t peer[SPLIT];
#pragma unroll
  for (int r = 0; r < SPLIT; ++r) {
    peer[r] = at + part * V * 4;
    if (SPLIT > 1) asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(peer[r]) : "r"(r));
  }
  if (mine_is_out) {
#pragma unroll 1
    while (t < live) {
      float z[U][SPLIT][V], g[U][SPLIT][V];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < SPLIT; ++r) {
          const int at_t = min(t + u * dt, live - 1) * 512;
          sums<(SPLIT > 1)>(peer[r] + at_t + (GATED ? 256 : 0), z[u][r]);
          if (GATED) sums<(SPLIT > 1)>(peer[r] + at_t, g[u][r]);
        }
      with_act(o.act, [&](auto act) {
        constexpr int kAct = decltype(act)::kAct;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float y[V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            float a = z[u][0][j], b = GATED ? g[u][0][j] : 0.f;
#pragma unroll
            for (int r = 1; r < SPLIT; ++r) {
              a += z[u][r][j];
              if (GATED) b += g[u][r][j];
            }
            a += bias[j];
            y[j] = (GATED ? a * activate(b + gate_bias[j], kAct) : activate(a, kAct)) + res[u][j];
          }
          if (t + u * dt < live) store_row<T>(o.out + (int64_t)(tok0 + t + u * dt) * o.out_stride + f, y);
        }
      });
      t += U * dt;
      if (t < live) fetch();
    }
  }
  if (SPLIT > 1) cluster_sync();  // (the others have read this CTA's sums)
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

constexpr size_t kSmemHalf = 112 * 1024, kSmemWhole = 224 * 1024;  // two CTAs an SM, or one

int sm_count(int device) {
  static int known[kLinearDevices];  // (a race writes the same value)
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

template <typename T, int SPLIT, bool GATED, int V>
cudaError_t launch(const LinearParams& p, int device, unsigned grid, size_t smem, const CUtensorMap& w,
                   const CUtensorMap& g, const CUtensorMap& x, cudaStream_t s) {
  const auto kernel = linear_kernel<T, SPLIT, GATED, V>;
  static bool ready[kLinearDevices];
  if (!ready[device]) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemWhole);
    if (e != cudaSuccess) return e;
    ready[device] = true;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = SPLIT;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT > 1 ? 2 : 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, kernel, p, w, g, x);
}

template <typename T, bool GATED, int V>
cudaError_t launch_split(const LinearParams& p, int device, unsigned grid, size_t smem, const CUtensorMap& w,
                         const CUtensorMap& g, const CUtensorMap& x, cudaStream_t s) {
  switch (p.split) {
    case 2: return launch<T, 2, GATED, V>(p, device, grid, smem, w, g, x, s);
    case 4: return launch<T, 4, GATED, V>(p, device, grid, smem, w, g, x, s);
    case 8: return launch<T, 8, GATED, V>(p, device, grid, smem, w, g, x, s);
    default: return launch<T, 1, GATED, V>(p, device, grid, smem, w, g, x, s);
  }
}

template <typename T>
cudaError_t launch_few(const LinearParams& p, int device, unsigned grid, size_t smem, const CUtensorMap& w,
                       const CUtensorMap& g, const CUtensorMap& x, cudaStream_t s) {
  if (p.gated)
    return p.o.wide > 1 ? launch_split<T, true, 4>(p, device, grid, smem, w, g, x, s)
                        : launch_split<T, true, 1>(p, device, grid, smem, w, g, x, s);
  return p.o.wide > 1 ? launch_split<T, false, 4>(p, device, grid, smem, w, g, x, s)
                      : launch_split<T, false, 1>(p, device, grid, smem, w, g, x, s);
}

// How a call is computed, and about how long it takes.
//
// The sizes and the number of SMs decide, and not where the output lies: the order of a sum follows from this, and the same
// inputs have the same bits in any output.  (Where rows of 1024 or 2732 features lie at odd addresses and the way with the
// lowest estimate would be another one for that: 11 % less to 14 % more time than with it, for 130 to 520 tokens.)
//
// Up to 128 tokens are one tile (pairs were never more than 4 % faster there).  More take the way with the lowest estimate.
// The estimates' constants are a fit to 209 calls (in_features 304 to 14336, out_features 500 to 14336, with and without
// a gate, 1 to 4000 tokens, each measured in all four ways): the way that they choose took 1.2 % longer than the best of
// the four on average and 16 % at most.  A few of those calls, in us, as tokens of a tile 256 / 128 / pairs with 128 rows of
// the weights a CTA / 64:
//   4096 x 6144, 256 tokens     24.2 / 21.9 / 25.8 / 24.1       14336 x 4096, 512 tokens    50.9 / 54.4 / 71.0 / 69.8
//   1000 x 2731, 512 tokens     15.8 / 14.6 / 14.8 / 11.2       4096 x 14336 gated, 512     89.2 / 93.8 / 72.5 / 117.4
struct Plan {
  double ns;
  bool many;         // linear_pair.cu
  int tile, tok_tiles, split;
  int64_t grid;      // CTAs, or pairs
};

// Bytes of the weights at 6 TB/s.
double weights_ns(const tc_linear_t& l) {
  return (l.gate ? 4. : 2.) * l.in_features * l.out_features / 6000.;
}

// Tiles of up to `cap` tokens, of about the same size each.  Tiles of 128 leave room for two CTAs an SM, larger ones for
// one.  The sums are cut while that keeps everything resident at once and each part has two steps or more; in clusters
// of at most four where a CTA takes a whole SM (of eight, some had to wait for the others: 256 tokens of 2048 x 2048
// 17.8 us instead of 10.3), and in halves only (clusters of six do not fill the GPU either: 64 tokens of 4096 x 6144
// 21.8 us instead of 14.2 with four).
Plan plan_few(const tc_linear_t& l, int n_tokens, int cap, int sms) {
  const bool wide = l.out_features % 4 == 0;  // (if the output's and the residual's rows are aligned as well)
  Plan r{};
  r.tok_tiles = (n_tokens + cap - 1) / cap;
  r.tile = ((n_tokens + r.tok_tiles - 1) / r.tok_tiles + 15) / 16 * 16;
  const bool alone = r.tile > 128;
  const int k_tiles = (l.in_features + 63) / 64, rows = l.gate ? 64 : 128;
  const int64_t tiles = (int64_t)((l.out_features + rows - 1) / rows) * r.tok_tiles;
  r.split = 1;
  while (r.split < (alone ? 4 : 8) && tiles * r.split * 2 <= (alone ? sms : 2 * sms) && k_tiles >= r.split * 4)
    r.split *= 2;
  r.grid = tiles * r.split;
  const double turns = (double)((r.grid + sms - 1) / sms);
  const double products = turns * ((k_tiles + r.split - 1) / r.split) * (60. + 1.5 * r.tile);
  r.ns = 5500. + (products > weights_ns(l) ? products : weights_ns(l)) + (wide ? 18. : 43.) * r.tile / r.split * turns;
  return r;
}

Plan plan_many(const tc_linear_t& l, int n_tokens, int rows, int sms) {
  Plan r{};
  r.many = true;
  r.tile = rows;
  r.split = 1;
  r.tok_tiles = (n_tokens + 255) / 256;
  const int features = l.gate ? rows : 2 * rows, pairs = sms / 2 > 0 ? sms / 2 : 1;
  const int64_t tiles = (int64_t)((l.out_features + features - 1) / features) * r.tok_tiles;
  r.grid = tiles < pairs ? tiles : pairs;
  const double products =
      (double)((tiles + pairs - 1) / pairs) * ((l.in_features + 63) / 64) * (rows == 128 ? 333. : 310.);
  r.ns = 3000. + (products > weights_ns(l) ? products : weights_ns(l)) + 29. * rows;
  // (tiles are counted in 32 bits there)
  if (tiles > INT32_MAX / 2) r.grid = tiles;
  return r;
}

// Rows of 2-byte elements that a call reads or writes.
struct Rows {
  const void* base;
  int64_t n, width, stride;
};
// Whether an element lies in both.  Of different strides (of several rows each) only that neither lies behind the other
// is asked for.
bool overlap(const Rows& a, const Rows& b) {
  if (!a.base || !b.base) return false;
  const int64_t pa = (int64_t)((uintptr_t)a.base / 2), pb = (int64_t)((uintptr_t)b.base / 2);
  if (pa + (a.n - 1) * a.stride + a.width <= pb || pb + (b.n - 1) * b.stride + b.width <= pa) return false;
  const int64_t s = a.n > 1 ? a.stride : b.stride;
  if ((a.n == 1 && b.n == 1) || (a.n > 1 && b.n > 1 && a.stride != b.stride)) return true;
  const int64_t r = ((pb - pa) % s + s) % s;  // where rows of b begin in rows of a
  return r < a.width || r + b.width > s;
}

}  // namespace
}  // namespace tcd

using namespace tcd;

extern "C" tc_status tc_linear(const tc_linear_t* l, const tc_linear_call_t* c, int32_t* status, void* stream) {
  if (!l || !c || !status) return fail_with(TC_ERR_INVALID_ARG, "tc_linear: an argument is NULL");
  if (l->device < 0 || l->device >= kLinearDevices || l->in_features < 1 || l->out_features < 1 || c->n_tokens < 0 ||
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
  const Rows out{c->out, c->n_tokens, l->out_features, c->out_stride};
  const Rows residual{c->residual, c->n_tokens, l->out_features, c->residual_stride};
  const bool in_place = c->residual == c->out && (c->n_tokens == 1 || c->residual_stride == c->out_stride);
  if (overlap(out, {c->x, c->n_tokens, l->in_features, c->x_stride}) || (!in_place && overlap(out, residual)) ||
      overlap(out, {l->weight, l->out_features, l->in_features, l->weight_stride}) ||
      overlap(out, {l->gate, l->out_features, l->in_features, l->gate_stride}) ||
      overlap(out, {l->bias, 1, l->out_features, l->out_features}) ||
      overlap(out, {l->gate_bias, 1, l->out_features, l->out_features}))
    return fail_with(TC_ERR_INVALID_ARG, "tc_linear: out overlaps what the call reads (only the residual may be out itself)");
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
  p.o.wide = l->out_features % 4 == 0 && !kv_misaligned(c->out, 8) && c->out_stride % 4 == 0 &&
                     (!c->residual || (!kv_misaligned(c->residual, 8) && c->residual_stride % 4 == 0))
                 ? 4
                 : 1;
  p.k_tiles = (l->in_features + 63) / 64;
  p.gated = l->gate != nullptr;
  p.status = status;
  p.wait_limit = c->wait_polls > 0 ? (int32_t)(c->wait_polls < 1 << 30 ? c->wait_polls : 1 << 30) : kLinearWaitLimit;
  p.withhold = c->withhold;

  Plan plan = plan_few(*l, c->n_tokens, 256, sms);
  if (c->n_tokens > 128)
    for (const Plan& other : {plan_few(*l, c->n_tokens, 128, sms), plan_many(*l, c->n_tokens, 128, sms),
                              plan_many(*l, c->n_tokens, 64, sms)})
      if (other.ns < plan.ns) plan = other;
  if (plan.grid > INT32_MAX / 2) return fail_with(TC_ERR_CAPACITY, "tc_linear: the output has too many tiles");
  p.tile = plan.tile;
  p.tok_tiles = plan.tok_tiles;
  p.split = plan.split;
  const size_t stage = kWeightBytes + (size_t)p.tile * kRowBytes;
  if (!plan.many) {
    p.tmem_cols = 32;
    while (p.tmem_cols < p.tile) p.tmem_cols *= 2;
    p.stages = (int)(((p.tile > 128 ? kSmemWhole : kSmemHalf) - 1024) / stage);
    if (p.stages > kMaxStages) p.stages = kMaxStages;
  }
  const int w_box = plan.many ? plan.tile : 64, x_box = plan.many ? 128 : plan.tile;

  CUtensorMap w, g, x;
  if (!encode(&w, l->dtype, l->weight, l->in_features, l->out_features, l->weight_stride, w_box) ||
      (l->gate && !encode(&g, l->dtype, l->gate, l->in_features, l->out_features, l->gate_stride, w_box)) ||
      !encode(&x, l->dtype, c->x, l->in_features, c->n_tokens, c->x_stride, x_box))
    return fail_with(TC_ERR_UNSUPPORTED, "tc_linear: the sizes or strides do not fit a tensor map");
  if (!l->gate) g = w;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (plan.many) {
    e = launch_linear_pair(p, l->device, l->dtype, (int)plan.grid, w, g, x, s);
  } else {
    const size_t smem = 1024 + p.stages * stage;
    e = l->dtype == TC_DT_BF16 ? launch_few<Bf16>(p, l->device, (unsigned)plan.grid, smem, w, g, x, s)
                               : launch_few<F16>(p, l->device, (unsigned)plan.grid, smem, w, g, x, s);
  }
  return e == cudaSuccess ? TC_OK : kv_cuda_fail(e, "tc_linear: ");
}
