// Projections of many tokens (linear.cu has the few): pairs of SMs on one tile.
//
// A pair of CTAs (a cluster of two) computes 256 tokens by 256 rows of the
// weights (with a gate: 128 of it and the same 128 of the weights, side by
// side), so that each SM reads half of both operands for a whole tile's
// product.  Each CTA loads its 128 tokens and its half of the weights' rows
// into a ring of its own; the first CTA's issuer multiplies over both
// (cta_group::2), and each CTA's tensor memory receives its 128 tokens' sums.
// Two accumulators: a tile's outputs are finished beside the next one's products.
//
// One CTA, 10 warps: warp 0 loads by TMA, warp 1 issues the products (first
// CTA), warps 2 to 9 finish the outputs, 32 tokens and half of the features
// each.  Tensor memory gives a thread one token's sums; they are turned in
// shared memory, so that a thread has the same features of many tokens: biases stay
// in registers, rows are read and written in whole pieces whatever their
// alignment, and the code is a short loop.  (A thread takes several tokens' values
// before it stores the first: one by one nothing would overlap.)  Rows on
// whole fours are still cheaper: 1111 tokens of 1000 x 2731 take 17.9 us, of 1000 x 2732 14.2.
//
// Bound: the tensor cores, busy 88 to 90 % of the kernel, and the power limit in
// continuous runs: 8192 tokens of 14336 x 4096 527 us in short runs and 609 in
// continuous ones, 4096 gated of 4096 x 14336 511 and 584.
#include <type_traits>

#include "linear.h"

namespace tcd {
namespace {

constexpr int kThreads = 320, kStages = 6, kFinishers = 8;
constexpr uint32_t kHalf = 128 * kRowBytes, kStage = 2 * kHalf;
// A warp's 32 x 32 sums: four floats i of row r lie in place i ^ (r % 8), so that threads with a row each and threads
// with four floats each both find all banks.
__device__ __forceinline__ int sums_place(int r, int i) { return r * 32 + 4 * (i ^ (r & 7)); }

struct Hdr {
  uint64_t full[kStages];   // (first CTA's) both CTAs' loads
  uint64_t empty[kStages];
  uint64_t sums[2];         // an accumulator is complete
  uint64_t read[2];         // (first CTA's) both CTAs have read it
  uint64_t drain;
  uint32_t tmem;
  int32_t abort;
  int32_t armed;            // stages that this CTA has armed
};
constexpr size_t kSmem = 1024 + kStages * kStage + kFinishers * 32 * 32 * sizeof(float) + sizeof(Hdr);
static_assert(kSmem <= 232448, "shared memory of one CTA");

__device__ __forceinline__ uint32_t in_first(uint32_t a) {  // the same place in the pair's first CTA
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t in_second(uint32_t a) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void pair_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// (relaxed: it orders nothing, and a release waits for the thread's loads: 0.8 us a step instead of 0.3)
__device__ __forceinline__ void pair_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool pair_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
// bar_wait for a barrier that the other CTA arrives at.
__device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity, int limit, volatile int32_t* abort) {
  if (pair_try(bar, parity)) return true;
  int i = 1;
#pragma unroll 1
  do {
    if (pair_try(bar, parity)) return true;
    ++i;
  } while (i < limit && !*abort);
  *abort = 1;
  return false;
}
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_product(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
// Arrives at the barrier in both CTAs when the products so far are done.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
// Waits for the loads; no use of their registers can be moved ahead of it.
__device__ __forceinline__ void tmem_arrived(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// What one warp finishes of a tile: 32 tokens, in chunks of W features (with a gate two halves of W columns lie side by
// side in a row).  V: features of a thread, of every kRows-th token: four where rows are aligned, else one, so that a
// store still covers whole pieces of rows (two or four features of a thread, stored one by one, take twice as long).
template <typename T, bool GATED, int V>
struct Finish {
  static constexpr int W = GATED ? 16 : 32, kRows = 32 * V / W;
  static constexpr int kN = 32 / kRows < 8 ? 32 / kRows : 8, kBatches = 32 / kRows / kN;  // tokens of a batch
  using Held = std::conditional_t<V == 4, uint2, uint32_t>;             // elements of a token
  const LinearOut& o;
  int rows, row, col, first;  // tokens from this thread's first one on; that one; its first feature of a chunk, and of all
  const uint16_t* residual;
  uint16_t* out;

  __device__ Finish(const LinearOut& out_, int tok0, int f0) : o(out_) {
    const int lane = threadIdx.x & 31;
    row = lane / (W / V);
    col = lane % (W / V) * V;
    rows = o.n_tokens - tok0 - row;
    first = f0 + col;
    residual = o.residual ? o.residual + (int64_t)(tok0 + row) * o.residual_stride + first : nullptr;
    out = o.out + (int64_t)(tok0 + row) * o.out_stride + first;
  }
  // Residuals of batch b of chunk c.
  __device__ __forceinline__ void fetch(int c, int b, Held (&r)[kN]) const {
    if (!residual || o.features - first - c * W < V) return;
    const int64_t step = kRows * o.residual_stride;
    const uint16_t* p = residual + c * W + b * kN * step;
#pragma unroll
    for (int i = 0; i < kN; ++i, p += step)
      if ((b * kN + i) * kRows < rows) {
        if constexpr (V == 4)
          r[i] = *reinterpret_cast<const uint2*>(p);
        else
          r[i] = *p;
      }
  }
  // Batch b of chunk c: all values, then all stores (one by one nothing would overlap: 300 cycles each).
  template <int ACT>
  __device__ __forceinline__ void finish(const float* sums, int c, int b, const Held (&r)[kN], const float (&bias)[V],
                                         const float (&gate_bias)[V]) const {
    if (o.features - first - c * W < V) return;
    Held y[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at_row = row + (b * kN + i) * kRows;
      float z[V];
      if constexpr (V == 4) {
        const float4 v = *reinterpret_cast<const float4*>(sums + sums_place(at_row, col / 4));
        z[0] = v.x, z[1] = v.y, z[2] = v.z, z[3] = v.w;
      } else {
        z[0] = sums[sums_place(at_row, col / 4) + col % 4];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) z[j] += bias[j];
      if constexpr (GATED) {
        float g[V];
        if constexpr (V == 4) {
          const float4 v = *reinterpret_cast<const float4*>(sums + sums_place(at_row, (W + col) / 4));
          g[0] = v.x, g[1] = v.y, g[2] = v.z, g[3] = v.w;
        } else {
          g[0] = sums[sums_place(at_row, (W + col) / 4) + col % 4];
        }
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] *= activate(g[j] + gate_bias[j], ACT);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] = activate(z[j], ACT);
      }
      if (residual) {
        if constexpr (V == 4) {
          const float2 d = T::unpack(r[i].x), e = T::unpack(r[i].y);
          z[0] += d.x, z[1] += d.y, z[2] += e.x, z[3] += e.y;
        } else {
          z[0] += T::unpack(r[i]).x;
        }
      }
      if constexpr (V == 4)
        y[i] = make_uint2(T::pack(z[0], z[1]), T::pack(z[2], z[3]));
      else
        y[i] = T::pack(z[0], 0.f);
    }
    const int64_t step = kRows * o.out_stride;
    uint16_t* p = out + c * W + b * kN * step;
#pragma unroll
    for (int i = 0; i < kN; ++i, p += step)
      if ((b * kN + i) * kRows < rows) {
        if constexpr (V == 4)
          *reinterpret_cast<uint2*>(p) = y[i];
        else
          *p = (uint16_t)y[i];
      }
  }
  // A bias of this thread's features of chunk c.
  __device__ __forceinline__ void get(const uint16_t* p, int c, float (&v)[V]) const {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = p && first + c * W + j < o.features ? one<T>(p + first + c * W + j) : 0.f;
  }
};

// The tiles of a pair, of which a warp finishes its 32 tokens and half of the features.
template <typename T, bool GATED, int V>
__device__ __forceinline__ void finish_tile(const LinearParams& p, Hdr* hdr, float* pass, uint32_t acc, int a, int n,
                                            int tok0, int f0, int cols, bool& ok) {
  using F = Finish<T, GATED, V>;
  const int lane = threadIdx.x & 31, chunks = cols / F::W;
  const F fin(p.o, tok0, f0);
  typename F::Held res[F::kN] = {}, now[F::kN];
  float bias[V], gate_bias[V];
  fin.fetch(0, 0, res);
  fin.get(p.o.bias, 0, bias);
  fin.get(GATED ? p.o.gate_bias : nullptr, 0, gate_bias);
  ok = __all_sync(0xffffffffu, pair_wait(smem_at(&hdr->sums[a]), (n >> 1) & 1, p.wait_limit, &hdr->abort));
  if (!ok) return;
  tmem_fence_after();
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    uint32_t v[32];
    __syncwarp();  // (the chunk before has been read, by threads that went ways of their own)
    tmem_ld16(acc + (GATED ? p.tile : 0) + c * F::W, v);
    tmem_ld16(acc + (GATED ? 0 : 16) + c * F::W, v + 16);
    tmem_arrived(v);
    tmem_arrived(v + 16);
    if (c + 1 == chunks) {  // the accumulator has been read
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) pair_arrive(in_first(smem_at(&hdr->read[a])));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<uint4*>(pass + sums_place(lane, i)) =
          make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    __syncwarp();
#pragma unroll 1
    for (int b = 0; b < F::kBatches; ++b) {
#pragma unroll
      for (int i = 0; i < F::kN; ++i) now[i] = res[i];
      // (the next residuals are on their way meanwhile)
      if (b + 1 < F::kBatches)
        fin.fetch(c, b + 1, res);
      else if (c + 1 < chunks)
        fin.fetch(c + 1, 0, res);
      with_act(p.o.act, [&](auto act) {
        fin.template finish<decltype(act)::kAct>(pass, c, b, now, bias, gate_bias);
      });
    }
    if (c + 1 < chunks) {
      fin.get(p.o.bias, c + 1, bias);
      fin.get(GATED ? p.o.gate_bias : nullptr, c + 1, gate_bias);
    }
  }
}

template <typename T, bool GATED, int V>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const LinearParams p, const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ CUtensorMap map_g, const __grid_constant__ CUtensorMap map_x) {
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* base = smem + ((1024 - (smem_at(smem) & 1023)) & 1023);
  float* turn = reinterpret_cast<float*>(base + kStages * kStage);
  Hdr* hdr = reinterpret_cast<Hdr*>(turn + kFinishers * 32 * 32);
  const uint32_t at = smem_at(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  volatile int32_t* abort = &hdr->abort;
  const int wl = p.wait_limit, kt = p.k_tiles, nb = p.tile;  // weights' rows of a CTA
  const int wide = GATED ? nb : 2 * nb;                    // features of a tile
  const int tok_tiles = p.tok_tiles, tiles = tok_tiles * ((p.o.features + wide - 1) / wide);
  const bool held = p.withhold != 0 && blockIdx.x == 0;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(smem_at(&hdr->full[s]), 2);
      bar_init(smem_at(&hdr->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      bar_init(smem_at(&hdr->sums[a]), 1);
      bar_init(smem_at(&hdr->read[a]), 2 * kFinishers);
    }
    bar_init(smem_at(&hdr->drain), 1);
    hdr->abort = 0;
    hdr->armed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(&hdr->tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tmem_fence_before();
  cluster_sync();
  tmem_fence_after();
  // (linear.cu says why here)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t tmem = hdr->tmem;
  // Tiles in bands of 8 tiles of tokens, the features' tiles outside: what runs at a time shares both operands.
  const auto place = [&](int t, int& tm, int& tf) {
    constexpr int kBand = 8;
    const int per = kBand * (tiles / tok_tiles), band = t / per, r = t - band * per;
    const int deep = min(kBand, tok_tiles - band * kBand);
    tf = r / deep;
    tm = band * kBand + r - tf * deep;
  };

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      const uint32_t bytes = kHalf + (uint32_t)nb * kRowBytes;
      for (int t = pair; t < tiles && ok; t += pairs) {
        int tm, tf;
        place(t, tm, tf);
        const CUtensorMap* mb = GATED && rank == 0 ? &map_g : &map_w;
        const int row = GATED ? tf * nb : (2 * tf + rank) * nb, tok = (2 * tm + rank) * 128;
        for (int i = 0; i < kt; ++i, ++it) {
          const int s = it % kStages, turn_no = it / kStages;
          if (turn_no > 0 && !bar_wait(smem_at(&hdr->empty[s]), (turn_no - 1) & 1, wl, abort)) {
            ok = false;
            break;
          }
          if (held && it == 0) continue;
          const uint32_t bar = in_first(smem_at(&hdr->full[s])), dst = at + s * kStage;
          pair_expect(bar, bytes);
          pair_load(dst, &map_x, i * 64, tok, bar);
          pair_load(dst + kHalf, mb, i * 64, row, bar);
        }
      }
      hdr->armed = it;
      // (the issuer's arrivals here come from another CTA: this one stays until they are in)
      for (int i = max(0, it - kStages); i < it && ok; ++i)
        ok = bar_wait(smem_at(&hdr->empty[i % kStages]), (i / kStages) & 1, wl, abort);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t id = product_desc<T>(256, 2 * nb);
      int it = 0, n = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs, ++n) {
        const int a = n & 1;
        if (n > 1 && !pair_wait(smem_at(&hdr->read[a]), ((n >> 1) - 1) & 1, wl, abort)) break;
        tmem_fence_after();
        for (int i = 0; i < kt; ++i, ++it) {
          const int s = it % kStages;
          if (!pair_wait(smem_at(&hdr->full[s]), (it / kStages) & 1, wl, abort)) {
            ok = false;
            break;
          }
          tmem_fence_after();
          const uint64_t x = tile_desc(at + s * kStage), w = tile_desc(at + s * kStage + kHalf);
#pragma unroll
          for (int e = 0; e < 4; ++e) pair_product(tmem + a * 256, x + 2 * e, w + 2 * e, id, i > 0 || e > 0);
          pair_commit(smem_at(&hdr->empty[s]));
        }
        if (ok) pair_commit(smem_at(&hdr->sums[a]));
      }
    }
    __syncwarp();
  } else {
    const int half = (warp - 2) >> 2, quarter = warp & 3;
    float* pass = turn + (warp - 2) * 32 * 32;
    int n = 0;
    for (int t = pair; t < tiles; t += pairs, ++n) {
      int tm, tf;
      place(t, tm, tf);
      const int a = n & 1, tok0 = (2 * tm + rank) * 128 + quarter * 32;
      const int cols = wide / 2;
      bool ok;
      finish_tile<T, GATED, V>(p, hdr, pass, tmem + ((uint32_t)(quarter * 32) << 16) + a * 256 + half * cols, a, n, tok0,
                               tf * wide + half * cols, cols, ok);
      if (!ok) break;
    }
  }

  tmem_fence_before();
  cluster_sync();
  // A wait that ran out in either CTA: what the pair has issued has to end before it leaves (waits bounded again).
  int32_t other;
  asm volatile("ld.shared::cluster.b32 %0, [%1];"
               : "=r"(other)
               : "r"(rank ? in_first(smem_at(&hdr->abort)) : in_second(smem_at(&hdr->abort)))
               : "memory");
  if (*abort || other) {
    const int wl = max(p.wait_limit, kLinearWaitLimit);
    int32_t none = 0;
    if (warp == 1 && lane == 0) {
      // (in both CTAs, behind the issuer's other arrivals there)
      if (rank == 0) pair_commit(smem_at(&hdr->drain));
      pair_wait(smem_at(&hdr->drain), 0, wl, &none);
    }
    if (rank == 0 && tid == 0) {
      // (the arrivals that a CTA which stopped earlier has left out)
      int32_t theirs;
      asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(theirs) : "r"(in_second(smem_at(&hdr->armed))) : "memory");
      const int mine = hdr->armed, most = max(mine, theirs);
      for (int i = max(0, most - kStages); i < most; ++i) {
        const uint32_t bar = smem_at(&hdr->full[i % kStages]);
        if (i >= mine || (held && i == 0)) pair_arrive(in_first(bar));
        if (i >= theirs) pair_arrive(in_first(bar));
        pair_wait(bar, (i / kStages) & 1, wl, &none);
      }
      *p.status = TC_ERR_DEVICE_TIMEOUT;
    }
    __syncwarp();
  }
  cluster_sync();
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <typename T, bool GATED, int V>
cudaError_t launch(const LinearParams& p, int device, int pairs, const CUtensorMap& w, const CUtensorMap& g,
                   const CUtensorMap& x, cudaStream_t s) {
  static bool ready[kLinearDevices];
  if (!ready[device]) {
    const cudaError_t e =
        cudaFuncSetAttribute(linear_pair_kernel<T, GATED, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    ready[device] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  return cudaLaunchKernelEx(&cfg, linear_pair_kernel<T, GATED, V>, p, w, g, x);
}

}  // namespace

cudaError_t launch_linear_pair(const LinearParams& p, int device, int dtype, int pairs, const CUtensorMap& w,
                               const CUtensorMap& g, const CUtensorMap& x, cudaStream_t s) {
  const auto go = [&](auto type) {
    using T = decltype(type);
    if (p.gated)
      return p.o.wide > 1 ? launch<T, true, 4>(p, device, pairs, w, g, x, s)
                          : launch<T, true, 1>(p, device, pairs, w, g, x, s);
    return p.o.wide > 1 ? launch<T, false, 4>(p, device, pairs, w, g, x, s)
                        : launch<T, false, 1>(p, device, pairs, w, g, x, s);
  };
  return dtype == TC_DT_BF16 ? go(Bf16()) : go(F16());
}

}  // namespace tcd
