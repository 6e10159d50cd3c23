// Kernels that write and rearrange the paged key-value cache: the append of
// new tokens (norms, rotation, write), page copies, the compaction of an
// accepted branch, and the masks of drafted trees.  All of them move bytes;
// none has arithmetic worth a tensor core.
#include <climits>

#include "kv_cache.h"

namespace tcd {

static_assert(TC_KV_MAX_BATCH == 65536 && TC_PATH_MAX == 256, "the messages name these");

tc_status kv_check(const char* who, const tc_kv_t* kv) {
  if (!kv) return kv_fail(TC_ERR_INVALID_ARG, who, ": the cache is NULL");
  if (!kv->pool || kv_misaligned(kv->pool, 16) || kv->layers < 1 || kv->pages < 1 || kv->kv_heads < 1 ||
      kv->device < 0)
    return kv_fail(TC_ERR_INVALID_ARG, who, ": the cache wants a 16-byte aligned pool and sizes >= 1");
  if ((kv->dtype != TC_DT_BF16 && kv->dtype != TC_DT_F16) || (kv->head_dim != 64 && kv->head_dim != 128) ||
      (kv->page_size != 16 && kv->page_size != 32 && kv->page_size != 64 && kv->page_size != 128))
    return kv_fail(TC_ERR_UNSUPPORTED,
                   who, ": the cache wants bf16 or f16, head_dim 64 or 128, page_size 16, 32, 64 or 128");
  if (kv->kv_heads > 65535) return kv_fail(TC_ERR_CAPACITY, who, ": more than 65535 kv_heads");
  return TC_OK;
}

tc_status kv_check_tokens(const char* who, const tc_tokens_t* t, bool rows) {
  if (!t || t->batch < 1 || t->n_tokens < 0 || !t->ctx_lens || (rows && !t->cu_tokens))
    return kv_fail(TC_ERR_INVALID_ARG, who, ": the tokens want batch >= 1, cu_tokens and ctx_lens");
  if (t->batch > TC_KV_MAX_BATCH)
    return kv_fail(TC_ERR_CAPACITY, who, ": more than 65536 sequences");
  return TC_OK;
}

KvView kv_view(const tc_kv_t* kv, int32_t layer) {
  const size_t page_bytes = (size_t)4 * kv->kv_heads * kv->page_size * kv->head_dim;
  KvView v;
  v.base = static_cast<uint8_t*>(kv->pool) + (size_t)layer * kv->pages * page_bytes;
  v.pages = kv->pages;
  v.kv_heads = kv->kv_heads;
  v.page_size = kv->page_size;
  v.page_shift = __builtin_ctz((unsigned)kv->page_size);
  v.keep = kv->keep_status != 0;
  return v;
}

namespace {

constexpr int kBlock = 256;
constexpr int kBlockWarps = kBlock / 32;

// ------------------------------------------------------------------ append

struct AppendParams {
  KvView kv;
  TokensView tok;
  const uint8_t* qkv;
  int64_t qkv_stride;  // elements
  int32_t q_heads;
  const uint8_t* q_weight;
  const uint8_t* k_weight;
  float eps;
  const float* rope;
  int32_t rope_len;
  const int32_t* positions;
  int32_t interleaved;
  uint8_t* q_out;
  int64_t q_out_stride;
  int32_t* status;
  int32_t split;       // warps per token
};

// The sequence b with cu[b] <= i < cu[b + 1], or -1: each round the warp's
// lanes cut the range into 32 parts (two rounds up to 1024 sequences, where a
// binary search would take ten dependent loads).
__device__ __forceinline__ int find_seq(const int32_t* cu, int batch, int i, int lane) {
  int lo = 0, n = batch;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool le = lane * step < n && __ldg(cu + at) <= i;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int part = m ? 31 - __clz(m) : 0;
    n = min(step, n - part * step);
    lo += part * step;
  }
  return __ldg(cu + lo) <= i && i < __ldg(cu + lo + 1) ? lo : -1;
}

// One warp per token and share of its heads.  A head of D elements is held by
// D / 8 lanes; lane l has elements [4 l, 4 l + 4) and D / 2 + [4 l, 4 l + 4), so
// that both members of every rotated pair, (i, i + D / 2) or (2 i, 2 i + 1), lie
// in one thread and the only exchange between lanes is the norm's sum.  A warp
// keeps its token's angles and the weights in registers across the heads and
// has U heads' loads in flight.  Norm and rotation are in 32 bits, rounded once
// when they are written; values are copied.  Bound: bytes (each row once in, once out), and
// at few tokens the chain of dependent reads that finds a token's place; so a
// token's heads are spread over more warps only where there are few tokens.
// Four blocks an SM (64 registers) against three: 74 against 80 us for 15,925
// tokens of 32 + 2 x 8 heads of 128 (5.3 TB/s); several tokens a warp with the
// next one's place looked up ahead: 81 us; twice the warps per token: 112 us.
template <typename T, int D, int U>
__global__ void __launch_bounds__(kBlock, 4) append_kernel(const AppendParams p) {
  constexpr int L = D / 8;    // lanes per head
  constexpr int HPW = 32 / L; // heads per warp and round
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kBlockWarps + (threadIdx.x >> 5);
  const int64_t n_work = (int64_t)p.tok.n_tokens * p.split;
  if (w >= n_work) {
    // The last warps look at one sequence each: its status.
    const int64_t b = w - n_work;
    if (b >= p.tok.batch) return;
    SeqSpan s;
    bool ok = seq_span(p.tok, p.kv.page_size, (int)b, &s);
    if (ok && s.n > 0) {
      const int first = s.ctx >> p.kv.page_shift, last = (s.ctx + s.n - 1) >> p.kv.page_shift;
      const int32_t* row = p.tok.table + b * p.tok.width;
      for (int i = first + lane; i <= last; i += 32) ok &= (uint32_t)__ldg(row + i) < (uint32_t)p.kv.pages;
      if (p.rope)
        for (int i = lane; i < s.n; i += 32) {
          const int pos = p.positions ? __ldg(p.positions + s.row0 + i) : s.ctx + i;
          ok &= (uint32_t)pos < (uint32_t)p.rope_len;
        }
    }
    ok = __all_sync(0xffffffffu, ok);
    if (lane == 0) set_status(p.status, b, ok ? TC_OK : TC_ERR_BOUNDS, p.kv.keep);
    return;
  }
  const int i = (int)(w / p.split), part = (int)(w % p.split);
  const int heads = p.q_heads + 2 * p.kv.kv_heads;
  const int sub = lane / L, l = lane % L;
  const uint8_t* row = p.qkv + (int64_t)i * p.qkv_stride * 2 + l * 8;
  // The first heads' loads go out before the token's place is known.
  const int step = p.split * HPW;
  int h0 = part * HPW + sub;
  uint2 lo[U], hi[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * step;
    if (h < heads) {
      lo[u] = __ldcs(reinterpret_cast<const uint2*>(row + (int64_t)h * D * 2));
      hi[u] = __ldcs(reinterpret_cast<const uint2*>(row + (int64_t)h * D * 2 + D));
    }
  }
  const int b = find_seq(p.tok.cu, p.tok.batch, i, lane);
  SeqSpan s;
  if (b < 0 || !seq_span(p.tok, p.kv.page_size, b, &s)) return;
  const int slot = s.ctx + (i - s.row0);
  const int page = __ldg(p.tok.table + (int64_t)b * p.tok.width + (slot >> p.kv.page_shift));
  const int pos = p.positions ? __ldg(p.positions + i) : slot;
  if ((uint32_t)page >= (uint32_t)p.kv.pages || (p.rope && (uint32_t)pos >= (uint32_t)p.rope_len)) return;
  // Angles of this lane's four pairs: (c, s) of the low and of the high half.
  float2 cs[4] = {{1.f, 0.f}, {1.f, 0.f}, {1.f, 0.f}, {1.f, 0.f}};
  if (p.rope) {
    const float* r = p.rope + (int64_t)pos * D;
    const float4 a = __ldg(reinterpret_cast<const float4*>(r + (p.interleaved ? 4 * l : 8 * l)));
    const float4 c = __ldg(reinterpret_cast<const float4*>(r + (p.interleaved ? D / 2 + 4 * l : 8 * l + 4)));
    cs[0] = {a.x, a.y};
    cs[1] = {a.z, a.w};
    cs[2] = {c.x, c.y};
    cs[3] = {c.z, c.w};
  }
  uint2 wq[2], wk[2];
  if (p.q_weight) {
    wq[0] = __ldg(reinterpret_cast<const uint2*>(p.q_weight + l * 8));
    wq[1] = __ldg(reinterpret_cast<const uint2*>(p.q_weight + l * 8 + D));
  }
  if (p.k_weight) {
    wk[0] = __ldg(reinterpret_cast<const uint2*>(p.k_weight + l * 8));
    wk[1] = __ldg(reinterpret_cast<const uint2*>(p.k_weight + l * 8 + D));
  }
  uint8_t* q_row = p.q_out + (int64_t)i * p.q_out_stride * 2 + l * 8;
  const int64_t head_bytes = (int64_t)p.kv.page_size * D * 2;
  uint8_t* kv_row = p.kv.base + (int64_t)page * 2 * p.kv.kv_heads * head_bytes +
                    (int64_t)(slot & (p.kv.page_size - 1)) * D * 2 + l * 8;
  while (true) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * step;
      const bool is_q = h < p.q_heads, is_k = !is_q && h < p.q_heads + p.kv.kv_heads;
      float x[8];
      const uint2 a = lo[u], c = hi[u];
      float2 t = T::unpack(a.x); x[0] = t.x; x[1] = t.y;
      t = T::unpack(a.y); x[2] = t.x; x[3] = t.y;
      t = T::unpack(c.x); x[4] = t.x; x[5] = t.y;
      t = T::unpack(c.y); x[6] = t.x; x[7] = t.y;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      // (all lanes take part, whatever their head: the lanes of one head only add up among themselves)
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (h >= heads) continue;
      uint8_t* dst;
      if (is_q || is_k) {
        if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          const uint2 w0 = is_q ? wq[0] : wk[0], w1 = is_q ? wq[1] : wk[1];
          t = T::unpack(w0.x); x[0] *= r * t.x; x[1] *= r * t.y;
          t = T::unpack(w0.y); x[2] *= r * t.x; x[3] *= r * t.y;
          t = T::unpack(w1.x); x[4] *= r * t.x; x[5] *= r * t.y;
          t = T::unpack(w1.y); x[6] *= r * t.x; x[7] *= r * t.y;
        }
        if (p.rope) {
          if (p.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y0 = x[2 * e], y1 = x[2 * e + 1];
              x[2 * e] = y0 * cs[e].x - y1 * cs[e].y;
              x[2 * e + 1] = y1 * cs[e].x + y0 * cs[e].y;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y0 = x[e], y1 = x[e + 4];
              x[e] = y0 * cs[e].x - y1 * cs[e].y;
              x[e + 4] = y1 * cs[e].x + y0 * cs[e].y;
            }
          }
        }
        dst = is_q ? q_row + (int64_t)h * D * 2 : kv_row + (int64_t)(h - p.q_heads) * head_bytes;
        *reinterpret_cast<uint2*>(dst) = make_uint2(T::pack(x[0], x[1]), T::pack(x[2], x[3]));
        *reinterpret_cast<uint2*>(dst + D) = make_uint2(T::pack(x[4], x[5]), T::pack(x[6], x[7]));
      } else {
        dst = kv_row + (int64_t)(h - p.q_heads) * head_bytes;  // (the value heads' pages follow the key heads')
        *reinterpret_cast<uint2*>(dst) = a;
        *reinterpret_cast<uint2*>(dst + D) = c;
      }
    }
    h0 += U * step;
    if (h0 - sub >= heads) break;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * step;
      if (h < heads) {
        lo[u] = __ldcs(reinterpret_cast<const uint2*>(row + (int64_t)h * D * 2));
        hi[u] = __ldcs(reinterpret_cast<const uint2*>(row + (int64_t)h * D * 2 + D));
      }
    }
  }
}

// -------------------------------------------------------------- tree masks

// One warp per sequence, one lane per drafted token: a token walks up its
// ancestors (parents precede their children, so the walk ends).  Up to 256
// tokens a sequence, read and written once: bound by the launch and the walk's
// dependent reads: 256 trees of 3 to 16 tokens take 4.1 us, one chain of 256 tokens
// 51 us.
template <int W>
__global__ void __launch_bounds__(kBlock) tree_mask_kernel(const TokensView t, const int32_t* parents, int64_t* masks,
                                                          int32_t* positions, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x * kBlockWarps + (threadIdx.x >> 5);
  if (b >= t.batch) return;
  const int lo = __ldg(t.cu + b), hi = __ldg(t.cu + b + 1), ctx = __ldg(t.ctx + b);
  const int n = hi - lo;
  if (lo < 0 || hi < lo || hi > t.n_tokens || ctx < 0 || ctx > INT_MAX - n) {
    if (lane == 0) status[b] = TC_ERR_BOUNDS;
    return;
  }
  bool ok = n <= 64 * W;
  for (int i = lane; i < n; i += 32) {
    const int par = __ldg(parents + lo + i);
    ok &= par >= -1 && par < i;
  }
  ok = __all_sync(0xffffffffu, ok);
  for (int i = lane; i < n; i += 32) {
    uint64_t m[W];
#pragma unroll
    for (int k = 0; k < W; ++k) m[k] = 0;
    int depth = -1;
    if (ok)
      for (int a = i; a >= 0; a = __ldg(parents + lo + a)) {
        ++depth;
#pragma unroll
        for (int k = 0; k < W; ++k) m[k] |= a >> 6 == k ? 1ull << (a & 63) : 0ull;
      }
#pragma unroll
    for (int k = 0; k < W; ++k) masks[(int64_t)(lo + i) * W + k] = (int64_t)m[k];
    if (positions) positions[lo + i] = ctx + (ok ? depth : 0);
  }
  if (lane == 0) status[b] = ok ? TC_OK : TC_ERR_BOUNDS;
}

// -------------------------------------------------------------- page copies

constexpr int kCopyUnroll = 8;

// A page of one layer is one run of bytes; a block copies kBlock * kCopyUnroll
// 16-byte words of it, every load before the first store.  Grid (blocks of a page
// x pairs, layers): the second and third axes end at 65,535.  Bound: bytes: 61
// pages of 64 slots, 8 heads of 128, in 16 layers take 77 us (6.6 TB/s, 98 % of
// a plain copy); 4 or 16 words a thread make no difference.
__global__ void __launch_bounds__(kBlock) copy_pages_kernel(uint8_t* pool, int32_t pages, int64_t page_bytes,
                                                           const int32_t* src, const int32_t* dst, int32_t* status,
                                                           int32_t keep, unsigned blocks) {
  const int pair = blockIdx.x / blocks, part = blockIdx.x % blocks, layer = blockIdx.y;
  const int a = __ldg(src + pair), b = __ldg(dst + pair);
  const bool ok = (uint32_t)a < (uint32_t)pages && (uint32_t)b < (uint32_t)pages;
  if (part == 0 && layer == 0 && threadIdx.x == 0) set_status(status, pair, ok ? TC_OK : TC_ERR_BOUNDS, keep);
  if (!ok) return;
  const uint4* from = reinterpret_cast<const uint4*>(pool + ((int64_t)layer * pages + a) * page_bytes);
  uint4* to = reinterpret_cast<uint4*>(pool + ((int64_t)layer * pages + b) * page_bytes);
  const int n = (int)(page_bytes / 16), at = part * kBlock * kCopyUnroll + threadIdx.x;
  uint4 v[kCopyUnroll];
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u)
    if (at + u * kBlock < n) v[u] = __ldcs(from + at + u * kBlock);
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u)
    if (at + u * kBlock < n) __stcs(to + at + u * kBlock, v[u]);
}

// --------------------------------------------------------------- compaction

struct CompactParams {
  uint8_t* pool;
  TokensView tok;
  int32_t layers, pages, kv_heads, page_size, page_shift;
  int32_t row_words;  // 16-byte words of one slot of one head
  const int32_t* path;
  int32_t path_width;
  const int32_t* n_path;
  int32_t* lens_out;
  int32_t* status;
  int32_t keep;
  uint32_t blocks;    // of a sequence
};

constexpr int kMoveUnroll = 4;

// Grid: for each sequence, blocks of kBlock columns.  A column is one 16-byte word of one head
// of one layer's keys or values; its thread moves that word of every slot of
// the branch, in ascending order.  Indices ascend strictly, so path[i] >= i:
// the slot that move i writes is the source of no later move, and an earlier
// move has read it before (same thread, program order).  Reading kMoveUnroll
// moves before writing them keeps that order.  Bound: the chain of path, page
// table, load and store: 64 branches of up to 12 tokens in 16 layers of 8 heads
// of 128 take 8.5 us (3.6 TB/s); two moves at a time 10.5, eight 9.4 (more
// registers, fewer blocks).
__global__ void __launch_bounds__(kBlock) compact_kernel(const CompactParams p) {
  __shared__ int64_t s_src[TC_PATH_MAX], s_dst[TC_PATH_MAX];  // slot offsets in rows of one head
  const int b = blockIdx.x / p.blocks, part = blockIdx.x % p.blocks, tid = threadIdx.x;
  const int ctx = __ldg(p.tok.ctx + b), n = __ldg(p.n_path + b);
  bool ok = ctx >= 0 && n >= 0 && n <= p.path_width;
  if (ok && tid < n) {
    const int32_t* path = p.path + (int64_t)b * p.path_width;
    const int x = __ldg(path + tid), before = tid > 0 ? __ldg(path + tid - 1) : -1;
    const int64_t frm = (int64_t)ctx + x, to = (int64_t)ctx + tid;
    ok = x > before && frm < (int64_t)p.tok.width * p.page_size && frm < kMaxSlots;
    if (ok && x >= tid) {
      const int32_t* row = p.tok.table + (int64_t)b * p.tok.width;
      const int pa = __ldg(row + (frm >> p.page_shift)), pb = __ldg(row + (to >> p.page_shift));
      ok = (uint32_t)pa < (uint32_t)p.pages && (uint32_t)pb < (uint32_t)p.pages;
      s_src[tid] = (int64_t)pa * 2 * p.kv_heads * p.page_size + (frm & (p.page_size - 1));
      s_dst[tid] = (int64_t)pb * 2 * p.kv_heads * p.page_size + (to & (p.page_size - 1));
    }
  }
  ok = __syncthreads_and(ok);
  if (part == 0 && tid == 0) {
    p.lens_out[b] = ok ? ctx + n : ctx;
    set_status(p.status, b, ok ? TC_OK : TC_ERR_BOUNDS, p.keep);
  }
  if (!ok) return;
  const int64_t col = (int64_t)part * kBlock + tid;
  const int word = (int)(col % p.row_words);
  const int64_t head = col / p.row_words;  // layer * 2 * kv_heads + (keys or values) * kv_heads + head
  if (head >= (int64_t)p.layers * 2 * p.kv_heads) return;
  const int64_t layer = head / (2 * p.kv_heads), in_layer = head % (2 * p.kv_heads);
  uint4* base = reinterpret_cast<uint4*>(p.pool) +
                ((layer * p.pages * 2 * p.kv_heads + in_layer) * p.page_size) * p.row_words + word;
  for (int i = 0; i < n; i += kMoveUnroll) {
    uint4 v[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (i + u < n && s_src[i + u] != s_dst[i + u]) v[u] = base[s_src[i + u] * p.row_words];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (i + u < n && s_src[i + u] != s_dst[i + u]) base[s_dst[i + u] * p.row_words] = v[u];
  }
}

template <typename T, int D>
cudaError_t launch_append(const AppendParams& p, int64_t warps, cudaStream_t s) {
  append_kernel<T, D, 4><<<(unsigned)((warps + kBlockWarps - 1) / kBlockWarps), kBlock, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace tcd

using namespace tcd;

extern "C" tc_status tc_kv_append(const tc_kv_t* kv, int32_t layer, const tc_tokens_t* tokens,
                                  const tc_append_t* a, int32_t* status, void* stream) {
  tc_status rc = kv_check("tc_kv_append", kv);
  if (rc == TC_OK) rc = kv_check_tokens("tc_kv_append", tokens, true);
  if (rc != TC_OK) return rc;
  if (!a || !status || layer < 0 || layer >= kv->layers || a->q_heads < 1 || !tokens->page_table ||
      tokens->table_width < 1)
    return kv_fail(TC_ERR_INVALID_ARG, "tc_kv_append: invalid arguments");
  const int64_t heads = (int64_t)a->q_heads + 2 * kv->kv_heads;
  if (tokens->n_tokens > 0 &&
      (!a->qkv || !a->q_out || kv_misaligned(a->qkv, 16) || kv_misaligned(a->q_out, 16) || a->qkv_stride % 8 != 0 ||
       a->q_out_stride % 8 != 0 || a->qkv_stride < heads * kv->head_dim ||
       a->q_out_stride < (int64_t)a->q_heads * kv->head_dim))
    return kv_fail(TC_ERR_INVALID_ARG,
                   "tc_kv_append: qkv and q_out must be 16-byte aligned, with row strides that are multiples of 8 "
                   "and hold a row");
  if (kv_misaligned(a->q_weight, 8) || kv_misaligned(a->k_weight, 8) || kv_misaligned(a->rope, 16) ||
      (a->rope && a->rope_len < 1))
    return kv_fail(TC_ERR_INVALID_ARG, "tc_kv_append: weights must be 8-byte, the angles 16-byte aligned");
  if (heads > 65535) return kv_fail(TC_ERR_CAPACITY, "tc_kv_append: more than 65535 heads");
  KvDevice dev(kv->device);
  if (!dev.ok) return kv_fail(TC_ERR_CUDA, "tc_kv_append: cannot use the cache's device");
  AppendParams p;
  p.kv = kv_view(kv, layer);
  p.tok = tokens_view(tokens);
  p.qkv = static_cast<const uint8_t*>(a->qkv);
  p.qkv_stride = a->qkv_stride;
  p.q_heads = a->q_heads;
  p.q_weight = static_cast<const uint8_t*>(a->q_weight);
  p.k_weight = static_cast<const uint8_t*>(a->k_weight);
  p.eps = a->eps;
  p.rope = a->rope;
  p.rope_len = a->rope_len;
  p.positions = a->positions;
  p.interleaved = a->interleaved != 0;
  p.q_out = static_cast<uint8_t*>(a->q_out);
  p.q_out_stride = a->q_out_stride;
  p.status = status;
  // Few tokens: their heads are spread over more warps, down to one round of
  // one load per lane (a whole token in one warp takes its rounds one after
  // another); more than 4096 warps of them cost more than they hide.  1, 512,
  // 2048 and 4096 tokens: 4.3, 6.5, 14.6 and 24.8 us; always a warp per token
  // 7.4, 14.6, 18.7, 24.8; always a round per warp 4.3, 10.5, 28.9, 56.7.
  const int hpw = 256 / kv->head_dim;
  const int64_t rounds = (heads + hpw - 1) / hpw;
  int64_t split = 1;
  while (split < rounds && (int64_t)tokens->n_tokens * split < 4096) split *= 2;
  p.split = (int32_t)(split < rounds ? split : rounds);
  const int64_t warps = (int64_t)tokens->n_tokens * p.split + tokens->batch;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (kv->dtype == TC_DT_BF16)
    e = kv->head_dim == 128 ? launch_append<Bf16, 128>(p, warps, s) : launch_append<Bf16, 64>(p, warps, s);
  else
    e = kv->head_dim == 128 ? launch_append<F16, 128>(p, warps, s) : launch_append<F16, 64>(p, warps, s);
  return e == cudaSuccess ? TC_OK : kv_cuda_fail(e, "tc_kv_append: ");
}

extern "C" tc_status tc_tree_masks(const tc_tokens_t* tokens, const int32_t* parents, int32_t words, int64_t* masks,
                                   int32_t* positions, int32_t* status, void* stream) {
  const tc_status rc = kv_check_tokens("tc_tree_masks", tokens, true);
  if (rc != TC_OK) return rc;
  if (!status || words < 1 || words > TC_TREE_MAX_WORDS || (tokens->n_tokens > 0 && (!parents || !masks)))
    return kv_fail(TC_ERR_INVALID_ARG, "tc_tree_masks: invalid arguments");
  const TokensView t = tokens_view(tokens);
  const unsigned grid = (unsigned)((tokens->batch + kBlockWarps - 1) / kBlockWarps);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (words == 1) tree_mask_kernel<1><<<grid, kBlock, 0, s>>>(t, parents, masks, positions, status);
  if (words == 2) tree_mask_kernel<2><<<grid, kBlock, 0, s>>>(t, parents, masks, positions, status);
  if (words == 3) tree_mask_kernel<3><<<grid, kBlock, 0, s>>>(t, parents, masks, positions, status);
  if (words == 4) tree_mask_kernel<4><<<grid, kBlock, 0, s>>>(t, parents, masks, positions, status);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TC_OK : kv_cuda_fail(e, "tc_tree_masks: ");
}

extern "C" tc_status tc_kv_copy_pages(const tc_kv_t* kv, const int32_t* src, const int32_t* dst, int32_t n,
                                      int32_t* status, void* stream) {
  const tc_status rc = kv_check("tc_kv_copy_pages", kv);
  if (rc != TC_OK) return rc;
  if (n < 0 || (n > 0 && (!src || !dst || !status)))
    return kv_fail(TC_ERR_INVALID_ARG, "tc_kv_copy_pages: invalid arguments");
  if (n > TC_KV_MAX_BATCH || kv->layers > 65535)
    return kv_fail(TC_ERR_CAPACITY, "tc_kv_copy_pages: more than 65536 pairs or 65535 layers");
  if (n == 0) return TC_OK;
  const int64_t page_bytes = (int64_t)4 * kv->kv_heads * kv->page_size * kv->head_dim;
  const int64_t per_block = (int64_t)kBlock * kCopyUnroll * 16;
  const int64_t blocks = (page_bytes + per_block - 1) / per_block;
  if (blocks * n > INT_MAX) return kv_fail(TC_ERR_CAPACITY, "tc_kv_copy_pages: pairs x page size is too large");
  KvDevice dev(kv->device);
  if (!dev.ok) return kv_fail(TC_ERR_CUDA, "tc_kv_copy_pages: cannot use the cache's device");
  const dim3 grid((unsigned)(blocks * n), (unsigned)kv->layers);
  copy_pages_kernel<<<grid, kBlock, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<uint8_t*>(kv->pool), kv->pages,
                                                                           page_bytes, src, dst, status,
                                                                           kv->keep_status != 0, (unsigned)blocks);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TC_OK : kv_cuda_fail(e, "tc_kv_copy_pages: ");
}

extern "C" tc_status tc_kv_compact(const tc_kv_t* kv, const tc_tokens_t* tokens, const int32_t* path,
                                   int32_t path_width, const int32_t* n_path, int32_t* lens_out, int32_t* status,
                                   void* stream) {
  tc_status rc = kv_check("tc_kv_compact", kv);
  if (rc == TC_OK) rc = kv_check_tokens("tc_kv_compact", tokens, false);
  if (rc != TC_OK) return rc;
  if (!path || !n_path || !lens_out || !status || !tokens->page_table || tokens->table_width < 1 || path_width < 1)
    return kv_fail(TC_ERR_INVALID_ARG, "tc_kv_compact: invalid arguments");
  if (path_width > TC_PATH_MAX)
    return kv_fail(TC_ERR_CAPACITY, "tc_kv_compact: path_width is more than 256");
  if (lens_out < tokens->ctx_lens + tokens->batch && tokens->ctx_lens < lens_out + tokens->batch)
    return kv_fail(TC_ERR_INVALID_ARG, "tc_kv_compact: lens_out overlaps ctx_lens");
  const int64_t cols = (int64_t)kv->layers * 2 * kv->kv_heads * (kv->head_dim / 8);
  const int64_t blocks = (cols + kBlock - 1) / kBlock;
  if (blocks * tokens->batch > INT_MAX)
    return kv_fail(TC_ERR_CAPACITY, "tc_kv_compact: sequences x layers x kv_heads is too large");
  KvDevice dev(kv->device);
  if (!dev.ok) return kv_fail(TC_ERR_CUDA, "tc_kv_compact: cannot use the cache's device");
  CompactParams p;
  const KvView v = kv_view(kv, 0);
  p.pool = v.base;
  p.tok = tokens_view(tokens);
  p.layers = kv->layers;
  p.pages = kv->pages;
  p.kv_heads = kv->kv_heads;
  p.page_size = v.page_size;
  p.page_shift = v.page_shift;
  p.row_words = kv->head_dim / 8;
  p.path = path;
  p.path_width = path_width;
  p.n_path = n_path;
  p.lens_out = lens_out;
  p.status = status;
  p.keep = v.keep;
  p.blocks = (uint32_t)blocks;
  compact_kernel<<<(unsigned)(blocks * tokens->batch), kBlock, 0, static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TC_OK : kv_cuda_fail(e, "tc_kv_compact: ");
}
