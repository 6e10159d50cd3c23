// Attention of a call's tokens (a prompt, a drafted tree, single tokens) over
// the paged cache.
#include <climits>

#include "kv_cache.h"

namespace tcd {
namespace {

struct AttendParams {
  KvView kv;
  TokensView tok;
  const uint8_t* q;
  int64_t q_stride;
  int32_t q_heads;
  int32_t max_tokens;
  float scale_log2;
  const int64_t* tree;
  int32_t words;
  uint8_t* out;
  int64_t out_stride;
  float* lse;
  int32_t* status;
};

// One warp per token and query head: one pass over the slots with the running
// maximum and sum of the softmax, the row's elements spread over the lanes.
template <typename T, int D>
__global__ void __launch_bounds__(256) attend_rows_kernel(const AttendParams p) {
  constexpr int E = D / 64;  // 32-bit words (two elements) per lane
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t n_work = (int64_t)p.tok.n_tokens * p.q_heads;
  if (w >= n_work) {
    const int64_t b = w - n_work;
    if (b >= p.tok.batch) return;
    SeqSpan s;
    bool ok = seq_span(p.tok, p.kv.page_size, (int)b, &s) && s.n <= p.max_tokens;
    if (ok && s.n > 0)
      for (int i = lane; i <= (s.ctx + s.n - 1) >> p.kv.page_shift; i += 32)
        ok &= (uint32_t)__ldg(p.tok.table + b * p.tok.width + i) < (uint32_t)p.kv.pages;
    ok = __all_sync(0xffffffffu, ok);
    if (lane == 0) p.status[b] = ok ? TC_OK : TC_ERR_BOUNDS;
    return;
  }
  const int i = (int)(w / p.q_heads), h = (int)(w % p.q_heads);
  int lo = 0, hi = p.tok.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__ldg(p.tok.cu + mid) <= i) lo = mid; else hi = mid;
  }
  SeqSpan s;
  if (!seq_span(p.tok, p.kv.page_size, lo, &s) || s.n > p.max_tokens || i < s.row0 || i >= s.row0 + s.n) return;
  const int t = i - s.row0, g = h / (p.q_heads / p.kv.kv_heads);
  const int64_t head_words = (int64_t)p.kv.page_size * (D / 2);
  const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q) + ((int64_t)i * p.q_stride + (int64_t)h * D) / 2;
  float2 qf[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qf[e] = T::unpack(__ldg(q + e * 32 + lane));
    o[e] = make_float2(0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  const int last = p.tree ? s.ctx + s.n : s.ctx + t + 1;
  for (int j = 0; j < last; ++j) {
    const int x = j - s.ctx;
    if (x >= 0 && p.tree && ((x >> 6) >= p.words || !((p.tree[(int64_t)i * p.words + (x >> 6)] >> (x & 63)) & 1)))
      continue;
    const int page = __ldg(p.tok.table + (int64_t)lo * p.tok.width + (j >> p.kv.page_shift));
    if ((uint32_t)page >= (uint32_t)p.kv.pages) continue;
    const uint32_t* k = reinterpret_cast<const uint32_t*>(p.kv.base) +
                        ((int64_t)page * 2 * p.kv.kv_heads + g) * head_words +
                        (int64_t)(j & (p.kv.page_size - 1)) * (D / 2);
    float dot = 0.f;
    float2 v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float2 kf = T::unpack(__ldg(k + e * 32 + lane));
      v[e] = T::unpack(__ldg(k + p.kv.kv_heads * head_words + e * 32 + lane));
      dot = fmaf(qf[e].x, kf.x, fmaf(qf[e].y, kf.y, dot));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    dot *= p.scale_log2;
    const float m2 = fmaxf(m, dot), ref = m2 == -INFINITY ? 0.f : m2;
    const float a = exp2f(m - ref), w2 = exp2f(dot - ref);
    l = l * a + w2;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e].x = fmaf(w2, v[e].x, o[e].x * a);
      o[e].y = fmaf(w2, v[e].y, o[e].y * a);
    }
    m = m2;
  }
  const float r = l == 0.f ? 0.f : 1.f / l;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out) + ((int64_t)i * p.out_stride + (int64_t)h * D) / 2;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e * 32 + lane] = T::pack(o[e].x * r, o[e].y * r);
  if (p.lse && lane == 0)
    p.lse[(int64_t)i * p.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace
}  // namespace tcd

using namespace tcd;

extern "C" tc_status tc_attend_workspace(const tc_kv_t* kv, int64_t* bytes) {
  const tc_status rc = kv_check("tc_attend_workspace", kv);
  if (rc != TC_OK) return rc;
  if (!bytes) return kv_fail(TC_ERR_INVALID_ARG, "tc_attend_workspace: bytes is NULL");
  *bytes = 16;
  return TC_OK;
}

extern "C" tc_status tc_attend(const tc_kv_t* kv, int32_t layer, const tc_tokens_t* tokens, const tc_attend_t* a,
                               void* workspace, int64_t workspace_bytes, int32_t* status, void* stream) {
  tc_status rc = kv_check("tc_attend", kv);
  if (rc == TC_OK) rc = kv_check_tokens("tc_attend", tokens, true);
  if (rc != TC_OK) return rc;
  if (!a || !status || layer < 0 || layer >= kv->layers || a->q_heads < 1 || a->max_tokens < 0 ||
      !tokens->page_table || tokens->table_width < 1 || !(a->scale == a->scale))
    return kv_fail(TC_ERR_INVALID_ARG, "tc_attend: invalid arguments");
  if (a->q_heads % kv->kv_heads != 0 || a->q_heads / kv->kv_heads > 128)
    return kv_fail(TC_ERR_UNSUPPORTED,
                   "tc_attend: q_heads must be a multiple of kv_heads, with at most 128 of them for each");
  if (a->tree && (a->tree_words < 1 || a->tree_words > TC_TREE_MAX_WORDS || a->max_tokens > 64 * a->tree_words))
    return kv_fail(TC_ERR_CAPACITY, "tc_attend: a tree wants 1 to 4 words and at most 64 tokens a word");
  int64_t need = 0;
  rc = tc_attend_workspace(kv, &need);
  if (rc != TC_OK) return rc;
  if (!workspace || kv_misaligned(workspace, 16) || workspace_bytes < need)
    return kv_fail(TC_ERR_CAPACITY, "tc_attend: the workspace is too small or not 16-byte aligned");
  const int64_t row = (int64_t)a->q_heads * kv->head_dim;
  if (tokens->n_tokens > 0 &&
      (!a->q || !a->out || kv_misaligned(a->q, 16) || kv_misaligned(a->out, 16) || a->q_stride % 8 != 0 ||
       a->out_stride % 8 != 0 || a->q_stride < row || a->out_stride < row))
    return kv_fail(TC_ERR_INVALID_ARG,
                   "tc_attend: q and out must be 16-byte aligned, with row strides that are multiples of 8 and hold "
                   "a row");
  KvDevice dev(kv->device);
  if (!dev.ok) return kv_fail(TC_ERR_CUDA, "tc_attend: cannot use the cache's device");
  AttendParams p;
  p.kv = kv_view(kv, layer);
  p.tok = tokens_view(tokens);
  p.q = static_cast<const uint8_t*>(a->q);
  p.q_stride = a->q_stride;
  p.q_heads = a->q_heads;
  p.max_tokens = a->max_tokens;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.tree = a->tree;
  p.words = a->tree ? a->tree_words : 0;
  p.out = static_cast<uint8_t*>(a->out);
  p.out_stride = a->out_stride;
  p.lse = a->lse;
  p.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)(((int64_t)tokens->n_tokens * a->q_heads + tokens->batch + 7) / 8);
  if (kv->dtype == TC_DT_BF16) {
    if (kv->head_dim == 128) attend_rows_kernel<Bf16, 128><<<grid, 256, 0, s>>>(p);
    else attend_rows_kernel<Bf16, 64><<<grid, 256, 0, s>>>(p);
  } else {
    if (kv->head_dim == 128) attend_rows_kernel<F16, 128><<<grid, 256, 0, s>>>(p);
    else attend_rows_kernel<F16, 64><<<grid, 256, 0, s>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TC_OK : kv_cuda_fail(e, "tc_attend");
}
