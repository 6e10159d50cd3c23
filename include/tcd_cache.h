/*
 * tcd_cache.h - C ABI of the paged key-value cache and of the attention that
 * reads it: what a model's attention layers do in front of the constrained
 * decode step of tcd.h.
 *
 * A decoder of catalog pointers reads a prompt (tc_kv_append, tc_attend with
 * the causal mask), then emits tokens one by one or verifies drafted branches
 * of the catalog's trie ("Understanding Inference for Systems Engineers",
 * section 7.5: forced spans are ingested by one forward pass): the drafts are
 * appended behind the cached tokens, attended under their tree's mask
 * (tc_tree_masks, tc_attend), the constrained step picks the branch, and
 * tc_kv_compact moves the accepted branch together.  tc_pages keeps the pages:
 * growing, forking (pages shared until written), trimming and freeing.
 *
 * Conventions are tcd.h's: the caller owns every buffer, calls that take a
 * stream are asynchronous and capturable, argument errors are returned at once
 * and launch nothing, errors found on the device are recorded per sequence.
 * Calls are stateless (no handle holds anything between calls) and may be
 * made from several threads and streams as long as they write different
 * memory; a workspace belongs to one call at a time.  A captured call keeps the
 * addresses it was given: graphs that may run at the same time, or beside calls
 * on a stream, need workspaces of their own, for as long as they exist
 * (tc_capture_id and tc_capture_watch tell a caller when).
 */
#ifndef TCD_CACHE_H
#define TCD_CACHE_H

#include "tcd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of a cache, and of the queries, keys, values and outputs of its calls. */
enum {
  TC_DT_BF16 = 0,
  TC_DT_F16 = 1
};

/*
 * A paged cache.
 *
 *  pool       (device) [layers][pages][2][kv_heads][page_size][head_dim]
 *             (index 0 of the third axis: keys, 1: values), 16-byte aligned.
 *  dtype      TC_DT_BF16 or TC_DT_F16.
 *  page_size  16, 32, 64 or 128 tokens.      head_dim  64 or 128.
 *  device     the CUDA device the pool lies on; calls run there.
 *  keep_status  0: a call writes its whole status array.  1: it writes the
 *             code of a sequence (or pair) only if that is an error and the
 *             array has TC_OK there, so that one array, which the caller has
 *             set to TC_OK, gathers the first errors of many calls.
 *
 * Token i of a sequence lies in slot i % page_size of the page that entry
 * i / page_size of the sequence's page table names, in every layer.
 */
typedef struct tc_kv_t {
  void* pool;
  int32_t device;
  int32_t dtype;
  int32_t layers;
  int32_t pages;
  int32_t kv_heads;
  int32_t page_size;
  int32_t head_dim;
  int32_t keep_status;
} tc_kv_t;

/*
 * The tokens of one call: packed sequences of different lengths, each behind
 * what its pages already hold.
 *
 *  batch        sequences (1 .. TC_KV_MAX_BATCH).
 *  n_tokens     rows of the packed token arrays (>= 0; 0 only does the status).
 *  cu_tokens    (device) int32[batch + 1], ascending: sequence b's tokens are
 *               rows [cu_tokens[b], cu_tokens[b + 1]); none is allowed.  (Where
 *               it descends, that sequence gets TC_ERR_BOUNDS; a row that other
 *               sequences then have in common belongs to any one of them.)
 *  ctx_lens     (device) int32[batch]: tokens of sequence b already cached.
 *               Its new token t lies in slot ctx_lens[b] + t.
 *  page_table   (device) int32[batch][table_width] page ids; entries past a
 *               sequence's last page are not read.  A sequence has at most
 *               table_width * page_size slots, and fewer than 2^31 - 2^16.
 *
 * A sequence whose rows, lengths, slots or page ids are out of range gets
 * TC_ERR_BOUNDS in the call's status.  Nothing outside the given buffers and
 * the pool is touched for it, and what the call writes for it is invalid.
 */
typedef struct tc_tokens_t {
  int32_t batch;
  int32_t n_tokens;
  const int32_t* cu_tokens;
  const int32_t* ctx_lens;
  const int32_t* page_table;
  int32_t table_width;
} tc_tokens_t;

#define TC_KV_MAX_BATCH 65536

/*
 * tc_kv_append - norms of queries and keys for each head, rotation by
 * position, and the write of keys and values into the cache, in one pass over
 * the packed output of the query-key-value projection.
 *
 * For each token and each query or key head, x of head_dim elements:
 *   y = x * rsqrt(mean(x^2) + eps) * weight     (skipped where the weight is NULL)
 *   (a, b) -> (a cos - b sin, b cos + a sin)    for each of head_dim / 2 pairs
 * in 32 bits, rounded once to the cache's type.  Pair i is elements
 * (i, i + head_dim / 2), or (2 i, 2 i + 1) with `interleaved`.  Values are
 * copied.
 *
 *  qkv        (device) [n_tokens] rows of (q_heads + 2 kv_heads) * head_dim
 *             elements: query heads, key heads, value heads; rows qkv_stride
 *             elements apart (a multiple of 8), 16-byte aligned.
 *  q_weight   (device) [head_dim] of the cache's type, or NULL; 8-byte aligned.
 *  k_weight   the same for keys.
 *  rope       (device) float[rope_len][head_dim / 2][2], cosine and sine of
 *             each position's angles, 16-byte aligned; NULL: no rotation.
 *  positions  (device) int32[n_tokens], rows of `rope`; NULL: the token's slot.
 *             A token at a position outside [0, rope_len) is not written, and
 *             its sequence gets TC_ERR_BOUNDS.
 *  q_out      (device) [n_tokens][q_heads][head_dim], rows q_out_stride
 *             elements apart (a multiple of 8), 16-byte aligned.
 *  status     (device) int32[batch]: TC_OK or TC_ERR_BOUNDS for each sequence.
 *
 * Pages written must belong to one sequence of the call only.
 */
typedef struct tc_append_t {
  const void* qkv;
  int64_t qkv_stride;
  int32_t q_heads;
  const void* q_weight;
  const void* k_weight;
  float eps;
  const float* rope;
  int32_t rope_len;
  const int32_t* positions;
  int32_t interleaved;
  void* q_out;
  int64_t q_out_stride;
} tc_append_t;

tc_status tc_kv_append(const tc_kv_t* kv, int32_t layer, const tc_tokens_t* tokens,
                       const tc_append_t* args, int32_t* status, void* stream);

/*
 * tc_attend - attention of the call's tokens over the cache.
 *
 * out[i, h] = sum_j softmax_j(scale * q[i, h] . k[j, g]) v[j, g],
 * g = h / (q_heads / kv_heads), over the slots j that token i of sequence b
 * (index t within the sequence) sees:
 *   every cached slot        j < ctx_lens[b], and
 *   with tree == NULL        j <= ctx_lens[b] + t (causal: a prompt or a chunk
 *                            of one; one token is a plain decode step);
 *   with tree                slot ctx_lens[b] + s where bit s % 64 of
 *                            tree[i][s / 64] is set (bits past the sequence's
 *                            tokens are ignored).
 * The call's own keys and values have to be in the cache (tc_kv_append).
 * A slot that a token does not see contributes nothing, whatever it holds
 * (infinities and NaN included).  A token that sees nothing gets zeros.
 * Scores, maxima, sums and outputs are held in 32 bits; the weights of one
 * tile are rounded to the cache's type for the tensor cores (f16:
 * as far as 2^-21 of the row's largest weight, smaller ones to multiples of 2^-31
 * of it).
 *
 *  q           (device) [n_tokens][q_heads][head_dim] of the cache's type,
 *              rows q_stride elements apart (a multiple of 8), 16-byte aligned.
 *              q_heads is a multiple of kv_heads, at most 128 of them share one.
 *  max_tokens  at least the tokens of the longest sequence in this call
 *              (a longer one gets TC_ERR_BOUNDS).
 *  tree        (device) int64[n_tokens][tree_words] or NULL; with it
 *              max_tokens <= 64 * tree_words, tree_words <= TC_TREE_MAX_WORDS.
 *  out         (device) like q, rows out_stride elements apart.
 *  lse         (device) float[n_tokens][q_heads] or NULL: the logarithm of the
 *              sum of exp(scale * q . k) over the slots seen (-inf for none).
 *  workspace   (device) tc_attend_workspace bytes (about 40 MB: two partial
 *              results per SM), 16-byte aligned; its content before and after the
 *              call means nothing.
 *  status      (device) int32[batch]: TC_OK, TC_ERR_BOUNDS, or
 *              TC_ERR_DEVICE_TIMEOUT for every sequence if a bounded wait of
 *              the kernel gave up (the outputs are then invalid).
 */
#define TC_TREE_MAX_WORDS 4

typedef struct tc_attend_t {
  const void* q;
  int64_t q_stride;
  int32_t q_heads;
  int32_t max_tokens;
  float scale;
  const int64_t* tree;
  int32_t tree_words;
  void* out;
  int64_t out_stride;
  float* lse;
  int64_t wait_polls;  /* polls of one wait inside the kernel before it gives up; 0: the default (seconds) */
  int32_t withhold;    /* 0; tests: the kernel leaves out its first load, so that its waits run out */
} tc_attend_t;

tc_status tc_attend(const tc_kv_t* kv, int32_t layer, const tc_tokens_t* tokens, const tc_attend_t* args,
                    void* workspace, int64_t workspace_bytes, int32_t* status, void* stream);

/* tc_attend_workspace - bytes of workspace tc_attend needs with this cache, whatever its tokens. */
tc_status tc_attend_workspace(const tc_kv_t* kv, int64_t* bytes);

/*
 * tc_tree_masks - the masks and positions of drafted trees from their parents.
 *
 *  parents    (device) int32[n_tokens]: a drafted token's parent as its index
 *             within the sequence, smaller than the token's own; -1 for a token
 *             that follows the cached tokens directly.
 *  masks      (device) int64[n_tokens][words]: bit s of a token's words is set
 *             for each of its ancestors s and for itself.
 *  positions  (device) int32[n_tokens] or NULL: ctx_lens[b] + number of ancestors.
 *  words      1 .. TC_TREE_MAX_WORDS.
 *  status     (device) int32[batch]: TC_ERR_BOUNDS for a sequence with a parent
 *             out of range or with more than 64 * words tokens (its masks are
 *             zero).
 *
 * Reads cu_tokens and ctx_lens of `tokens` only; runs on the current device.
 */
tc_status tc_tree_masks(const tc_tokens_t* tokens, const int32_t* parents, int32_t words, int64_t* masks,
                        int32_t* positions, int32_t* status, void* stream);

/*
 * tc_kv_copy_pages - copy whole pages, in every layer: page dst[i] becomes
 * page src[i].  src and dst (device) int32[n], n <= TC_KV_MAX_BATCH; no page may
 * be written twice, nor be both read and written by one call.  status (device)
 * int32[n]: TC_ERR_BOUNDS for a pair with a page id out of range (not copied).
 */
tc_status tc_kv_copy_pages(const tc_kv_t* kv, const int32_t* src, const int32_t* dst, int32_t n, int32_t* status,
                           void* stream);

/*
 * tc_kv_compact - move the accepted branch of each sequence's drafted tokens
 * together, in every layer: slot ctx_lens[b] + i becomes what slot
 * ctx_lens[b] + path[b][i] held, for i < n_path[b].
 *
 *  path       (device) int32[batch][path_width], strictly ascending indices of
 *             drafted tokens (a branch in topological order); path_width <=
 *             TC_PATH_MAX.
 *  n_path     (device) int32[batch], 0 .. path_width.
 *  lens_out   (device) int32[batch]: ctx_lens[b] + n_path[b]; must not overlap
 *             ctx_lens.
 *  status     (device) int32[batch]: TC_ERR_BOUNDS for a path that does not
 *             ascend, or slots or page ids out of range (nothing of that
 *             sequence moves and lens_out[b] = ctx_lens[b]).
 *
 * n_tokens and cu_tokens of `tokens` are not read (cu_tokens may be NULL).
 */
#define TC_PATH_MAX 256

tc_status tc_kv_compact(const tc_kv_t* kv, const tc_tokens_t* tokens, const int32_t* path, int32_t path_width,
                        const int32_t* n_path, int32_t* lens_out, int32_t* status, void* stream);

/*
 * tc_pages - which pages of a cache belong to which sequence (host object;
 * needs no GPU).  Pages are counted by their holders: a fork shares the full
 * pages of its parent, and a page that is shared is copied before it is
 * written.  Free pages are handed out lowest id first.
 *
 * Calls that need pages fail with TC_ERR_CAPACITY when there are not enough
 * and then change nothing.  Copies that a call asks for are appended to
 * src / dst (host; a call never asks for more than one pair).  Run them with
 * tc_kv_copy_pages before anything is written to any sequence (another holder of
 * the source page may be its only one by now, and write to it without a copy) and
 * before a sequence is closed or trimmed (a source page may become free, and be
 * handed out again as another copy's target).
 * One host thread at a time per object.
 */
typedef struct tc_pages tc_pages;

tc_status tc_pages_create(int32_t pages, int32_t page_size, tc_pages** out);
void tc_pages_destroy(tc_pages* p);

/* A new, empty sequence: *seq receives its id (ids of closed sequences are used again, lowest first). */
tc_status tc_pages_open(tc_pages* p, int32_t* seq);

/* Drop a sequence; pages without another holder become free. */
tc_status tc_pages_close(tc_pages* p, int32_t seq);

/*
 * Make room to write slots [from, upto) of a sequence: pages are added, and if
 * the page of slot `from` is shared and holds earlier slots, it is replaced by
 * a copy (one pair, *n_copies = 1, else 0); shared pages further on are
 * replaced by fresh ones without a copy: slots from `from` on count as given up,
 * what a shared page held there, behind `upto` as well, is the sequence's no more.
 */
tc_status tc_pages_reserve(tc_pages* p, int32_t seq, int64_t from, int64_t upto, int32_t* src, int32_t* dst,
                           int32_t* n_copies);

/*
 * Fork the first `len` tokens of a sequence: *child receives a new sequence
 * that shares their pages (all of them; the first write into the last, partly
 * filled one makes tc_pages_reserve ask for a copy).
 */
tc_status tc_pages_fork(tc_pages* p, int32_t seq, int64_t len, int32_t* child);

/* Free the pages of a sequence past its first `len` tokens. */
tc_status tc_pages_trim(tc_pages* p, int32_t seq, int64_t len);

/* Page ids of a sequence into row[width] (host); the rest of the row is set to -1.  *n receives their number. */
tc_status tc_pages_row(const tc_pages* p, int32_t seq, int32_t* row, int32_t width, int32_t* n);

/* Pages that nobody holds. */
tc_status tc_pages_free_count(const tc_pages* p, int32_t* n);

/*
 * For callers that manage the buffers of captured calls.
 *
 * tc_capture_id - *id receives a number that names the capture a stream is part
 * of (another for each capture of the process), 0 if it is being captured into no
 * graph.
 *
 * tc_capture_watch - *gone receives a host word that is 0 and becomes 1 when the
 * graph that `stream` is being captured into, all graphs made from it and their
 * last launch have ended: buffers given to its calls may be freed then.
 * TC_ERR_INVALID_ARG if the stream is not being captured.
 *
 * tc_capture_unwatch - frees such a word, once it is 1.
 *
 * tc_capture_mode - swaps the calling thread's capture mode with *mode (0 global,
 * 1 thread, 2 relaxed: memory for the buffers may be allocated during a capture).
 *
 * tc_clear_now - sets device memory to zero by way of `stream`, which must not be
 * part of a capture, and waits for it; allowed while other streams are captured.
 */
tc_status tc_capture_id(void* stream, uint64_t* id);
tc_status tc_capture_watch(void* stream, int32_t** gone);
void tc_capture_unwatch(int32_t* gone);
tc_status tc_capture_mode(int32_t* mode);
tc_status tc_clear_now(void* ptr, int64_t bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TCD_CACHE_H */
