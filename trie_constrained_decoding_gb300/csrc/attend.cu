// Attention of a call's tokens (a prompt, a drafted tree, single tokens) over
// the paged cache, on the tensor cores.
//
// Rows.  The queries of all heads that share a key-value head see the same
// keys, so they are rows of one product: row r of an M tile is token r / G,
// query head r % G of the group (G = q_heads / kv_heads), 128 / G whole tokens
// a tile.  A single token of a decode step is a tile of G rows; a drafted tree
// or a prompt fills tiles of 128.
//
// Work.  An item is one sequence, one key-value head and up to two M tiles;
// its units are 128-slot tiles of the cache, one or two more before them and
// two after them for what its beginning (first loads, first product) and its
// end (last product, output) take.  The units of all items form one line that is
// cut into equal parts, one per CTA (one CTA per SM), whatever the mixture of
// lengths: a long context is split over many CTAs, many short ones share one, and
// a cut that falls into an item's beginning or end splits nothing.  (Against
// tiles alone: a prompt of 8192 416 us, was 488; 16 short prompts 45.5, was 53; a
// decode step of 64 sequences 180, was 192.  With three units before and none
// after four prompts of 2048 take 156 us instead of 148, with two and two 151.)
// Every CTA works its part out from the lengths on the device, so the launch
// depends on none of them and can be captured.  An item that a cut falls into leaves
// unnormalised partial results in 32 bits, at most two per CTA, which a second
// kernel joins.
//
// One CTA, 16 warps:
//  - warps 0, 5 and 7 load keys, values and queries by TMA (128-byte swizzle),
//    keys and values in turn into one ring of 128 x head_dim tiles, a copy per
//    page and 64 columns; pages past the sequence's end are not loaded.  One
//    warp for all three sets the pace where pages have 16 slots (drafts of 16
//    sequences: 85 us against 80), and makes no difference for larger ones;
//  - warps 1 and 3 issue the score products S = Q K^T of one softmax group each
//    (both operands in shared memory), warps 4 and 6 the output products
//    O += P V (P in tensor memory), in steps of 64 slots (head_dim 128) or 128
//    (64).  One thread each, which does nothing but wait for its operands and
//    issue: one that has both products of a group to look at reacts too late
//    (a prompt of 8192 took 696 us so when it took 512 with two);
//  - warp 2 hands out the CTA's segments (an item's part) through a small ring;
//  - warps 8-11 and 12-15 are two softmax groups, one row per thread: a thread
//    reads its row of S from tensor memory, keeps the row's maximum and sum in
//    32 bits, and writes the weights P beside it in the cache's type, which is
//    what the tensor cores multiply.  The sum is of the weights before that
//    rounding: the rounding's errors have a common sign only where weights
//    coincide, and are then at most half a unit of the type.
// The two groups always alternate with the tensor cores: with two M tiles each
// takes one and both use every key-value tile; with one M tile they take the
// even and the odd tiles of the cache and are joined at the end.
//
// Tensor memory, 512 columns of 32 bits: each group has its scores S, its
// weights P and its accumulator O, 64 + 2 x 32 + 128 columns (head_dim 128) or
// 128 + 64 + 64 (64).  S and P are apart, so that the next step's scores are
// computed while the group works on this one's weights, and at head_dim 128 P
// has two places, so that the next weights need not wait for the product of
// the last (the issuer of the scores waits for the one before that, while its own
// product runs, and announces both: the group waits once a step, 418 us against
// 436 for a prompt of 8192).  Steps of 128 slots there would leave room for S and
// P in one place only, and a step would be one chain of products and softmax.  The
// scores of a step of 64 read 6 KB of shared memory for 32 cycles of products and take 50;
// beside the other product, which reads less, a step of 128 slots takes 576
// cycles instead of 512 (measured).
//
// The maximum that the weights refer to is only moved when a row's maximum
// has grown by more than 2^8: the accumulator in tensor memory is rescaled then
// and rarely otherwise.  bf16 and the sums in 32 bits hold such weights as well as
// smaller ones.  f16 has few exponents: below 2^-14 a weight would lose bits, below
// 2^-25 it would vanish from the products but not from the sum, always to one side
// (131,072 slots of 2^-25 of the largest weight hold 0.4 % of a row).  So its weights,
// and with them sum and accumulator, carry a factor of 2^7, the most that stays
// under f16's largest number with the 2^8: what a slot may lose is 2^-32 of the
// largest weight, below the output's rounding up to 2^20 slots.  (Moving the maximum
// sooner leaves room for a larger factor but costs time: 2^6 and 2^9 357 us for
// prompt chunks of head_dim 64, 2^4 and 2^11 375, these 353, as without a factor.)
//
// Steps that every row sees entirely run in a loop without masks.  The others
// (the end of the sequence, the drafted tokens, the diagonal of a prompt) take
// the masked path: a mask of the step's slots per row; and, as a weight of zero
// times an infinity would be NaN, infinities and NaN among the values of slots
// that only some rows see are taken out of the tile and added at the end to the
// rows that see them.
//
// What it measured (bf16, 32 query and 8 key-value heads of 128, pages of 64):
// a prompt of 8192 tokens in 439 us back to back, 1.25 PFLOP/s, 65 % of what the
// library's matrix product reaches (417 us in short runs, 68 %); 16 prompts of 5 to
// 261 tokens in 45 us; a decode step of 64 sequences with 97 to 8011 slots in 179 us,
// 6.1 TB/s, 90 % of a copy's rate; one token over 1500 slots in 16.3 us; one token of
// 253 sequences with 20 to 81 slots and 16 heads of their own in 166 us.  Bound: long
// prompts by the chain of waits and exponentials that a softmax group goes through
// in a step (0.96 us for both groups' 64 slots, of which the products take 0.53);
// decode by bytes; small calls and many short items by latencies one after another
// and the fetch of instructions, as each part of the code runs once an item (6 us
// for an item of one tile).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <climits>
#include <cstddef>

#include "kv_cache.h"

namespace tcd {
namespace {

constexpr int kTile = 128;                  // slots of a key-value tile, rows of an M tile
constexpr int kThreads = 512;
constexpr uint32_t kHalfBytes = kTile * 128; // 128 rows of 64 elements
constexpr float kRescale = 8.f;             // log2 of the growth that moves the reference maximum
constexpr int kSegs = 4;                    // segments ahead of the softmax groups
constexpr int kWaitLimit = 1 << 22; // default polls of one wait before giving up
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kTileBytes = kHalves * kHalfBytes;
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kStep = D == 128 ? 64 : 128;  // slots of a step
  static constexpr int kSteps = kTile / kStep;       // steps of a tile
  // What an item's beginning and its end take, in tiles.
  static constexpr int kBegin = D == 128 ? 1 : 2, kEnd = 2;
  // Tensor memory of a group: scores, weights, accumulator.
  static constexpr int kPs = D == 128 ? 2 : 1;  // places of the weights
  static constexpr uint32_t kP = kStep, kO = kP + kPs * (kStep / 2), kCols = 256;
  static_assert(kO + D <= kCols, "tensor memory of a group");
  static_assert(kSteps == kHalves, "the clearing of values shares out a step's rows in these parts");
};

// A CTA's part of an item.
struct Seg {
  int32_t valid;     // 0: no more
  int32_t seq, row0, n, ctx, head;
  int32_t tok0;      // the item's first token
  int32_t t0, t1;    // its key-value tiles [t0, t1)
  int32_t end;       // no row of the item sees this slot or a later one
  int32_t two;       // two M tiles
  int32_t part;      // -1: the whole item; else the slot of the partial result
  int32_t last;      // (slot 1) the last worker that has a part of the item
};

struct AttendParams {
  KvView kv;
  TokensView tok;
  int32_t q_heads, group, tile_tokens;  // tile_tokens = 128 / group
  int32_t max_tokens;
  int32_t q_rows;                       // rows of one query load
  float c;                              // |scale| log2(e), the factor of the exponents
  int32_t negate;                       // the scale is negative
  const int64_t* tree;
  int32_t words;
  uint8_t* out;
  int64_t out_stride;
  int32_t wide_out;                     // 32-byte stores are aligned
  float* lse;
  int32_t* status;
  int32_t workers;
  Seg* descs;        // [workers] item that starts in a worker and goes on in the next (valid = 0: none)
  int32_t* errs;     // [workers] a wait ran out
  float2* part_ml;   // [workers][2][256] maximum and sum of each row
  float* part_o;     // [workers][2][D / 4][256][4]
  int32_t wait_limit;
  int32_t withhold;  // test switch: the first workers' first loads are not issued
};

constexpr size_t part_rows(int workers) { return (size_t)workers * 2 * 2 * kTile; }

struct Hdr {
  // Key-value ring (twice as many barriers as stages) and query tiles (four for
  // two places): a waiter looks at its own turns only, and a parity
  // tells a phase from the one before only if that one is known to be over.
  // It is: a place is filled when the one before in the same place has been
  // handed back, so what lies a whole ring further back than the waiter's
  // last turn is done.
  uint64_t full[20], empty[20];
  uint64_t q_full[4], q_empty[2];
  uint64_t s_full[2], o_full[2];
  uint64_t s_read[2], p_ready[2][2];  // (two: by step, even and odd)
  uint64_t pv_done[2][2];
  uint64_t o_free;                   // both groups have read the accumulators
  uint64_t meet;                     // both groups
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t drain;
  uint32_t tmem_base;
  int32_t abort;
  int64_t off0;                      // the worker's first unit within its sequence
  int32_t seq0, row0, n0, ctx0;      // its sequence
  uint32_t bad[3][8];                // tokens whose values are not finite, by segment
  Seg seg[kSegs];
  float2 ml[2][kTile];               // (the prologue's sums before the first segment)
};
template <int D>
constexpr size_t smem_bytes() {
  return (2 + Cfg<D>::kStages) * (size_t)Cfg<D>::kTileBytes + sizeof(Hdr);
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory of one CTA");

// -------------------------------------------------------------- PTX wrappers

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// One poll of a phase (it waits a while in hardware).
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
// Waits for a phase, at most `limit` polls; false if it gave up or another wait
// of the CTA has.  (One poll by itself in front, as most waits of the softmax groups
// are over when they begin: with a counted loop in front a prompt of 8192 took
// 475 us where this took 436.)
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, int limit, volatile int32_t* abort) {
  if (mbar_try(bar, parity)) return true;
  int i = 1;
#pragma unroll 1
  do {
    if (mbar_try(bar, parity)) return true;
    ++i;
  } while (i < limit && !*abort);
  *abort = 1;
  return false;
}
// The same for a whole warp, with one answer for all of it.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int limit, volatile int32_t* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit, abort));
}
__device__ __forceinline__ void tma_kv(uint32_t dst, const CUtensorMap* map, int slot, int half, int head, int page,
                                       uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
      "%6}], [%7];" ::"r"(dst),
      "l"(map), "r"(0), "r"(slot), "r"(half), "r"(head), "r"(page), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_q(uint32_t dst, const CUtensorMap* map, int x, int head, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(head), "r"(row), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptors, 128-byte swizzle.  K-major (queries,
// keys): rows of 128 bytes, groups of 8 rows 1024 bytes apart.  N-major
// (values: a row is one slot, the columns are N): groups of 8 slots 1024 bytes
// apart (stride offset), blocks of 64 columns further apart (leading offset).
__device__ __forceinline__ uint64_t desc_k_major(uint32_t a) {
  return (uint64_t)((a & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
__device__ __forceinline__ uint64_t desc_n_major(uint32_t a) {
  return (uint64_t)((a & 0x3FFFFu) >> 4) | (uint64_t)(kHalfBytes >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Instruction descriptor of kind::f16: 32-bit accumulator, M = 128.
template <typename T>
__device__ __forceinline__ constexpr uint32_t idesc(int n, bool b_n_major, bool negate_a = false) {
  const uint32_t ty = T::kMma;
  return (1u << 4) | (ty << 7) | (ty << 10) | (negate_a ? 1u << 13 : 0u) | (b_n_major ? 1u << 16 : 0u) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 32 columns of the warp's 32 rows (issued only: wait with tmem_ld_wait).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Ties the registers of a load to the wait before it, so that no use of them
// can be moved ahead of the wait.
__device__ __forceinline__ void tmem_arrived(uint32_t* r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint64_t f2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unf2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void stg256(void* a, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// ------------------------------------------------------------ the work's line

// (Divisions here are of 32 bits: the code of a 64-bit one is long, and a small
// call is bound by the fetch of its instructions.)

// sum over i < n of floor((a i + b) / m), in O(log m) steps like Euclid's algorithm
// (Graham, Knuth and Patashnik, "Concrete Mathematics", section 3.5); a n + b fits
// 32 bits.
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  int64_t ans = 0;
  while (n > 0) {
    const uint32_t qa = a / m, qb = b / m;
    ans += (int64_t)n * (n - 1) / 2 * qa + (int64_t)n * qb;
    a -= qa * m;
    b -= qb * m;
    const uint32_t y = a * n + b;
    n = y / m;
    b = y - n * m;
    const uint32_t t = m;
    m = a;
    a = t;
    if (n == 0) break;  // (m may be 0 now)
  }
  return ans;
}

// a / n for n < 2^16, in pieces of 16 bits.
__device__ __forceinline__ int64_t div_small(int64_t a, uint32_t n) {
  uint32_t rest = 0;
  int64_t q = 0;
#pragma unroll 1
  for (int i = (uint64_t)a >> 32 ? 48 : 16; i >= 0; i -= 16) {
    const uint32_t t = rest << 16 | ((uint32_t)(a >> i) & 0xffffu), d = t / n;
    rest = t - d * n;
    q = q << 16 | d;
  }
  return q;
}

// Items and units of one sequence's key-value head.
struct Line {
  int n, ctx, step;  // tokens, cached tokens, tokens of an item
  bool causal;
  int extra;         // units of an item beside its tiles
  __device__ int items() const { return (n + step - 1) / step; }
  // tiles of item i
  __device__ int tiles(int i) const {
    const int64_t end = causal ? min((int64_t)n, (int64_t)(i + 1) * step) : n;
    return (int)((ctx + end + kTile - 1) / kTile);
  }
  // units of the items before item i
  __device__ __forceinline__ int64_t before(int i) const {
    if (!causal) return (int64_t)i * (tiles(0) + extra);
    return floor_sum(i, kTile, step, (uint32_t)ctx + step + kTile - 1) + (int64_t)i * extra;
  }
  __device__ __forceinline__ int64_t units() const {
    if (n <= step) return n > 0 ? tiles(0) + extra : 0;  // (one item)
    return before(items() - 1) + tiles(items() - 1) + extra;
  }
  // The item that unit u is in; u becomes its number within the item.
  __device__ __forceinline__ int item_of(int64_t& u) const {
    if (n <= step) return 0;
    if (!causal) {  // (at most 256 tokens: the units of a head fit 32 bits)
      const uint32_t per = tiles(0) + extra, i = (uint32_t)u / per;
      u -= (int64_t)i * per;
      return (int)i;
    }
    int lo = 0, hi = items();
    int64_t at = 0;
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      const int64_t x = before(mid);
      if (x <= u) {
        lo = mid;
        at = x;
      } else {
        hi = mid;
      }
    }
    u -= at;
    return lo;
  }
};

__device__ __forceinline__ bool line_of(const AttendParams& p, int b, int extra, SeqSpan* s, Line* l) {
  const bool ok = seq_span(p.tok, p.kv.page_size, b, s) && s->n <= p.max_tokens;
  l->n = ok ? s->n : 0;
  l->ctx = ok ? s->ctx : 0;
  l->step = 2 * p.tile_tokens;
  l->causal = p.tree == nullptr;
  l->extra = extra;
  return ok;
}

// The first unit of worker w: total * w / active, in two parts that need no
// long division.
struct Cut {
  int64_t q;
  uint32_t r, active;
  __device__ Cut(int64_t total, int n) : q(n ? div_small(total, n) : 0), r((uint32_t)(total - q * n)), active(n) {}
  __device__ int64_t start(int w) const { return q * w + r * (uint32_t)w / active; }
};

// Which of the 32 NW slots from `start` a row sees.
template <int NW>
__device__ __forceinline__ void row_mask(const AttendParams& p, const Seg& g, int tok, int start, uint32_t (&m)[NW]) {
  int left = g.end - start;  // slots from `start` that any row sees
  if (!p.tree) left = g.ctx + tok + 1 - start;
  uint32_t v[NW + 1];
  // The first slot as a drafted token's number, and the row's words from the
  // one that holds its bit: all ones before the first, none after the last.
  // The loads do not wait for one another.
  const int x = start - g.ctx, first = x >> 5;
  if (p.tree) {
    const uint32_t* row = reinterpret_cast<const uint32_t*>(p.tree) + (int64_t)(g.row0 + tok) * p.words * 2;
#pragma unroll
    for (int w = 0; w <= NW; ++w) {
      const int i = first + w;
      v[w] = i < 0 ? 0xffffffffu : 0u;
      if (i >= 0 && i < 2 * p.words) v[w] = __ldg(row + i);
    }
  }
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int k = left - 32 * w;
    m[w] = k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u;
    if (p.tree) m[w] &= __funnelshift_r(v[w], v[w + 1], (uint32_t)x & 31u);
  }
}

// The first slot of an item that some row of it does not see.
__device__ __forceinline__ int first_hidden(const AttendParams& p, const Seg& g) {
  return p.tree ? g.ctx : g.ctx + g.tok0 + 1;
}

// Slots of the step that starts at `start` which any row of the item sees.
template <int D>
__device__ __forceinline__ int step_slots(const Seg& g, int start) {
  return min(Cfg<D>::kStep, g.end - start);
}
// Steps of a tile (the last one of an item may end in its first half).
template <int D>
__device__ __forceinline__ int steps_of(const Seg& g, int tile) {
  return min(Cfg<D>::kSteps, (g.end - tile * kTile + Cfg<D>::kStep - 1) / Cfg<D>::kStep);
}

// A pair with zeros for what is infinite or NaN.
template <typename T>
__device__ __forceinline__ uint32_t only_finite(uint32_t v) {
  if ((v & T::kExp) == T::kExp) v &= 0xffff0000u;
  if ((v & (T::kExp << 16)) == (T::kExp << 16)) v &= 0x0000ffffu;
  return v;
}
// What only_finite takes out.
template <typename T>
__device__ __forceinline__ float2 non_finite(uint32_t v) {
  const float2 f = T::unpack(v);
  return make_float2((v & T::kExp) == T::kExp ? f.x : 0.f, (v & (T::kExp << 16)) == (T::kExp << 16) ? f.y : 0.f);
}

// Logarithm of a row's sum of exponentials.
template <typename T>
__device__ __forceinline__ float log_sum(float m, float l, float c) {
  return l == 0.f ? -INFINITY : (m * c + (log2f(l) - T::kShift)) * kLn2;
}

// Adds to 32 columns of a row the infinities and NaN that were taken out of the
// values of slots it sees (from the cache itself; rare).
template <typename T, int D>
__device__ __forceinline__ void add_taken_out(const AttendParams& p, const Seg& g, const uint32_t* bad, int hidden,
                                           int tok, int c, float (&v)[32]) {
#pragma unroll 1
  for (int i = 0; i < 8; ++i)
#pragma unroll 1
    for (uint32_t w = bad[i]; w; w &= w - 1) {
      const int slot = hidden + i * 32 + __ffs(w) - 1;
      uint32_t mask[1];
      row_mask<1>(p, g, tok, slot, mask);
      if (!(mask[0] & 1u)) continue;
      const int page = __ldg(p.tok.table + (int64_t)g.seq * p.tok.width + (slot >> p.kv.page_shift));
      if ((uint32_t)page >= (uint32_t)p.kv.pages) continue;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          p.kv.base + ((((int64_t)page * 2 + 1) * p.kv.kv_heads + g.head) * p.kv.page_size +
                       (slot & (p.kv.page_size - 1))) * D * 2 + c * 2);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float2 x = non_finite<T>(__ldg(src + e));
        v[2 * e] += x.x;
        v[2 * e + 1] += x.y;
      }
    }
}

// ------------------------------------------------------------------- kernel

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const AttendParams p, const __grid_constant__ CUtensorMap map_kv,
                  const __grid_constant__ CUtensorMap map_q) {
  using C = Cfg<D>;
  constexpr int NS = C::kStages;
  extern __shared__ __align__(1024) unsigned char smem[];
  Hdr* hdr = reinterpret_cast<Hdr*>(smem + (2 + NS) * (size_t)C::kTileBytes);
  const uint32_t q_s = smem_u32(smem), kv_s = q_s + 2 * C::kTileBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int worker = blockIdx.x;
  volatile int32_t* abort = &hdr->abort;
  const int wl = p.wait_limit;

  // The swizzle wants tiles on 1024-byte boundaries; dynamic shared memory
  // starts on one where a kernel has no other.
  if (q_s & 1023u) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
      p.descs[worker].valid = 0;
      p.errs[worker] = 1;
    }
    return;
  }
  // Arrivals that complete a phase of each barrier (a thread each: one thread
  // for all of them takes a microsecond).
  constexpr int kBars = offsetof(Hdr, tmem_base) / 8;
  static_assert(kBars <= kThreads, "barriers");
  if (tid < kBars) {
    const uint32_t at = tid * 8;
    uint32_t n = 1;
    if (at >= offsetof(Hdr, empty) && at < offsetof(Hdr, q_full)) n = 2;      // a commit per group, or two of one
    if (at >= offsetof(Hdr, q_empty) && at < offsetof(Hdr, s_full)) n = 2;
    if (at >= offsetof(Hdr, s_read) && at < offsetof(Hdr, pv_done)) n = kTile;  // a group's threads
    if (at >= offsetof(Hdr, o_free) && at < offsetof(Hdr, seg_full)) n = 2 * kTile;
    if (at >= offsetof(Hdr, seg_empty) && at < offsetof(Hdr, drain)) n = 7 + 8;  // loaders, issuers, softmax warps
    if (at == offsetof(Hdr, drain)) n = 4;
    mbar_init(smem_u32(hdr) + at, n);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == kBars) {
    hdr->abort = 0;
    hdr->seq0 = -1;
    for (int i = 0; i < 24; ++i) hdr->bad[i >> 3][i & 7] = 0u;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_kv)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_q)) : "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&hdr->tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // The setup above touches only this CTA; everything read or written from
  // here on may belong to the kernel before.
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // Tiles and items of every sequence: thread i counts a run of them, then a
  // scan over the CTA gives the totals and who holds this worker's first unit.
  const int run = (p.tok.batch + kThreads - 1) / kThreads;
  int64_t* sums = reinterpret_cast<int64_t*>(hdr->ml);
  int64_t tiles = 0, items = 0;
  for (int i = 0; i < run; ++i) {
    const int b = tid * run + i;
    SeqSpan s;
    Line l;
    if (b < p.tok.batch && line_of(p, b, 0, &s, &l) && s.n > 0) {
      tiles += l.units() * p.kv.kv_heads;
      items += (int64_t)l.items() * p.kv.kv_heads;
    }
  }
  int64_t tiles_to = tiles, items_to = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, tiles_to, o), y = __shfl_up_sync(0xffffffffu, items_to, o);
    if (lane >= o) {
      tiles_to += x;
      items_to += y;
    }
  }
  if (lane == 31) {
    sums[warp] = tiles_to;
    sums[kThreads / 32 + warp] = items_to;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t all_tiles = 0, all_items = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) {
      tiles_to += sums[i];
      items_to += sums[kThreads / 32 + i];
    }
    all_tiles += sums[i];
    all_items += sums[kThreads / 32 + i];
  }
  constexpr int extra = C::kBegin + C::kEnd;
  const int64_t total = all_tiles + extra * all_items;
  const int active = (int)min((int64_t)p.workers, total);
  const Cut cut(total, active);
  const int64_t begin = worker < active ? cut.start(worker) : 0;
  const int64_t end = worker < active ? cut.start(worker + 1) : 0;
  const int64_t excl = tiles_to - tiles + extra * (items_to - items);
  if (begin < end && begin >= excl && begin < excl + tiles + extra * items) {
    int64_t at = excl;
    for (int i = 0; i < run; ++i) {
      const int b = tid * run + i;
      SeqSpan s;
      Line l;
      if (b >= p.tok.batch || !line_of(p, b, extra, &s, &l)) continue;
      const int64_t u = l.units() * p.kv.kv_heads;
      if (begin < at + u) {
        hdr->seq0 = b;
        hdr->row0 = s.row0;
        hdr->n0 = s.n;
        hdr->ctx0 = s.ctx;
        hdr->off0 = begin - at;
        break;
      }
      at += u;
    }
  }
  __syncthreads();
  const uint32_t tmem = hdr->tmem_base;
  // (a worker has one unit or more: one of these has the first item's first tile)
  const bool held = p.withhold != 0 && worker <= C::kBegin;
  uint32_t armed = 0;  // loaders: tiles armed, for the exit path
  // Registers: 512 threads launch with 128 each, 65,536 together.  A softmax
  // thread holds a step's row of scores: 64 (head_dim 128: 200 registers, the
  // others keep 56) or 128 (head_dim 64: 216 and 40); (56 + 200) * 256 and
  // (40 + 216) * 256 are 65,536.
  if (warp < 8) {
  if constexpr (D == 128)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
  if (warp == 0 || warp == 5) {
    // ------------------------------------------- loaders of keys and values
    // The warp's t-th tile lies in place 2 t (keys) or 2 t + 1 (values) of the ring.
    const uint32_t is_v = warp == 5;
    const int box = p.kv.page_size, pieces = kTile / box;
    const int piece = lane / C::kHalves, half = lane % C::kHalves;
    const uint32_t dst = kv_s + half * kHalfBytes + piece * box * 128;
    const uint32_t bytes = (uint32_t)box * 128;  // of one copy
    bool stop = false;
    for (int k = 0; !stop; ++k) {
      if (!warp_wait(smem_u32(&hdr->seg_full[k % kSegs]), (k / kSegs) & 1, wl, abort)) break;
      const Seg g = hdr->seg[k % kSegs];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&hdr->seg_empty[k % kSegs]));
      if (!g.valid) break;
      const int32_t* row = p.tok.table + (int64_t)g.seq * p.tok.width;
      const int head = (is_v ? p.kv.kv_heads : 0) + g.head;
      int slot = g.t0 * kTile + piece * box;
      bool load = piece < pieces && slot < g.end;
      int page = load ? __ldg(row + (slot >> p.kv.page_shift)) : 0;
      for (int t = g.t0; t < g.t1; ++t, ++armed) {
        // (the next tile's pages are looked up before this one's place is waited for)
        const int slot2 = slot + kTile;
        const bool load2 = piece < pieces && slot2 < g.end && t + 1 < g.t1;
        const int page2 = load2 ? __ldg(row + (slot2 >> p.kv.page_shift)) : 0;
        const uint32_t at = 2 * armed + is_v, before = at - NS;
        if (at >= NS && !warp_wait(smem_u32(&hdr->empty[before % (2 * NS)]), (before / (2 * NS)) & 1, wl, abort)) {
          stop = true;
          break;
        }
        const uint32_t bar = smem_u32(&hdr->full[at % (2 * NS)]);
        const uint32_t count = __popc(__ballot_sync(0xffffffffu, load));
        if (lane == 0) mbar_expect_tx(bar, count * bytes);
        __syncwarp();
        if (load && !(held && at == 0))
          tma_kv(dst + at % NS * C::kTileBytes, &map_kv, slot & (p.kv.page_size - 1), half, head, page, bar);
        slot = slot2;
        load = load2;
        page = page2;
      }
    }
  } else if (warp == 7) {
    // -------------------------------------------------- loader of queries
    if (lane == 0) {
      bool stop = false;
      for (int k = 0; !stop; ++k) {
        if (!mbar_wait(smem_u32(&hdr->seg_full[k % kSegs]), (k / kSegs) & 1, wl, abort)) break;
        const Seg g = hdr->seg[k % kSegs];
        mbar_arrive(smem_u32(&hdr->seg_empty[k % kSegs]));
        if (!g.valid) break;
        for (int m = 0; m <= g.two; ++m, ++armed) {
          if (!mbar_wait(smem_u32(&hdr->q_empty[armed & 1]), ((armed >> 1) & 1) ^ 1, wl, abort)) {
            stop = true;
            break;
          }
          const uint32_t bar = smem_u32(&hdr->q_full[armed & 3]);
          mbar_expect_tx(bar, (uint32_t)p.q_rows * 128u * C::kHalves);
          for (int h = 0; h < C::kHalves; ++h)
            tma_q(q_s + (armed & 1) * C::kTileBytes + h * kHalfBytes, &map_q, h * 64, g.head * p.group,
                  g.row0 + g.tok0 + m * p.tile_tokens, bar);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 3 || warp == 4 || warp == 6) {
    // ------------------------------------------------------------ issuers
    if (lane == 0) {
      const bool is_s = warp < 4;                          // score or output products
      const int slot = is_s ? warp >> 1 : (warp - 4) >> 1;        // whose
      const uint32_t t_s = tmem + slot * C::kCols, t_p = t_s + C::kP, t_o = t_s + C::kO;
      // (a negative scale is one of the negated products)
      const uint32_t id_s = idesc<T>(C::kStep, false, p.negate != 0);
      constexpr uint32_t id_o = idesc<T>(D, true);
      uint32_t it = 0, qi = 0, done = 0;  // ring places, query tiles, products
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && mbar_wait(smem_u32(bar), parity & 1, wl, abort);
        return ok;
      };
      // The stage is handed back when the products so far are done.
      auto release = [&](uint32_t at, bool two) {
        mma_commit(smem_u32(&hdr->empty[at % (2 * NS)]));
        if (!two) mma_commit(smem_u32(&hdr->empty[at % (2 * NS)]));
      };
      for (int k = 0; ok; ++k) {
        if (!wait(&hdr->seg_full[k % kSegs], k / kSegs)) break;
        const Seg g = hdr->seg[k % kSegs];
        mbar_arrive(smem_u32(&hdr->seg_empty[k % kSegs]));
        if (!g.valid) break;
        const int n = g.t1 - g.t0, hop = g.two ? 1 : 2, i0 = g.two ? 0 : slot;
        if (is_s) {
          const uint32_t q = qi + (g.two ? slot : 0);
          if (!wait(&hdr->q_full[q & 3], q >> 2)) break;
          const uint64_t q_desc = desc_k_major(q_s + (q & 1) * C::kTileBytes);
          for (int i = i0; i < n && ok; i += hop) {
            const uint32_t at = it + 2 * i, stage = at % NS;
            const int steps = steps_of<D>(g, g.t0 + i);
            if (!wait(&hdr->full[at % (2 * NS)], at / (2 * NS))) break;
            for (int u = 0; u < steps; ++u, ++done) {
              // (the scores before have been read)
              if (done > 0 && !wait(&hdr->s_read[slot], done - 1)) break;
              const uint64_t b = desc_k_major(kv_s + stage * C::kTileBytes + u * C::kStep * 128);
              tc_fence_after();
#pragma unroll
              for (int e = 0; e < D / 16; ++e) {
                const uint32_t o = (uint32_t)(e & 3) * 2, h = e >> 2;
                mma_ss(t_s, q_desc + h * (kHalfBytes >> 4) + o, b + h * (kHalfBytes >> 4) + o, id_s, e > 0);
              }
              // The product two steps ago is done as well when the scores are
              // announced: the softmax group need not wait for the weights' place.
              if (C::kPs > 1 && done > 1 && !wait(&hdr->pv_done[slot][done & 1], (done - 2) >> 1)) break;
              mma_commit(smem_u32(&hdr->s_full[slot]));
            }
            release(at, g.two);
          }
          if (!ok) break;
          mma_commit(smem_u32(&hdr->q_empty[q & 1]));
          if (g.two) mma_commit(smem_u32(&hdr->q_empty[q & 1]));
        } else {
          // (the accumulators of the segment before have been read)
          if (k > 0 && !wait(&hdr->o_free, k - 1)) break;
          for (int i = i0; i < n && ok; i += hop) {
            const uint32_t at = it + 2 * i + 1, stage = at % NS;
            const int steps = steps_of<D>(g, g.t0 + i);
            if (!wait(&hdr->full[at % (2 * NS)], at / (2 * NS))) break;
            for (int u = 0; u < steps; ++u, ++done) {
              const uint64_t b = desc_n_major(kv_s + stage * C::kTileBytes + u * C::kStep * 128);
              // over the 16-slot groups that the step has
              const int groups = (step_slots<D>(g, (g.t0 + i) * kTile + u * C::kStep) + 15) / 16;
              const bool more = i > i0 || u > 0;
              const uint32_t p_at = t_p + done % C::kPs * (C::kStep / 2);
              if (!wait(&hdr->p_ready[slot][done & 1], done >> 1)) break;
              tc_fence_after();
#pragma unroll
              for (int e = 0; e < C::kStep / 16; ++e)
                if (e < groups) mma_ts(t_o, p_at + e * 8, b + e * (2048 >> 4), id_o, more || e > 0);
              mma_commit(smem_u32(&hdr->pv_done[slot][done & 1]));
            }
            release(at, g.two);
          }
          mma_commit(smem_u32(&hdr->o_full[slot]));
        }
        it += 2 * n;
        qi += 1 + g.two;
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------------------------------------------------- segments
    if (lane == 0) {
      int64_t left = end - begin, off = hdr->off0;
      int b = hdr->seq0, k = 0;
      bool open_end = false, ok = true;
      if (b < 0) left = 0;
      Seg d{};
      while (ok) {
        Seg g{};
        if (left > 0) {
          SeqSpan s{hdr->row0, hdr->n0, hdr->ctx0};
          Line l{s.n, s.ctx, 2 * p.tile_tokens, p.tree == nullptr, extra};
          int64_t per = 0;
          if (b == hdr->seq0) {
            per = l.units();
          } else {
            // (sequences without units are passed over)
            while (b < p.tok.batch && !(line_of(p, b, extra, &s, &l) && (per = l.units()) > 0)) ++b;
            if (b >= p.tok.batch) break;  // (cannot be: the units add up)
          }
          // (kv_heads < 2^16)
          int h = 0;
          int64_t r = off;
#pragma unroll 1
          for (int i = 15; i >= 0; --i)
            if (r >= per << i) {
              r -= per << i;
              h |= 1 << i;
            }
          int item = l.item_of(r);
          // the rest of this sequence, segment by segment
          while (left > 0 && h < p.kv.kv_heads) {
            const int tiles = l.tiles(item);
            const int64_t take = min((int64_t)extra + tiles - r, left);
            g.t0 = (int)min(max(r - C::kBegin, (int64_t)0), (int64_t)tiles);
            g.t1 = (int)min(max(r + take - C::kBegin, (int64_t)0), (int64_t)tiles);
            if (g.t1 > g.t0) {
              g.valid = 1;
              g.seq = b;
              g.row0 = s.row0;
              g.n = s.n;
              g.ctx = s.ctx;
              g.head = h;
              g.tok0 = item * l.step;
              g.two = s.n - g.tok0 > p.tile_tokens;
              g.end = s.ctx + (p.tree ? s.n : min(s.n, g.tok0 + l.step));
              g.part = g.t1 - g.t0 == tiles ? -1 : g.t0 > 0 ? 0 : 1;
              g.last = worker;
              if (g.part == 1) {
                // the item's last unit lies with the worker that this finds
                const int64_t last_unit = end - left - r + C::kBegin + tiles - 1;
                int w = worker + 1;
                while (cut.start(w + 1) <= last_unit) ++w;
                g.last = w;
                d = g;
                open_end = true;
              }
              if (!mbar_wait(smem_u32(&hdr->seg_empty[k % kSegs]), ((k / kSegs) & 1) ^ 1, wl, abort)) {
                ok = false;
                break;
              }
              hdr->seg[k % kSegs] = g;
              mbar_arrive(smem_u32(&hdr->seg_full[k % kSegs]));
              ++k;
            }
            left -= take;
            r = 0;
            if (++item == l.items()) {
              item = 0;
              ++h;
            }
          }
          off = 0;
          ++b;
        } else {
          if (mbar_wait(smem_u32(&hdr->seg_empty[k % kSegs]), ((k / kSegs) & 1) ^ 1, wl, abort)) {
            hdr->seg[k % kSegs].valid = 0;
            mbar_arrive(smem_u32(&hdr->seg_full[k % kSegs]));
          }
          break;
        }
      }
      d.valid = open_end;
      p.descs[worker] = d;
    }
    __syncwarp();
  }
  } else {
    // ----------------------------------------------------- softmax groups
    if constexpr (D == 128)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int grp = (warp - 8) >> 2;               // which slot
    const int r = tid - 256 - grp * kTile;         // row of the M tile (TMEM lane)
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + grp * C::kCols;
    const uint32_t t_p = t_s + C::kP, t_o = t_s + C::kO, t_o0 = tmem + lane_base + C::kO;
    uint32_t n_s = 0, n_meet = 0, it = 0;
    auto meet = [&]() {
      mbar_arrive(smem_u32(&hdr->meet));
      const bool ok = warp_wait(smem_u32(&hdr->meet), n_meet & 1, wl, abort);
      ++n_meet;
      return ok;
    };
    for (int k = 0;; ++k) {
      if (!warp_wait(smem_u32(&hdr->seg_full[k % kSegs]), (k / kSegs) & 1, wl, abort)) break;
      const Seg g = hdr->seg[k % kSegs];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&hdr->seg_empty[k % kSegs]));
      if (!g.valid) break;
      const int n = g.t1 - g.t0;
      const int tok = g.tok0 + (g.two ? grp * p.tile_tokens : 0) + r / p.group;
      const bool live = r < p.tile_tokens * p.group && tok < g.n;
      const bool any = __any_sync(0xffffffffu, live);
      const int hidden = first_hidden(p, g);
      uint32_t* bad = hdr->bad[k % 3];
      float m = -INFINITY, l = 0.f;
      bool stop = false;
      constexpr int W = C::kStep;
      const int hop = g.two ? 1 : 2;
      const uint64_t c2 = f2(p.c, p.c);
      float off = 0.f;     // T::kShift - m c, or 0 while m is -inf
      bool first = true;   // no step of this segment yet
      // The scores of a step, read and handed back.
      auto load = [&](uint32_t(&s)[W]) {
#pragma unroll
        for (int c = 0; c < W; c += 32) tmem_ld32(t_s + c, s + c);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < W; c += 32) tmem_arrived(s + c);
        tc_fence_before();
        mbar_arrive(smem_u32(&hdr->s_read[grp]));
      };
      // The output product `back` steps ago is done.  One step ago: the
      // accumulator is at rest, and with one place for the weights it is free.
      // (With two, the scores' announcement says that the place is free.  In
      // either case warps without rows wait as well: a warp must not announce a
      // step's weights before the group's others have announced those that were in
      // the same place.)
      auto product_done = [&](uint32_t back) {
        const uint32_t j = n_s - back;
        return n_s < back || mbar_wait(smem_u32(&hdr->pv_done[grp][j & 1]), (j >> 1) & 1, wl, abort);
      };
      // Weights of a step's scores.
      auto weigh = [&](const uint32_t(&s)[W]) {
        float mx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = __uint_as_float(s[j]);
#pragma unroll
        for (int j = 4; j < W; j += 2)
          mx[(j >> 1) & 3] = max3(mx[(j >> 1) & 3], __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        bool ok = true;
        if (C::kPs == 1) {
          ok = product_done(1);
          tc_fence_after();
        }
        // Move the reference maximum only for a large growth (the first finite
        // score's among them); the accumulator exists from the second step on.
        const bool grow = (top - m) * p.c > kRescale;
        if (__any_sync(0xffffffffu, grow)) {
          if (!first) {
            if (C::kPs > 1) {
              ok &= product_done(1);
              __syncwarp();
              tc_fence_after();
            }
            const float f = grow ? ex2((m - top) * p.c) : 1.f;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(t_o + c, o);
              tmem_ld_wait();
              tmem_arrived(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st16(t_o + c, o);
              tmem_st16(t_o + c + 16, o + 16);
            }
            l *= f;
          }
          if (grow) {
            m = top;
            off = T::kShift - m * p.c;
          }
        }
        first = false;
        const uint64_t off2 = f2(off, off);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int q = 0; q < W / 32; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 x =
                unf2(fma2(f2(__uint_as_float(s[q * 32 + 2 * j]), __uint_as_float(s[q * 32 + 2 * j + 1])), c2, off2));
            const float a = ex2(x.x), b = ex2(x.y);
            sum[j & 1] = add2(sum[j & 1], f2(a, b));
            pk[j] = T::pack(a, b);
          }
          tmem_st16(t_p + n_s % C::kPs * (W / 2) + q * 16, pk);
        }
        const float2 t = unf2(add2(sum[0], sum[1]));
        l += t.x + t.y;
        tmem_st_wait();
        return ok;
      };
      // Steps that every row sees entirely, then those that some row does not.
      // (In the first loop a wait that ran out is noticed at the tile's end:
      // nothing in between leaves its bounds.)
      int i = g.two ? 0 : grp, u = 0;
      for (; i < n && !stop; i += hop) {
        const int steps = steps_of<D>(g, g.t0 + i);
        const int full = min(steps, max(0, hidden - (g.t0 + i) * kTile) / W);
        bool ok = true;
        for (u = 0; u < full; ++u, ++n_s) {
          ok &= mbar_wait(smem_u32(&hdr->s_full[grp]), n_s & 1, wl, abort);
          if (any) {
            __syncwarp();
            tc_fence_after();
            uint32_t s[W];
            load(s);
            ok &= weigh(s);
            tc_fence_before();
          } else {
            mbar_arrive(smem_u32(&hdr->s_read[grp]));
            if (C::kPs == 1) ok &= product_done(1);
          }
          mbar_arrive(smem_u32(&hdr->p_ready[grp][n_s & 1]));
        }
        stop = !__all_sync(0xffffffffu, ok);
        if (full < steps) break;
      }
      if (stop) break;
      for (; i < n && !stop; i += hop, u = 0) {
        const int steps = steps_of<D>(g, g.t0 + i);
        for (; u < steps; ++u, ++n_s) {
          const int start = (g.t0 + i) * kTile + u * W;  // the step's first slot
          const int slots = step_slots<D>(g, start);
          uint32_t mask[W / 32];
#pragma unroll
          for (int c = 0; c < W / 32; ++c) mask[c] = 0u;
          if (live) row_mask<W / 32>(p, g, tok, start, mask);
          if (!warp_wait(smem_u32(&hdr->s_full[grp]), n_s & 1, wl, abort)) {
            stop = true;
            break;
          }
          bool ok = true;
          if (any) {
            tc_fence_after();
            uint32_t s[W];
            load(s);
#pragma unroll
            for (int j = 0; j < W; ++j) s[j] = mask[j >> 5] & (1u << (j & 31)) ? s[j] : 0xff800000u;
            ok = weigh(s);
          } else {
            mbar_arrive(smem_u32(&hdr->s_read[grp]));
            ok = C::kPs > 1 || product_done(1);
          }
          if (!__all_sync(0xffffffffu, ok)) {
            stop = true;
            break;
          }
          {
            // Values of slots that some row must not see: zero past the item's
            // end, and infinities and NaN out (kept in `bad`).
            const uint32_t vi = it + 2 * i + 1;
            if (!warp_wait(smem_u32(&hdr->full[vi % (2 * NS)]), (vi / (2 * NS)) & 1, wl, abort)) {
              stop = true;
              break;
            }
            // A thread takes eight 16-byte words of one of the step's rows (four
            // with two M tiles: then each group takes half).  Past the end, only
            // the rest of its group of 16 slots is read.
            const int j = r % W, slot = start + j;
            const int c0 = r / W * 8 + (g.two ? grp * 4 : 0), c1 = c0 + (g.two ? 4 : 8);
            const uint32_t row = kv_s + (vi % NS) * C::kTileBytes + u * C::kStep * 128 + j * 128;
            if (slot >= g.end) {
              if (j < ((slots + 15) & ~15))
#pragma unroll 4
                for (int c = c0; c < c1; ++c)
                  sts128(row + (c >> 3) * kHalfBytes + (((c ^ j) & 7) << 4), make_uint4(0u, 0u, 0u, 0u));
            } else if (slot >= hidden) {
              bool found = false;
#pragma unroll 1
              for (int c = c0; c < c1; c += 4) {
                const uint32_t at = row + (c >> 3) * kHalfBytes;
                uint4 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = lds128(at + ((((c + e) ^ j) & 7) << 4));
                uint32_t odd = 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  odd = T::trace(v[e].w, T::trace(v[e].z, T::trace(v[e].y, T::trace(v[e].x, odd))));
                if (odd & 0x7fff7fffu) {
                  found = true;
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    sts128(at + ((((c + e) ^ j) & 7) << 4),
                           make_uint4(only_finite<T>(v[e].x), only_finite<T>(v[e].y), only_finite<T>(v[e].z),
                                      only_finite<T>(v[e].w)));
                }
              }
              if (found) {
                const int x = slot - hidden;  // fewer than 256: an item's tokens, or a tree's
                atomicOr(&bad[x >> 5], 1u << (x & 31));
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (g.two && !meet()) {
              stop = true;
              break;
            }
          }
          tc_fence_before();
          mbar_arrive(smem_u32(&hdr->p_ready[grp][n_s & 1]));
        }
      }
      if (stop) break;
      it += 2 * n;
      // ------------------------------------------------ end of the segment
      if (!g.two) hdr->ml[grp][r] = make_float2(m, l);
      if (tid == 256)
        for (int i = 0; i < 8; ++i) hdr->bad[(k + 1) % 3][i] = 0u;  // (last read before the groups met a segment ago)
      if (!meet()) break;
      const bool used1 = g.two || n > 1;
      if (!warp_wait(smem_u32(&hdr->o_full[0]), k & 1, wl, abort) ||
          !warp_wait(smem_u32(&hdr->o_full[1]), k & 1, wl, abort))
        break;
      tc_fence_after();
      // Factors of the two accumulators (one M tile: both are this row's; two: only the group's own).
      float f0 = 1.f, f1 = 1.f;
      if (!g.two) {
        const float2 a = hdr->ml[0][r], b = hdr->ml[1][r];
        m = fmaxf(a.x, b.x);
        f0 = m == -INFINITY ? 0.f : ex2((a.x - m) * p.c);
        f1 = m == -INFINITY ? 0.f : ex2((b.x - m) * p.c);
        l = a.y * f0 + b.y * f1;
      }
      uint32_t any_bad = 0;
      for (int i = 0; i < 8; ++i) any_bad |= bad[i];
      const int head = g.head * p.group + r % p.group;
      uint8_t* out = p.out + ((int64_t)(g.row0 + tok) * p.out_stride + (int64_t)head * D) * 2;
      const float norm = g.part >= 0 ? 1.f : l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // (NaN stays)
      const int rr = (g.two ? grp * kTile : 0) + r;
      const size_t part = ((size_t)worker * 2 + (g.part > 0)) * 2 * kTile;
      // Columns: all of the group's own accumulator, or half of both.
      const int c_lo = g.two ? 0 : grp * (D / 2), c_hi = g.two ? D : c_lo + D / 2;
      if (any) {
#pragma unroll 1
        for (int c = c_lo; c < c_hi; c += 32) {
          uint32_t o[32], o1[32];
          tmem_ld32((g.two ? t_o : t_o0) + c, o);
          if (!g.two && used1) tmem_ld32(t_o0 + C::kCols + c, o1);
          tmem_ld_wait();
          tmem_arrived(o);
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(o[j]) * f0;  // (two M tiles: f0 is 1)
          if (!g.two && used1) {
            tmem_arrived(o1);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = fmaf(__uint_as_float(o1[j]), f1, v[j]);
          }
          if (live && any_bad) add_taken_out<T, D>(p, g, bad, hidden, tok, c, v);
          if (live && g.part < 0) {
            // (64 bytes of a row: whole sectors, and no shared memory is held up
            // for the next item.  16 bytes a store: four prompts of 2048
            // 152 us against 148, 16 short ones 47 against 45.5)
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = T::pack(v[2 * j] * norm, v[2 * j + 1] * norm);
            if (p.wide_out) {
              stg256(out + c * 2, w);
              stg256(out + c * 2 + 32, w + 8);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                reinterpret_cast<uint4*>(out + c * 2)[j] =
                    make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            }
          } else if (live) {
            // (a warp's rows are neighbours: 512 bytes at a time)
            float4* dst = reinterpret_cast<float4*>(p.part_o + part * D) + (size_t)(c / 4) * (2 * kTile) + rr;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              dst[j * 2 * kTile] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
        }
      }
      // The accumulators have been read.
      tc_fence_before();
      mbar_arrive(smem_u32(&hdr->o_free));
      if (live && (g.two || grp == 0)) {
        if (g.part >= 0)
          p.part_ml[part + rr] = make_float2(m, l);
        else if (p.lse)
          p.lse[(int64_t)(g.row0 + tok) * p.q_heads + head] = log_sum<T>(m, l, p.c);
      }
      if (!g.two && !meet()) break;  // (ml has been read)
    }
  }

  tc_fence_before();
  __syncthreads();
  if (hdr->abort) {
    // A wait ran out.  Everything this CTA started has to end before it
    // leaves (waits bounded again): the products that were issued, and the
    // loads of stages that no product has consumed.
    if ((warp == 1 || warp == 3 || warp == 4 || warp == 6) && lane == 0) {
      mma_commit(smem_u32(&hdr->drain));
      int32_t none = 0;
      mbar_wait(smem_u32(&hdr->drain), 0u, wl, &none);
    }
    if ((warp == 0 || warp == 5) && lane == 0) {
      int32_t none = 0;
      constexpr uint32_t most = (NS + 1) / 2;  // tiles of one loader in the ring
      for (uint32_t t = armed > most ? armed - most : 0; t < armed; ++t) {
        const uint32_t at = 2 * t + (warp == 5);
        if (!(held && at == 0)) mbar_wait(smem_u32(&hdr->full[at % (2 * NS)]), (at / (2 * NS)) & 1, wl, &none);
      }
    }
    if (warp == 7 && lane == 0) {
      int32_t none = 0;
      for (uint32_t j = armed > 2 ? armed - 2 : 0; j < armed; ++j)
        mbar_wait(smem_u32(&hdr->q_full[j & 3]), (j >> 2) & 1, wl, &none);
    }
    __syncwarp();
  }
  if (tid == 0) p.errs[worker] = hdr->abort;
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ------------------------------------------------------------ joining kernel

constexpr int kJoinThreads = 256, kJoinBlocks = 8;

// kJoinBlocks blocks for each worker: the item that starts in it and goes on in
// the next.  A thread joins four columns of a row (the parts are laid out by
// columns, so neighbouring rows are neighbours); the parts are added in the
// order of the workers: the result does not depend on timing.  Bound: latency (a
// few parts of a few rows; up to 40 MB of partial results when every worker has
// two full ones, 6 us at a copy's rate).  Blocks a worker, 16 short prompts and
// drafts of 16 sequences: 4 50 and 74.6 us, 8 45.5 and 73.6, 16 43.6 and 75.2.
// Letting the blocks start while the first kernel still runs is slower (one token
// 18.1 us against 17.4).  The blocks after these write the status of a sequence
// each (one block, as a warp takes 10 us for the pages of 131,000 slots).
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const AttendParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x >= (unsigned)(p.workers * kJoinBlocks)) {
    const int b = blockIdx.x - p.workers * kJoinBlocks;
    SeqSpan s;
    bool ok = seq_span(p.tok, p.kv.page_size, b, &s) && s.n <= p.max_tokens;
    const int pages = ok && s.n > 0 ? (s.ctx + s.n - 1) / p.kv.page_size + 1 : 0;
    const int32_t* row = p.tok.table + (int64_t)b * p.tok.width;
#pragma unroll 4
    for (int i = threadIdx.x; i < pages; i += kJoinThreads) ok &= (uint32_t)__ldg(row + i) < (uint32_t)p.kv.pages;
    bool late = false;
    for (int i = threadIdx.x; i < p.workers; i += kJoinThreads) late |= __ldcg(p.errs + i) != 0;
    ok = __syncthreads_and(ok);
    late = __syncthreads_or(late);
    if (threadIdx.x == 0)
      set_status(p.status, b, late ? TC_ERR_DEVICE_TIMEOUT : ok ? TC_OK : TC_ERR_BOUNDS, p.kv.keep);
    return;
  }
  const int w0 = blockIdx.x / kJoinBlocks, y = blockIdx.x % kJoinBlocks;
  const Seg g = p.descs[w0];
  if (!g.valid) return;
  const int full = p.tile_tokens * p.group, left = (g.n - g.tok0) * p.group;
  const int v0 = min(left, full), rows = g.two ? min(left, 2 * full) : v0;  // rows of the first M tile, of both
  for (int i = y * kJoinThreads + threadIdx.x; i < rows * (D / 4); i += kJoinBlocks * kJoinThreads) {
    const int c = i / rows, k = i % rows;            // columns 4 c .. 4 c + 3 of row k
    const int rr = k < v0 ? k : kTile + k - v0;      // its place in a part
    auto at = [&](int w) { return ((size_t)w * 2 + (w == w0)) * 2 * kTile; };
    float m = -INFINITY;
#pragma unroll 8
    for (int w = w0; w <= g.last; ++w) m = fmaxf(m, __ldcg(&p.part_ml[at(w) + rr].x));
    float l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int w = w0; w <= g.last; ++w) {
      const float2 ml = __ldcg(p.part_ml + at(w) + rr);
      const float4 o = __ldcg(reinterpret_cast<const float4*>(p.part_o + at(w) * D) + (size_t)c * (2 * kTile) + rr);
      const float f = m == -INFINITY ? 0.f : ex2((ml.x - m) * p.c);
      l = fmaf(ml.y, f, l);
      v.x = fmaf(o.x, f, v.x);
      v.y = fmaf(o.y, f, v.y);
      v.z = fmaf(o.z, f, v.z);
      v.w = fmaf(o.w, f, v.w);
    }
    const float norm = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    const int tok = g.tok0 + k / p.group, head = g.head * p.group + k % p.group;
    const int64_t row = g.row0 + tok;
    *reinterpret_cast<uint2*>(p.out + (row * p.out_stride + (int64_t)head * D + 4 * c) * 2) =
        make_uint2(T::pack(v.x * norm, v.y * norm), T::pack(v.z * norm, v.w * norm));
    if (p.lse && c == 0)
      p.lse[row * p.q_heads + head] = log_sum<T>(m, l, p.c);
  }
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

bool encode(CUtensorMap* m, int dtype, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return fn && fn(m, dtype == TC_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

// SMs of a device (asked once).
int sm_count(int device) {
  static int known[kMaxDevices];  // (a race writes the same value)
  if (device < 0 || device >= kMaxDevices) return 0;
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

size_t workspace_bytes(int workers, int head_dim) {
  return (size_t)workers * (sizeof(Seg) + 16) + part_rows(workers) * (sizeof(float2) + sizeof(float) * head_dim) + 64;
}

template <typename T, int D>
cudaError_t launch(const AttendParams& p, const CUtensorMap& kv, const CUtensorMap& q, cudaStream_t s) {
  static bool ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(attend_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<D>());
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)p.workers);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D>();
  e = cudaLaunchKernelEx(&cfg, attend_kernel<T, D>, p, kv, q);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(p.workers * kJoinBlocks + p.tok.batch));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attend_join_kernel<T, D>, p);
}

}  // namespace
}  // namespace tcd

using namespace tcd;

extern "C" tc_status tc_attend_workspace(const tc_kv_t* kv, int64_t* bytes) {
  const tc_status rc = kv_check("tc_attend_workspace", kv);
  if (rc != TC_OK) return rc;
  if (!bytes) return kv_fail(TC_ERR_INVALID_ARG, "tc_attend_workspace: bytes is NULL");
  const int sms = sm_count(kv->device);
  if (sms < 1) return kv_fail(TC_ERR_CUDA, "tc_attend_workspace: no such device");
  *bytes = (int64_t)workspace_bytes(sms, kv->head_dim);
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
  // Keys and values of the layer: [page][keys or values, head][slot][element],
  const KvView v = kv_view(kv, layer);
  const cuuint64_t d = (cuuint64_t)kv->head_dim, sz = (cuuint64_t)kv->page_size;
  // in pieces of 64 columns.  A copy brings a page's slots of one piece.
  const int halves = kv->head_dim / 64;
  const cuuint64_t kv_dims[5] = {64, sz, (cuuint64_t)halves, (cuuint64_t)2 * kv->kv_heads, (cuuint64_t)kv->pages};
  const cuuint64_t kv_strides[4] = {d * 2, 128, sz * d * 2, (cuuint64_t)2 * kv->kv_heads * sz * d * 2};
  const cuuint32_t kv_box[5] = {64, (cuuint32_t)kv->page_size, 1, 1, 1};
  const int group = a->q_heads / kv->kv_heads, tile_tokens = kTile / group;
  // Queries: rows (token, head of the group) of one M tile, at most max_tokens of them.
  const int q_tokens = a->max_tokens < 1 ? 1 : a->max_tokens < tile_tokens ? a->max_tokens : tile_tokens;
  const bool none = tokens->n_tokens == 0;  // (no queries: the map is not used, any valid one does)
  const cuuint64_t q_dims[3] = {d, (cuuint64_t)(none ? group : a->q_heads), (cuuint64_t)(none ? 1 : tokens->n_tokens)};
  const cuuint64_t q_strides[2] = {d * 2, (cuuint64_t)(none ? row : a->q_stride) * 2};
  const cuuint32_t q_box[3] = {64, (cuuint32_t)group, (cuuint32_t)q_tokens};
  CUtensorMap map_kv, map_q;
  if (!encode(&map_kv, kv->dtype, 5, v.base, kv_dims, kv_strides, kv_box) ||
      !encode(&map_q, kv->dtype, 3, none ? kv->pool : a->q, q_dims, q_strides, q_box))
    return kv_fail(TC_ERR_UNSUPPORTED, "tc_attend: the sizes or strides do not fit a tensor map");
  AttendParams p{};
  p.kv = v;
  p.tok = tokens_view(tokens);
  p.q_heads = a->q_heads;
  p.group = group;
  p.tile_tokens = tile_tokens;
  p.max_tokens = a->max_tokens;
  p.q_rows = group * q_tokens;
  // A scale of zero weighs all slots alike; as a factor so small that every
  // product with a score is nothing, it keeps -inf times the factor -inf.
  p.c = fmaxf(fabsf(a->scale) * 1.4426950408889634f, 1e-30f);
  p.negate = a->scale < 0.f;
  p.tree = a->tree;
  p.words = a->tree ? a->tree_words : 0;
  p.out = static_cast<uint8_t*>(a->out);
  p.out_stride = a->out_stride;
  p.wide_out = !kv_misaligned(a->out, 32) && a->out_stride % 16 == 0;
  p.lse = a->lse;
  p.status = status;
  p.workers = sm_count(kv->device);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  ws += part_rows(p.workers) * sizeof(float) * kv->head_dim;
  p.part_ml = reinterpret_cast<float2*>(ws);
  ws += part_rows(p.workers) * sizeof(float2);
  p.descs = reinterpret_cast<Seg*>(ws);
  ws += (size_t)p.workers * sizeof(Seg);
  p.errs = reinterpret_cast<int32_t*>(ws);
  p.wait_limit = a->wait_polls > 0 ? (int32_t)(a->wait_polls < 1 << 30 ? a->wait_polls : 1 << 30) : kWaitLimit;
  p.withhold = a->withhold;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (kv->dtype == TC_DT_BF16)
    e = kv->head_dim == 128 ? launch<Bf16, 128>(p, map_kv, map_q, s) : launch<Bf16, 64>(p, map_kv, map_q, s);
  else
    e = kv->head_dim == 128 ? launch<F16, 128>(p, map_kv, map_q, s) : launch<F16, 64>(p, map_kv, map_q, s);
  return e == cudaSuccess ? TC_OK : kv_cuda_fail(e, "tc_attend: ");
}
