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
#include <type_traits>

#include "kv_cache.h"

namespace tcd {
namespace {

constexpr int kTile = 128;                  // slots of a key-value tile, rows of an M tile
constexpr int kThreads = 512;
constexpr uint32_t kHalfBytes = kTile * 128; // 128 rows of 64 elements
constexpr float kRescale = 8.f;             // log2 of the growth that moves the reference maximum
constexpr int kSegs = 4;                    // segments ahead of the softmax groups
constexpr int kWaitLimit = 1 << 22; // default polls of one wait before giving up, and the fewest of those at a CTA's end
                                    // for what it has in flight, which must not outlive it, however soon others give up
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

// What an item of a call with common prefixes (SH) is: a sequence that shares nothing,
// a group's prefix, the rest of one of its sequences.
enum { kWhole = 0, kPrefix = 1, kRest = 2 };
// In row_short.  (kBegun: in an item's first row only; where a wait ran out it stays, or is put back.)
enum { kLong = 0, kDone = 1, kBegun = 2 };
struct SharedSeg : Seg {
  int32_t kind;
  int64_t pages;     // where the item's page ids begin in the table
};
template <bool SH>
using SegOf = std::conditional_t<SH, SharedSeg, Seg>;

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
  SharedSeg* descs;  // [workers] item that starts in a worker and goes on in the next (valid = 0: none)
  int32_t* errs;     // [workers] a wait ran out
  float2* part_ml;   // [workers][2][256] maximum and sum of each row
  float* part_o;     // [workers][2][D / 4][256][4]
  int32_t wait_limit;
  int32_t withhold;  // test switch: the first workers' first loads are not issued
  // Groups with a common prefix:
  int32_t rest_wait_limit, rest_withhold;  // attend_rest_kernel's
  const int32_t* cu_seqs;
  const int32_t* shared_lens;
  int32_t all_groups, groups;  // 0 of them: their prefixes are not taken by themselves
  int32_t prefix_q_rows;  // rows of one query load of a prefix
  int32_t rest_q_rows;    // and of a short rest
  int32_t rest_items;     // items of attend_rest_kernel; 0: it is not used
  int32_t join_shift;     // log2 of attend_join_shared_kernel's tasks for an item
  // Results of rows before they are joined, by key-value head, of the prefix and of the rest.  (Columns in fours outside:
  // the threads of a warp have neighbouring rows.)
  float* row_o;        // [prefix or rest][kv_head][D / 4][row][4]
  float2* row_ml;      // [prefix or rest][kv_head][row] maxima and sums
  int32_t* row_short;  // [kv_head][row] whether what the row's sequence has for itself is attend_rest_kernel's, and there
};

// In errs: the groups do not ascend; rows of some sequence are out of range or descend, and nothing was shared.
constexpr int kMisfit = 2, kAlone = 3;

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
  int32_t kind0;
  int64_t pages0;
  uint32_t bad[3][8];                // tokens whose values are not finite, by segment
  Seg seg[kSegs];
  int32_t seg_kind[kSegs];           // (beside them, for calls with common prefixes)
  int64_t seg_pages[kSegs];
  float2 ml[2][kTile];               // (the prologue's sums before the first segment)
};
template <bool SH>
__device__ __forceinline__ SegOf<SH> read_seg(const Hdr* hdr, int i) {
  SegOf<SH> g;
  static_cast<Seg&>(g) = hdr->seg[i];
  if constexpr (SH) {
    g.kind = hdr->seg_kind[i];
    g.pages = hdr->seg_pages[i];
  }
  return g;
}
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
  bool prefix = false;  // the tokens have no slots of their own among these
  __device__ int items() const { return (n + step - 1) / step; }
  // tiles of item i
  __device__ int tiles(int i) const {
    const int64_t end = prefix ? 0 : causal ? min((int64_t)n, (int64_t)(i + 1) * step) : n;
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
    if (prefix) {  // (any number of tokens)
      const int64_t per = tiles(0) + extra, i = u / per;
      u -= i * per;
      return (int)i;
    }
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

// The group of sequence b among the first `groups`, which ascend, or -1.
__device__ __forceinline__ int group_of(const AttendParams& p, int b, int groups) {
  int lo = -1, hi = groups;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__ldg(p.cu_seqs + mid) <= b)
      lo = mid;
    else
      hi = mid;
  }
  return lo >= 0 && __ldg(p.cu_seqs + lo + 1) > b ? lo : -1;
}
// Slots of group g's prefix: whole pages; 0 where fewer than two sequences share it; -1: out of range.
__device__ __forceinline__ int prefix_of(const AttendParams& p, int g) {
  const int len = __ldg(p.shared_lens + g);
  const int64_t room = (int64_t)p.tok.width * p.kv.page_size;
  if (len < 0 || len > (room < kMaxSlots ? room : kMaxSlots)) return -1;
  return __ldg(p.cu_seqs + g + 1) - __ldg(p.cu_seqs + g) < 2 ? 0 : len & -p.kv.page_size;
}

// What a sequence has for itself is short (attend_rest_kernel) up to so many rows (tokens and heads of a group) and slots.
// Rows: the place that its queries have.  Slots, own ones of each sequence up to 1000, in us, short and long: one token of
// 64 sequences behind 8000 84 and 103, of 24 sequences 55 and 58, 8 tokens of 256 sequences behind 2000 259 and 343; up
// to 1500, long and short: 123 and 100, 66 and 62, 420 and 327; up to 4000: 225 and 191, 100 and 101, 817 and 670.  (So
// the border could lie higher, at 3000 and more where items are many.)
constexpr int kRestRows = 64, kRestSlots = 1024;

// A line of the work: a sequence, or (SH: there are groups with a common prefix) first
// the prefix of each of `groups` groups, then what each sequence has for itself.
struct Span : SeqSpan {
  int32_t kind = kWhole;
  int64_t pages = 0;
};
template <bool SH>
__device__ __forceinline__ void set_line(const AttendParams& p, const Span& s, int extra, Line* l) {
  l->n = s.n;
  l->ctx = s.ctx;
  l->step = 2 * p.tile_tokens;
  l->causal = p.tree == nullptr && !(SH && s.kind == kPrefix);
  l->extra = extra;
  l->prefix = SH && s.kind == kPrefix;
}
// Sequence b without what its group among the first `groups` shares.
__device__ __forceinline__ bool rest_of(const AttendParams& p, int b, Span* s, int groups) {
  bool ok = seq_span(p.tok, p.kv.page_size, b, s) && s->n <= p.max_tokens;
  const int g = group_of(p, b, groups), len = g < 0 ? 0 : prefix_of(p, g);
  ok = ok && len >= 0 && len <= s->ctx;
  s->kind = len > 0 ? kRest : kWhole;
  s->pages = (int64_t)b * p.tok.width + (len >> p.kv.page_shift);
  s->ctx -= len;
  return ok;
}
__device__ __forceinline__ bool rest_of(const AttendParams& p, int b, Span* s) { return rest_of(p, b, s, p.groups); }
__device__ __forceinline__ bool is_short(const AttendParams& p, const Span& s) {
  return p.rest_items > 0 && s.kind == kRest && (int64_t)s.n * p.group <= kRestRows && (int64_t)s.ctx + s.n <= kRestSlots;
}
template <bool SH>
__device__ __forceinline__ bool line_of(const AttendParams& p, int groups, int v, int extra, Span* s, Line* l) {
  if constexpr (SH) {
    bool ok;
    if (v < groups) {
      const int lo = __ldg(p.cu_seqs + v), hi = __ldg(p.cu_seqs + v + 1), len = prefix_of(p, v);
      s->kind = kPrefix;
      ok = len > 0;
      if (ok) {
        s->row0 = __ldg(p.tok.cu + lo);
        const int end = __ldg(p.tok.cu + hi);
        s->n = end - s->row0;
        s->ctx = len;
        s->pages = (int64_t)lo * p.tok.width;
        ok = s->row0 >= 0 && end >= s->row0 && end <= p.tok.n_tokens;
      }
    } else {
      ok = rest_of(p, v - groups, s, groups);
      if (ok && is_short(p, *s)) s->n = s->ctx = 0;  // (attend_rest_kernel's)
    }
    if (!ok) s->n = s->ctx = 0;
    set_line<SH>(p, *s, extra, l);
    return ok;
  }
  const int b = v;
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
template <bool SH, int NW>
__device__ __forceinline__ void row_mask(const AttendParams& p, const SegOf<SH>& g, int tok, int start,
                                         uint32_t (&m)[NW]) {
  int left = g.end - start;  // slots from `start` that any row sees
  if constexpr (SH) {
    if (g.kind == kPrefix) {
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int k = left - 32 * w;
        m[w] = k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u;
      }
      return;
    }
  }
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
template <bool SH>
__device__ __forceinline__ int first_hidden(const AttendParams& p, const SegOf<SH>& g) {
  if constexpr (SH) {
    if (g.kind == kPrefix) return g.end;
  }
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

// A row's places in row_ml (and row_short), and in row_o (columns c .. c + 3).
__device__ __forceinline__ size_t ml_at(const AttendParams& p, int rest, int head, int64_t row) {
  return ((size_t)rest * p.kv.kv_heads + head) * ((size_t)p.tok.n_tokens * p.group) + row;
}
template <int D>
__device__ __forceinline__ float4* o_at(const AttendParams& p, int rest, int head, int64_t row, int c) {
  return reinterpret_cast<float4*>(p.row_o) +
         (((size_t)rest * p.kv.kv_heads + head) * (D / 4) + c / 4) * ((size_t)p.tok.n_tokens * p.group) + row;
}

// Two results over different slots as one: factors of their values, and its maximum and sum.
struct Pair {
  float e, f, m, l;
};
__device__ __forceinline__ Pair join(float2 x, float2 y, float c) {
  Pair r;
  r.m = fmaxf(x.x, y.x);
  r.e = r.m == -INFINITY ? 0.f : ex2((x.x - r.m) * c);
  r.f = r.m == -INFINITY ? 0.f : ex2((y.x - r.m) * c);
  r.l = fmaf(x.y, r.e, y.y * r.f);
  return r;
}

// Logarithm of a row's sum of exponentials.
template <typename T>
__device__ __forceinline__ float log_sum(float m, float l, float c) {
  return l == 0.f ? -INFINITY : (m * c + (log2f(l) - T::kShift)) * kLn2;
}

// The page ids of an item.
template <bool SH>
__device__ __forceinline__ const int32_t* page_row(const AttendParams& p, const SegOf<SH>& g) {
  if constexpr (SH)
    return p.tok.table + g.pages;
  else
    return p.tok.table + (int64_t)g.seq * p.tok.width;
}

// Adds to 32 columns of a row the infinities and NaN that were taken out of the
// values of slots it sees (from the cache itself; rare).
template <typename T, int D, bool SH>
__device__ __forceinline__ void add_taken_out(const AttendParams& p, const SegOf<SH>& g, const uint32_t* bad, int hidden,
                                           int tok, int c, float (&v)[32]) {
#pragma unroll 1
  for (int i = 0; i < 8; ++i)
#pragma unroll 1
    for (uint32_t w = bad[i]; w; w &= w - 1) {
      const int slot = hidden + i * 32 + __ffs(w) - 1;
      uint32_t mask[1];
      row_mask<SH, 1>(p, g, tok, slot, mask);
      if (!(mask[0] & 1u)) continue;
      const int page = __ldg(page_row<SH>(p, g) + (slot >> p.kv.page_shift));
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

template <typename T, int D, bool SH>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const AttendParams p, const __grid_constant__ CUtensorMap map_kv,
                  const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_pq) {
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
  __syncwarp();
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&hdr->tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // The setup above touches only this CTA; everything read or written from
  // here on may belong to the kernel before.  (With attend_rest_kernel in front, which
  // lets this one begin when it has waited itself, that kernel's results are the only
  // ones that are not there yet: they are waited for where they are joined.  64 tokens
  // behind 8003 slots 52 us instead of 57, drafts of 256 sequences 198 instead of 212.)
  if (!SH || p.rest_items == 0) asm volatile("griddepcontrol.wait;" ::: "memory");

  // Tiles and items of every sequence: thread i counts a run of them, then a
  // scan over the CTA gives the totals and who holds this worker's first unit.
  bool fits = true;
  int groups = p.groups;  // (SH)
  if constexpr (SH) {
    // Groups that do not ascend: no work, and an error of every sequence.  (Short code: with these loops unrolled a call
    // takes 0.3 us longer.)
#pragma unroll 1
    for (int g = tid; g < p.all_groups; g += kThreads) {
      const int lo = __ldg(p.cu_seqs + g), hi = __ldg(p.cu_seqs + g + 1);
      fits &= lo >= 0 && hi >= lo && hi <= p.tok.batch;
    }
    // The rows of a group are those from its first sequence's to its last one's, and each of them is one sequence's, only
    // where all sequences' rows ascend.  Else every sequence is read by itself: those whose rows are in range are right.
    bool ascend = true;
#pragma unroll 1
    for (int b = tid; groups > 0 && b < p.tok.batch; b += kThreads) {
      const int lo = __ldg(p.tok.cu + b), hi = __ldg(p.tok.cu + b + 1);
      ascend &= lo >= 0 && hi >= lo && hi <= p.tok.n_tokens;
    }
    if (!__syncthreads_and(fits && ascend)) {
      fits = __syncthreads_and(fits);
      if (!__syncthreads_and(ascend)) groups = 0;
    }
  }
  const int n_lines = (SH ? groups : 0) + p.tok.batch, run = (n_lines + kThreads - 1) / kThreads;
  int64_t* sums = reinterpret_cast<int64_t*>(hdr->ml);
  int64_t tiles = 0, items = 0;
  for (int i = 0; i < run; ++i) {
    const int b = tid * run + i;
    Span s;
    Line l;
    if (b < n_lines && fits && line_of<SH>(p, groups, b, 0, &s, &l) && s.n > 0) {
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
      Span s;
      Line l;
      if (b >= n_lines || !line_of<SH>(p, groups, b, extra, &s, &l)) continue;
      const int64_t u = l.units() * p.kv.kv_heads;
      if (begin < at + u) {
        hdr->seq0 = b;
        hdr->row0 = s.row0;
        hdr->n0 = s.n;
        hdr->ctx0 = s.ctx;
        hdr->off0 = begin - at;
        if (SH) {
          hdr->kind0 = s.kind;
          hdr->pages0 = s.pages;
        }
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
      const SegOf<SH> g = read_seg<SH>(hdr, k % kSegs);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&hdr->seg_empty[k % kSegs]));
      if (!g.valid) break;
      const int32_t* row = page_row<SH>(p, g);
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
        const SegOf<SH> g = read_seg<SH>(hdr, k % kSegs);
        mbar_arrive(smem_u32(&hdr->seg_empty[k % kSegs]));
        if (!g.valid) break;
        for (int m = 0; m <= g.two; ++m, ++armed) {
          if (!mbar_wait(smem_u32(&hdr->q_empty[armed & 1]), ((armed >> 1) & 1) ^ 1, wl, abort)) {
            stop = true;
            break;
          }
          const uint32_t bar = smem_u32(&hdr->q_full[armed & 3]);
          bool of_prefix = false;
          if constexpr (SH) of_prefix = g.kind == kPrefix;
          mbar_expect_tx(bar, (uint32_t)(of_prefix ? p.prefix_q_rows : p.q_rows) * 128u * C::kHalves);
          for (int h = 0; h < C::kHalves; ++h)
            tma_q(q_s + (armed & 1) * C::kTileBytes + h * kHalfBytes, of_prefix ? &map_pq : &map_q, h * 64,
                  g.head * p.group,
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
        const SegOf<SH> g = read_seg<SH>(hdr, k % kSegs);
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
      SegOf<SH> d{};
      while (ok) {
        SegOf<SH> g{};
        if (left > 0) {
          Span s;
          s.row0 = hdr->row0;
          s.n = hdr->n0;
          s.ctx = hdr->ctx0;
          if (SH) {
            s.kind = hdr->kind0;
            s.pages = hdr->pages0;
          }
          Line l;
          set_line<SH>(p, s, extra, &l);
          int64_t per = 0;
          if (b == hdr->seq0) {
            per = l.units();
          } else {
            // (sequences without units are passed over)
            while (b < n_lines && !(line_of<SH>(p, groups, b, extra, &s, &l) && (per = l.units()) > 0)) ++b;
            if (b >= n_lines) break;  // (cannot be: the units add up)
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
              g.end = s.ctx + (l.prefix ? 0 : p.tree ? s.n : min(s.n, g.tok0 + l.step));
              if constexpr (SH) {
                g.kind = s.kind;
                g.pages = s.pages;
              }
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
              if constexpr (SH) {
                hdr->seg_kind[k % kSegs] = g.kind;
                hdr->seg_pages[k % kSegs] = g.pages;
              }
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
      static_cast<SegOf<SH>&>(p.descs[worker]) = d;
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
      const SegOf<SH> g = read_seg<SH>(hdr, k % kSegs);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&hdr->seg_empty[k % kSegs]));
      if (!g.valid) break;
      const int n = g.t1 - g.t0;
      const int tok = g.tok0 + (g.two ? grp * p.tile_tokens : 0) + r / p.group;
      const bool live = r < p.tile_tokens * p.group && tok < g.n;
      const bool any = __any_sync(0xffffffffu, live);
      const int hidden = first_hidden<SH>(p, g);
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
          m = grow ? top : m;
          off = grow ? T::kShift - m * p.c : off;
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
          if (live) row_mask<SH, W / 32>(p, g, tok, start, mask);
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
      bool joined = false;  // (a result to be joined with another's later)
      const int64_t row = SH ? (int64_t)(g.row0 + tok) * p.group + r % p.group : 0;
      int kind = kWhole;
      Pair pair;
      bool with_rest = false;
      if constexpr (SH) {
        kind = g.kind;
        joined = kind != kWhole;
        if (kind == kPrefix && g.part < 0 && any) {
          // What the row's sequence has for itself is there, if it is short: joined here.
          asm volatile("griddepcontrol.wait;" ::: "memory");
          if (live) {
            const float2 y = __ldcg(p.row_ml + ml_at(p, 1, g.head, row));
            if (p.rest_items > 0 && __ldcg(p.row_short + ml_at(p, 0, g.head, row)) == kDone) {
              pair = join(make_float2(m, l), y, p.c);
              m = pair.m;
              l = pair.l;
              with_rest = true;
              joined = false;
            }
          }
        }
      }
      const float norm = g.part >= 0 || joined ? 1.f : l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // (NaN stays)
      const int rr = (g.two ? grp * kTile : 0) + r;
      const size_t part = ((size_t)worker * 2 + (g.part > 0)) * 2 * kTile;
      // Columns: all of the group's own accumulator, or half of both.
      const int c_lo = g.two ? 0 : grp * (D / 2), c_hi = g.two ? D : c_lo + D / 2;
      if (any) {
#pragma unroll 1
        for (int c = c_lo; c < c_hi; c += 32) {
          uint32_t o[32], o1[32];
          __syncwarp();  // (rows without work, or with other results to join, went other ways)
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
          if (live && any_bad) add_taken_out<T, D, SH>(p, g, bad, hidden, tok, c, v);
          if constexpr (SH) {
            if (with_rest) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float4 y = __ldcg(o_at<D>(p, 1, g.head, row, c + 4 * j));
                v[4 * j] = fmaf(v[4 * j], pair.e, y.x * pair.f);
                v[4 * j + 1] = fmaf(v[4 * j + 1], pair.e, y.y * pair.f);
                v[4 * j + 2] = fmaf(v[4 * j + 2], pair.e, y.z * pair.f);
                v[4 * j + 3] = fmaf(v[4 * j + 3], pair.e, y.w * pair.f);
              }
            }
          }
          if (joined && live && g.part < 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *o_at<D>(p, kind == kRest, g.head, row, c + 4 * j) =
                  make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          } else if (live && g.part < 0) {
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
        else if (joined)
          p.row_ml[ml_at(p, kind == kRest, g.head, row)] = make_float2(m, l);
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
    const int wl = max(p.wait_limit, kWaitLimit);
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
  if constexpr (SH) asm volatile("griddepcontrol.wait;" ::: "memory");  // (the next kernel waits for this one only)
  if (tid == 0) p.errs[worker] = hdr->abort ? 1 : !fits ? kMisfit : SH && groups != p.groups ? kAlone : 0;
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// --------------------------------------------- short rests behind a prefix
//
// What a sequence has for itself behind a shared prefix is mostly one token or a
// draft over a few hundred slots.  Through the kernel above each of them has a
// whole SM, and 6 us, for itself.  Here two CTAs share an SM and go through items (a
// sequence and a key-value head, up to 64 rows) one after another, six warps each:
//  - warp 0 takes items (the next one is that of a CTA of the grid which has not
//    begun: it is called off, so that long and short items even out), looks their
//    pages up and loads queries, keys and values of 64 slots by TMA, ahead of the
//    others over the ends of items;
//  - warp 1 issues the products: S = Q K^T of the next tile beside the softmax of
//    this one, then O += P V;
//  - warps 2 to 5 have a row per thread, as in the kernel above, with the same lazy
//    maximum, masks and treatment of infinities and NaN in drafted values.
// Results are left in 32 bits, to be joined with the prefix's.
//
// What it measured (32 query and 8 key-value heads of 128): one token of 64 sequences
// with 20 to 300 slots 20 us; 3 to 16 tokens of 256 sequences with 50 to 500 slots 72 us,
// 4.4 TB/s.  Calls as a whole, behind 8003 and 1001 to 4001 shared slots: 49 and 196 us,
// with these items in the kernel above 59 and 278.  Bound: latencies where items begin
// and end.  (A form of it with the matrix instructions of single warps, mma.sync,
// three CTAs an SM, took 104 us for the drafts.)

constexpr int kRestThreads = 192, kRestTile = 64, kRestPerSm = 2, kUnits = 4;
constexpr int kRestAhead = 8;   // items that have been told of
constexpr int kRestHeld = 4;    // those that some warp may not have finished: the loader is at most three ahead of it

struct RestItem {
  int64_t pages;  // where its page ids begin in the table
  int32_t valid, row0, n, ctx, head;
};
struct alignas(16) RestHdr {
  uint32_t answer[4];                       // which CTA was called off
  uint64_t full[kUnits], empty[kUnits];     // keys or values of a tile
  uint64_t q_full[2], q_empty[2];
  uint64_t item_full[kRestAhead];
  uint64_t answer_full;
  uint64_t s_full, s_read, p_ready, pv_done, o_free, meet, drain;
  uint32_t tmem_base;
  int32_t abort;
  uint32_t bad[3][2];                       // drafted tokens with values that are not finite, by item
  RestItem item[kRestAhead];
};
template <int D>
struct RestCfg {
  static constexpr uint32_t kHalf = kRestTile * 128, kHalves = D / 64;
  static constexpr uint32_t kUnit = kHalves * kHalf;   // queries of 64 rows, keys or values of 64 slots
  // Tensor memory: scores, weights, accumulator.
  static constexpr uint32_t kCols = 256, kP = 64, kO = 128;
  // (a product reads 128 rows of queries: what lies behind their place, units of keys and values, makes rows that
  // nothing reads)
  static constexpr size_t kSmem = (2 + kUnits) * (size_t)kUnit + sizeof(RestHdr);
  static_assert(kRestPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

// Calls off a CTA of the grid that has not begun; 16 bytes at `to` will tell which.
__device__ __forceinline__ void call_off(uint32_t to, uint32_t bar) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the answer before has been read)
  mbar_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(to),
               "r"(bar)
               : "memory");
}
// Its number, or -1 if there was none.
__device__ __forceinline__ int called_off(uint32_t at) {
  int x;
  asm volatile(
      "{\n .reg .b128 a;\n .reg .pred p;\n .reg .b32 y, z;\n ld.shared.b128 a, [%1];\n mov.b32 %0, -1;\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, _}, a;\n}\n"
      : "=r"(x)
      : "r"(at)
      : "memory");
  return x;
}

// The call's tokens of a sequence (64 at most) that one of them sees.
__device__ __forceinline__ unsigned long long tokens_seen(const AttendParams& p, int row0, int n, int tok) {
  const unsigned long long m =
      p.tree ? (unsigned long long)__ldg(p.tree + (int64_t)(row0 + tok) * p.words) : (2ull << tok) - 1ull;
  return n < 64 ? m & ((1ull << n) - 1ull) : m;
}

template <typename T, int D>
__global__ void __launch_bounds__(kRestThreads, kRestPerSm)
    attend_rest_kernel(const AttendParams p, const __grid_constant__ CUtensorMap map_kv,
                       const __grid_constant__ CUtensorMap map_q) {
  using C = RestCfg<D>;
  extern __shared__ __align__(1024) unsigned char rest_smem[];
  RestHdr* hdr = reinterpret_cast<RestHdr*>(rest_smem + (2 + kUnits) * (size_t)C::kUnit);
  const uint32_t q_s = smem_u32(rest_smem), kv_s = q_s + 2 * C::kUnit;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int32_t* abort = &hdr->abort;
  const int wl = p.rest_wait_limit;
  if (tid == 0) {
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(smem_u32(&hdr->full[i]), 1);
      mbar_init(smem_u32(&hdr->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&hdr->q_full[i]), 1);
      mbar_init(smem_u32(&hdr->q_empty[i]), 1);
    }
    for (int i = 0; i < 3; ++i) hdr->bad[i][0] = hdr->bad[i][1] = 0u;
    for (int i = 0; i < kRestAhead; ++i) mbar_init(smem_u32(&hdr->item_full[i]), 1);
    mbar_init(smem_u32(&hdr->answer_full), 1);
    mbar_init(smem_u32(&hdr->s_full), 1);
    mbar_init(smem_u32(&hdr->s_read), kTile);
    mbar_init(smem_u32(&hdr->p_ready), kTile);
    mbar_init(smem_u32(&hdr->pv_done), 1);
    mbar_init(smem_u32(&hdr->o_free), kTile);
    mbar_init(smem_u32(&hdr->meet), kTile);
    mbar_init(smem_u32(&hdr->drain), 1);
    // (the swizzle wants tiles on 1024-byte boundaries; dynamic shared memory begins on one)
    hdr->abort = (q_s & 1023u) != 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_kv)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_q)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&hdr->tmem_base)),
                 "r"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = hdr->tmem_base;
  // (after the wait: what was there for this kernel is there for the next one, which does not wait itself)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const bool held = p.rest_withhold == 1 && blockIdx.x == 0, sound = hdr->abort == 0;
  __syncthreads();

  // Whether an item is a short rest; row_short is told of it, for all of its rows if it is a long one.
  const auto take = [&](int item, Span* s) {
    const int head = item % p.kv.kv_heads;
    if (!rest_of(p, item / p.kv.kv_heads, s) || s->kind != kRest || s->n == 0) return false;
    const bool found = is_short(p, *s);
    const int64_t row = (int64_t)s->row0 * p.group;
    for (int64_t r = lane; !found && r < (int64_t)s->n * p.group; r += 32)
      p.row_short[ml_at(p, 0, head, row + r)] = kLong;
    if (found && lane == 0) p.row_short[ml_at(p, 0, head, row)] = kBegun;
    return found;
  };
  // The loader's next item (-1: none is left), calls, tiles, keys and values of tiles, and items.
  int i = blockIdx.x, asked = 1, armed = 0, sent = 0, k_sent = 0;
  if (!sound) {
  } else if (warp == 0) {
    // ------------------------------------------------------------ loader
    const int box = min(p.kv.page_size, kRestTile), pieces = kRestTile / box;
    const int half = lane % C::kHalves, is_v = lane / C::kHalves & 1, piece = lane / (2 * C::kHalves);
    const uint32_t dst = kv_s + is_v * C::kUnit + half * C::kHalf + piece * box * 128;
    bool stop = false;
    if (lane == 0) call_off(smem_u32(hdr->answer), smem_u32(&hdr->answer_full));
    while (!stop) {
      // the next short item
      Span s;
      bool found = false;
      int head = 0;
      while (i >= 0 && !found) {
        head = i % p.kv.kv_heads;
        found = take(i, &s);
        if (!warp_wait(smem_u32(&hdr->answer_full), (asked - 1) & 1, wl, abort)) {
          stop = true;
          break;
        }
        i = called_off(smem_u32(hdr->answer));
        __syncwarp();
        if (i >= 0) {
          ++asked;
          if (lane == 0) call_off(smem_u32(hdr->answer), smem_u32(&hdr->answer_full));
        }
      }
      // (the place of the queries: those of the item before the last have been used)
      if (found && !warp_wait(smem_u32(&hdr->q_empty[k_sent & 1]), ((k_sent >> 1) & 1) ^ 1, wl, abort)) stop = true;
      if (stop) break;
      if (lane == 0) {
        hdr->item[k_sent % kRestAhead] = RestItem{s.pages, found, s.row0, s.n, s.ctx, head};
        mbar_arrive(smem_u32(&hdr->item_full[k_sent % kRestAhead]));
      }
      __syncwarp();
      if (!found) break;
      if (lane == 0) {
        const uint32_t bar = smem_u32(&hdr->q_full[k_sent & 1]);
        mbar_expect_tx(bar, (uint32_t)p.rest_q_rows * 128u * C::kHalves);
        for (int h = 0; h < (int)C::kHalves; ++h)
          tma_q(q_s + (k_sent & 1) * C::kUnit + h * C::kHalf, &map_q, h * 64, head * p.group, s.row0, bar);
      }
      __syncwarp();
      ++k_sent;
      const int end = s.ctx + s.n, tiles = (end + kRestTile - 1) / kRestTile;
      const int32_t* table = p.tok.table + s.pages;
      int slot = piece * box;
      bool load = piece < pieces && slot < end;
      int page = load ? __ldg(table + (slot >> p.kv.page_shift)) : 0;
      for (int t = 0; t < tiles; ++t, ++armed) {
        // (the next tile's pages are looked up before this one's places are waited for)
        const int slot2 = slot + kRestTile;
        const bool load2 = piece < pieces && slot2 < end;
        const int page2 = load2 ? __ldg(table + (slot2 >> p.kv.page_shift)) : 0;
        const uint32_t count = __popc(__ballot_sync(0xffffffffu, load && is_v == 0));
        const int u = 2 * (armed & 1);
        for (int v = 0; v < 2 && !stop; ++v) {
          if (armed > 1 && !warp_wait(smem_u32(&hdr->empty[u + v]), ((armed >> 1) - 1) & 1, wl, abort)) {
            stop = true;
            break;
          }
          const uint32_t bar = smem_u32(&hdr->full[u + v]);
          const bool leave = held && armed == 0 && v == 0;
          if (lane == 0 && !leave) mbar_expect_tx(bar, count * box * 128);
          __syncwarp();
          if (load && is_v == v && !leave)
            tma_kv(dst + u * C::kUnit, &map_kv, slot & (p.kv.page_size - 1), half, v * p.kv.kv_heads + head, page, bar);
          ++sent;
        }
        if (stop) break;
        slot = slot2;
        load = load2;
        page = page2;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ issuer
    if (lane == 0) {
      const uint32_t id_s = idesc<T>(kRestTile, false, p.negate != 0);
      constexpr uint32_t id_o = idesc<T>(D, true);
      int done = 0;    // tiles
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) {
        ok = ok && mbar_wait(smem_u32(bar), parity & 1, wl, abort);
        return ok;
      };
      for (int k = 0; ok; ++k) {
        if (!wait(&hdr->item_full[k % kRestAhead], k / kRestAhead)) break;
        const RestItem s = hdr->item[k % kRestAhead];
        if (!s.valid) break;
        const int end = s.ctx + s.n, tiles = (end + kRestTile - 1) / kRestTile;
        const uint64_t q = desc_k_major(q_s + (k & 1) * C::kUnit);
        if (!wait(&hdr->q_full[k & 1], k >> 1)) break;
        const auto scores = [&](int t) {   // of tile t, when the scores before have been read
          const int x = done + t, u = 2 * (x & 1);
          if (!wait(&hdr->full[u], x >> 1) || (x > 0 && !wait(&hdr->s_read, x - 1))) return;
          tc_fence_after();
          const uint64_t b = desc_k_major(kv_s + u * C::kUnit);
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const uint32_t o = (uint32_t)(e & 3) * 2 + (uint32_t)(e >> 2) * (C::kHalf >> 4);
            mma_ss(tmem, q + o, b + o, id_s, e > 0);
          }
          mma_commit(smem_u32(&hdr->s_full));
          mma_commit(smem_u32(&hdr->empty[u]));
          if (t + 1 == tiles) mma_commit(smem_u32(&hdr->q_empty[k & 1]));
        };
        scores(0);
        for (int t = 0; t < tiles && ok; ++t) {
          if (t + 1 < tiles) scores(t + 1);
          const int x = done + t, u = 2 * (x & 1) + 1;
          // (the accumulator of the item before has been read)
          if (t == 0 && k > 0 && !wait(&hdr->o_free, k - 1)) break;
          if (!wait(&hdr->p_ready, x) || !wait(&hdr->full[u], x >> 1)) break;
          tc_fence_after();
          // Values: rows of 64 columns, groups of 8 slots 1024 bytes apart, blocks of 64 columns C::kHalf apart.
          const uint32_t at = kv_s + u * C::kUnit;
          const uint64_t b = (uint64_t)((at & 0x3FFFFu) >> 4) | (uint64_t)(C::kHalf >> 4) << 16 |
                             (uint64_t)(1024u >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
          const int groups = (min(kRestTile, end - t * kRestTile) + 15) / 16;
#pragma unroll
          for (int e = 0; e < kRestTile / 16; ++e)
            if (e < groups) mma_ts(tmem + C::kO, tmem + C::kP + e * 8, b + e * (2048 >> 4), id_o, t > 0 || e > 0);
          mma_commit(smem_u32(&hdr->pv_done));
          mma_commit(smem_u32(&hdr->empty[u]));
        }
        done += tiles;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ rows
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t t_s = tmem + ((uint32_t)(quarter * 32) << 16), t_p = t_s + C::kP, t_o = t_s + C::kO;
    const uint64_t c2 = f2(p.c, p.c);
    int n_s = 0;
    for (int k = 0;; ++k) {
      if (!warp_wait(smem_u32(&hdr->item_full[k % kRestAhead]), (k / kRestAhead) & 1, wl, abort)) break;
      const RestItem s = hdr->item[k % kRestAhead];
      if (!s.valid) break;
      const int rows = s.n * p.group, end = s.ctx + s.n, tiles = (end + kRestTile - 1) / kRestTile;
      const bool live = r < rows, any = quarter * 32 < rows;
      const int tok = r / p.group;
      const unsigned long long seen = live ? tokens_seen(p, s.row0, s.n, tok) : 0ull;
      uint32_t* bad = hdr->bad[k % 3];
      float m = -INFINITY, l = 0.f, off = 0.f;
      bool stop = false;
#pragma unroll 1
      for (int t = 0; t < tiles; ++t, ++n_s) {
        const int start = t * kRestTile;
        const bool tail = start + kRestTile > s.ctx;       // drafted tokens among the slots, or the end
        if (!warp_wait(smem_u32(&hdr->s_full), n_s & 1, wl, abort)) {
          stop = true;
          break;
        }
        bool ok = true;
        if (any) {
          tc_fence_after();
          uint32_t w[kRestTile];
          tmem_ld32(t_s, w);
          tmem_ld32(t_s + 32, w + 32);
          tmem_ld_wait();
          tmem_arrived(w);
          tmem_arrived(w + 32);
          tc_fence_before();
          mbar_arrive(smem_u32(&hdr->s_read));
          if (tail) {
            const int x0 = start - s.ctx;                  // the tile's first slot as a drafted token, above -64
            const unsigned long long v = x0 >= 0 ? (x0 < 64 ? seen >> x0 : 0ull)
                                                 : live ? seen << -x0 | ((1ull << -x0) - 1ull) : 0ull;
            const uint32_t word[2] = {(uint32_t)v, (uint32_t)(v >> 32)};
#pragma unroll
            for (int j = 0; j < kRestTile; ++j) w[j] = word[j >> 5] & (1u << (j & 31)) ? w[j] : 0xff800000u;
          }
          float mx[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) mx[j] = __uint_as_float(w[j]);
#pragma unroll
          for (int j = 4; j < kRestTile; j += 2)
            mx[(j >> 1) & 3] = max3(mx[(j >> 1) & 3], __uint_as_float(w[j]), __uint_as_float(w[j + 1]));
          const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
          // (the product before is done: the weights' place is free, the accumulator at rest)
          ok = t == 0 || mbar_wait(smem_u32(&hdr->pv_done), (n_s - 1) & 1, wl, abort);
          __syncwarp();
          tc_fence_after();
          const bool grow = (top - m) * p.c > kRescale;
          if (__any_sync(0xffffffffu, grow)) {
            if (t > 0) {
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
            m = grow ? top : m;
            off = grow ? T::kShift - m * p.c : off;
          }
          const uint64_t off2 = f2(off, off);
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 x =
                  unf2(fma2(f2(__uint_as_float(w[q * 32 + 2 * j]), __uint_as_float(w[q * 32 + 2 * j + 1])), c2, off2));
              const float a = ex2(x.x), b = ex2(x.y);
              sum[j & 1] = add2(sum[j & 1], f2(a, b));
              pk[j] = T::pack(a, b);
            }
            tmem_st16(t_p + q * 16, pk);
          }
          const float2 y = unf2(add2(sum[0], sum[1]));
          l += y.x + y.y;
          tmem_st_wait();
        } else {
          mbar_arrive(smem_u32(&hdr->s_read));
          // (or this warp would announce weights before others have announced those before)
          ok = t == 0 || mbar_wait(smem_u32(&hdr->pv_done), (n_s - 1) & 1, wl, abort);
        }
        if (!__all_sync(0xffffffffu, ok)) {
          stop = true;
          break;
        }
        if (tail) {
          // Values of slots that some row must not see: zero past the end (as far as products read), infinities and NaN
          // of drafted tokens out (kept in `bad`).  Two threads a slot.
          const int u = 2 * (n_s & 1) + 1;
          if (!warp_wait(smem_u32(&hdr->full[u]), (n_s >> 1) & 1, wl, abort)) {
            stop = true;
            break;
          }
          const int j = r >> 1, slot = start + j, slots = min(kRestTile, end - start);
          const uint32_t row = kv_s + u * C::kUnit + j * 128;
          if (slot >= end) {
            if (j < ((slots + 15) & ~15))
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                const int x = (r & 1) * (D / 16) + c;
                sts128(row + (x >> 3) * C::kHalf + (((x ^ j) & 7) << 4), make_uint4(0u, 0u, 0u, 0u));
              }
          } else if (slot >= s.ctx) {
            bool odd = false;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              const int x = (r & 1) * (D / 16) + c;
              const uint32_t at = row + (x >> 3) * C::kHalf + (((x ^ j) & 7) << 4);
              const uint4 v = lds128(at);
              if (T::trace(v.w, T::trace(v.z, T::trace(v.y, T::trace(v.x, 0u)))) & 0x7fff7fffu) {
                odd = true;
                sts128(at, make_uint4(only_finite<T>(v.x), only_finite<T>(v.y), only_finite<T>(v.z),
                                      only_finite<T>(v.w)));
              }
            }
            if (odd) atomicOr(&bad[(slot - s.ctx) >> 5], 1u << ((slot - s.ctx) & 31));
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&hdr->p_ready));
      }
      if (stop) break;
      // All have noted what they found, and the last product is done.
      if (r == 0) hdr->bad[(k + 1) % 3][0] = hdr->bad[(k + 1) % 3][1] = 0u;  // (last read before all met an item ago)
      mbar_arrive(smem_u32(&hdr->meet));
      if (!warp_wait(smem_u32(&hdr->meet), k & 1, wl, abort) ||
          !warp_wait(smem_u32(&hdr->pv_done), (n_s - 1) & 1, wl, abort))
        break;
      if (p.rest_withhold > 1 && blockIdx.x == 0 && quarter == 1) {  // (test switch: as if that wait had run out here)
        *abort = 1;
        break;
      }
      tc_fence_after();
      const unsigned long long lost = ((unsigned long long)bad[1] << 32 | bad[0]) & seen;
      const int64_t row = (int64_t)s.row0 * p.group + r;
      if (any) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          __syncwarp();  // (rows of no token, or with values that were taken out, went other ways)
          tmem_ld32(t_o + c, o);
          tmem_ld_wait();
          tmem_arrived(o);
          if (!live) continue;
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(o[j]);
          // the infinities and NaN that were taken out (from the cache itself; rare)
#pragma unroll 1
          for (unsigned long long x = lost; x; x &= x - 1) {
            const int slot = s.ctx + __ffsll(x) - 1;
            const int page = __ldg(p.tok.table + s.pages + (slot >> p.kv.page_shift));
            const uint32_t* src = reinterpret_cast<const uint32_t*>(
                p.kv.base + ((((int64_t)page * 2 + 1) * p.kv.kv_heads + s.head) * p.kv.page_size +
                             (slot & (p.kv.page_size - 1))) * D * 2 + c * 2);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 y = non_finite<T>(__ldg(src + j));
              v[2 * j] += y.x;
              v[2 * j + 1] += y.y;
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *o_at<D>(p, 1, s.head, row, c + 4 * j) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
        if (live) {
          p.row_ml[ml_at(p, 1, s.head, row)] = make_float2(m, l);
          p.row_short[ml_at(p, 0, s.head, row)] = kDone;
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&hdr->o_free));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort) {
    // A wait ran out.  What this CTA started has to end before it leaves (waits bounded again).  Items that it was to
    // take are begun by no other: short ones will not be done, long ones are others' work all the same.  Those in hand may
    // have been finished by some warps and not by others: the first row says of each that it has been begun, no more.
    const int wl = max(p.rest_wait_limit, kWaitLimit);
    int32_t none = 0;
    if (warp == 1 && lane == 0 && sound) {
      mma_commit(smem_u32(&hdr->drain));
      mbar_wait(smem_u32(&hdr->drain), 0u, wl, &none);
    }
    if (warp == 0) {
      bool answered = false;
      if (sound) {
        for (int j = max(0, sent - kUnits); j < sent; ++j)
          if (!(held && j == 0)) mbar_wait(smem_u32(&hdr->full[j % kUnits]), (j / kUnits) & 1, wl, &none);
        for (int j = max(0, k_sent - 2); j < k_sent; ++j)
          mbar_wait(smem_u32(&hdr->q_full[j & 1]), (j >> 1) & 1, wl, &none);
        answered = mbar_wait(smem_u32(&hdr->answer_full), (asked - 1) & 1, wl, &none);
      }
      for (int x = 0; x < 2; ++x) {
        const int j = x == 0 ? i : answered && i >= 0 ? called_off(smem_u32(hdr->answer)) : -1;
        Span s;
        if (j >= 0) take(j, &s);
      }
      for (int k = max(0, k_sent - kRestHeld); k < k_sent; ++k) {
        const RestItem& s = hdr->item[k % kRestAhead];
        if (lane == 0) p.row_short[ml_at(p, 0, s.head, (int64_t)s.row0 * p.group)] = kBegun;
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
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

// The same for calls with common prefixes.  Few items may hold all rows (a long prefix with a part in every worker), or
// every worker may start one: the blocks share out the tasks of all of them.  A prefix's row takes what its sequence
// has for itself with it, if that is there.  Bound: latencies, among them the fetch of instructions, so the code is short
// (eight parts at a time, unrolled: 64 tokens behind 8003 slots 16.4 us instead of 11.4; blocks for each worker, as
// above, take 13).
//
// WAYS: 2 where prefixes are so few that their tasks leave half of the blocks idle: two threads share out a row's parts,
// the first half of them and the second, in that order (64 tokens behind 8003 slots, the whole call 49.2 us instead of
// 52.0, 8 tokens 31.7 and 33.9; for drafts of 256 sequences, 206 instead of 197, each task would cost more and none is
// idle.  Four threads: 51.2 and 228).  The host chooses: the kernel itself takes 2 us longer with both ways in it.
constexpr int kJoinSharedBlocks = 4;  // for each worker, at most
template <typename T, int D, int WAYS>
__global__ void __launch_bounds__(kJoinThreads) attend_join_shared_kernel(const AttendParams p) {
  constexpr int kTask = kJoinThreads / WAYS;  // pieces of four columns
  __shared__ uint32_t starts[32];
  __shared__ float4 other_o[WAYS > 1 ? kTask : 1];
  __shared__ float2 other_ml[WAYS > 1 ? kTask : 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int blocks = gridDim.x - p.tok.batch;
  if (blockIdx.x >= (unsigned)blocks) {
    const int b = blockIdx.x - blocks;
    Span s;
    bool late = false, fits = true;
    const bool shares = __ldcg(p.errs) != kAlone;  // (all workers find the same)
    for (int i = threadIdx.x; i < p.workers; i += kJoinThreads) {
      const int e = __ldcg(p.errs + i);
      late |= e == 1;
      fits &= e != kMisfit;
    }
    // (that it fits its group as well, whether or not the group's prefix was taken by itself)
    bool ok = __syncthreads_and(fits) && rest_of(p, b, &s, p.all_groups);
    if (ok && s.n > 0) {
      const int32_t* row = p.tok.table + (int64_t)b * p.tok.width;
      const int shared = (int)((s.pages - (int64_t)b * p.tok.width));  // pages
      const int pages = shared + (s.ctx + s.n - 1) / p.kv.page_size + 1;
      const int32_t* first = shared ? p.tok.table + (int64_t)__ldg(p.cu_seqs + group_of(p, b, p.all_groups)) * p.tok.width : row;
      if (shares && is_short(p, s))
        for (int i = threadIdx.x; i < p.kv.kv_heads; i += kJoinThreads)
          late |= __ldcg(p.row_short + ml_at(p, 0, i, (int64_t)s.row0 * p.group)) == kBegun;
      // the prefix lies in the same pages as the group's first sequence's
      for (int i = threadIdx.x; i < pages; i += kJoinThreads) {
        const int page = __ldg(row + i);
        ok &= (uint32_t)page < (uint32_t)p.kv.pages && (i >= shared || page == __ldg(first + i));
      }
    }
    ok = __syncthreads_and(ok);
    late = __syncthreads_or(late);
    if (threadIdx.x == 0)
      set_status(p.status, b, late ? TC_ERR_DEVICE_TIMEOUT : ok ? TC_OK : TC_ERR_BOUNDS, p.kv.keep);
    return;
  }
  if (threadIdx.x < 32) starts[threadIdx.x] = 0u;
  __syncthreads();
  for (int w = threadIdx.x; w / 32 * 32 < p.workers; w += kJoinThreads) {
    const uint32_t m = __ballot_sync(0xffffffffu, w < p.workers && __ldcg(&p.descs[w].valid) != 0);
    if (w % 32 == 0) starts[w / 32] = m;
  }
  __syncthreads();
  const bool second = WAYS > 1 && threadIdx.x >= kTask;
  int before = 0, word = 0;
  for (int slot = blockIdx.x;; slot += blocks) {
    const int item = slot >> p.join_shift, piece0 = (slot & ((1 << p.join_shift) - 1)) * kTask;
    // the item-th worker that starts one
    while (word < 32 && item - before >= __popc(starts[word])) before += __popc(starts[word++]);
    if (word == 32) break;
    uint32_t bits = starts[word];
    for (int i = before; i < item; ++i) bits &= bits - 1;
    const int w0 = word * 32 + __ffs(bits) - 1;
    const SharedSeg g = p.descs[w0];
    const int full = p.tile_tokens * p.group, left = (g.n - g.tok0) * p.group;
    const int v0 = min(left, full), rows = g.two ? min(left, 2 * full) : v0;  // rows of the first M tile, of both
    int i = piece0 + threadIdx.x % kTask;
    bool mine = i < rows * (D / 4);
    if (WAYS == 1) {
      if (!mine) continue;
    } else {
      if (piece0 >= rows * (D / 4)) continue;  // (all threads of the block)
      if (!mine) i = 0;
      mine = mine && !second;
    }
    const int c = i / rows * 4, k = i % rows;        // columns c .. c + 3 of row k
    const int rr = k < v0 ? k : kTile + k - v0;      // its place in a part
    const int tok = g.tok0 + k / p.group, of = k % p.group;
    const int64_t row = g.row0 + tok, r = row * p.group + of;
    int there = kLong;
    float2 rest_ml;
    float4 rest_o;
    if (mine && g.kind == kPrefix && p.rest_items > 0) {  // (on their way together with the parts)
      there = __ldcg(p.row_short + ml_at(p, 0, g.head, r));
      rest_ml = __ldcg(p.row_ml + ml_at(p, 1, g.head, r));
      rest_o = __ldcg(o_at<D>(p, 1, g.head, r, c));
    }
    float m = -INFINITY, l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto add = [&](float2 ml, float4 o) {
      const Pair z = join(make_float2(m, l), ml, p.c);
      m = z.m;
      l = z.l;
      v = make_float4(fmaf(v.x, z.e, o.x * z.f), fmaf(v.y, z.e, o.y * z.f), fmaf(v.z, z.e, o.z * z.f),
                      fmaf(v.w, z.e, o.w * z.f));
    };
    const int mid = (w0 + g.last) / 2;
    const int wa = second ? mid + 1 : w0, wb = WAYS == 1 || second ? g.last : mid;
#pragma unroll 4
    for (int w = wa; w <= wb; ++w) {
      const size_t at = ((size_t)w * 2 + (w == w0)) * 2 * kTile;
      add(__ldcg(p.part_ml + at + rr),
          __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D) + (size_t)(c / 4) * (2 * kTile) + rr));
    }
    if constexpr (WAYS > 1) {
      __syncthreads();  // (what the task before left has been read)
      if (second) {
        other_o[threadIdx.x - kTask] = v;
        other_ml[threadIdx.x - kTask] = make_float2(m, l);
      }
      __syncthreads();
      if (!mine) continue;
      add(other_ml[threadIdx.x], other_o[threadIdx.x]);
    }
    bool done = g.kind == kWhole;
    if (there == kDone) {
      add(rest_ml, rest_o);
      done = true;
    }
    if (!done) {
      *o_at<D>(p, g.kind == kRest, g.head, r, c) = v;
      if (c == 0) p.row_ml[ml_at(p, g.kind == kRest, g.head, r)] = make_float2(m, l);
      continue;
    }
    const float norm = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    const int head = g.head * p.group + of;
    *reinterpret_cast<uint2*>(p.out + (row * p.out_stride + (int64_t)head * D + c) * 2) =
        make_uint2(T::pack(v.x * norm, v.y * norm), T::pack(v.z * norm, v.w * norm));
    if (p.lse && c == 0) p.lse[row * p.q_heads + head] = log_sum<T>(m, l, p.c);
  }
}

// Rows whose sequence has much for itself: the prefix's part and the own part, out =
// sum of the parts, each times exp(its maximum - the larger one), over the sum of
// theirs.  A few blocks a sequence; a thread takes 4 columns of a row.
constexpr int kPairThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kPairThreads) attend_pair_kernel(const AttendParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x;
  Span s;
  const int e = __ldcg(p.errs);
  if (e == kMisfit || e == kAlone || !rest_of(p, b, &s) || s.kind != kRest || is_short(p, s)) return;
  const int64_t rows = (int64_t)s.n * p.group, all = rows * p.kv.kv_heads * (D / 4);
  for (int64_t i = blockIdx.y * kPairThreads + threadIdx.x; i < all; i += gridDim.y * kPairThreads) {
    const int64_t r = (int64_t)s.row0 * p.group + i % rows, x = i / rows;
    const int c = (int)(x % (D / 4)) * 4, head = (int)(x / (D / 4));
    const Pair z = join(__ldcg(p.row_ml + ml_at(p, 0, head, r)), __ldcg(p.row_ml + ml_at(p, 1, head, r)), p.c);
    const float4 u = __ldcg(o_at<D>(p, 0, head, r, c)), v = __ldcg(o_at<D>(p, 1, head, r, c));
    const float norm = z.l > 0.f ? 1.f / z.l : z.l == 0.f ? 0.f : z.l;  // (NaN stays)
    const int64_t row = r / p.group, q_head = (int64_t)head * p.group + r % p.group;
    *reinterpret_cast<uint2*>(p.out + (row * p.out_stride + q_head * D + c) * 2) =
        make_uint2(T::pack(fmaf(u.x, z.e, v.x * z.f) * norm, fmaf(u.y, z.e, v.y * z.f) * norm),
                   T::pack(fmaf(u.z, z.e, v.z * z.f) * norm, fmaf(u.w, z.e, v.w * z.f) * norm));
    if (p.lse && c == 0) p.lse[row * p.q_heads + q_head] = log_sum<T>(z.m, z.l, p.c);
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
  return (size_t)workers * (sizeof(SharedSeg) + 16) + part_rows(workers) * (sizeof(float2) + sizeof(float) * head_dim) + 64;
}

constexpr int64_t kShareBytes = 16 << 20, kShareRowBytes = 4 << 20;

// What joining two results of every row takes beside that.
size_t shared_bytes(int64_t rows, int head_dim) {
  return 2 * (size_t)rows * (sizeof(float2) + sizeof(float) * head_dim) + (size_t)rows * sizeof(int32_t) + 256;
}

template <typename T, int D>
cudaError_t launch_rest(const AttendParams& p, const CUtensorMap& kv, const CUtensorMap& q, cudaLaunchConfig_t& cfg) {
  static bool ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(attend_rest_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)RestCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  cfg.gridDim = dim3((unsigned)p.rest_items);
  cfg.blockDim = dim3(kRestThreads);
  cfg.dynamicSmemBytes = RestCfg<D>::kSmem;
  return cudaLaunchKernelEx(&cfg, attend_rest_kernel<T, D>, p, kv, q);
}

template <typename T, int D, bool SH>
cudaError_t launch(const AttendParams& p, const CUtensorMap& kv, const CUtensorMap& q, const CUtensorMap& pq,
                   const CUtensorMap& rest, const CUtensorMap& rest_q,
                   cudaStream_t s) {
  static bool ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(attend_kernel<T, D, SH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_bytes<D>());
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
  if constexpr (SH) {
    if (p.rest_items > 0) e = launch_rest<T, D>(p, rest, rest_q, cfg);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3((unsigned)p.workers);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D>();
  e = cudaLaunchKernelEx(&cfg, attend_kernel<T, D, SH>, p, kv, q, pq);
  if (e != cudaSuccess) return e;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  if constexpr (SH) {
    // An item's rows are of two tiles at most, and of no more tokens than the call has (without prefixes: a sequence).  No
    // more blocks than the tasks of the items that can be in parts: four sequences behind 32 slots 14.2 us, with all blocks
    // 15.9.
    const int64_t blocks = p.workers * kJoinSharedBlocks, step = 2 * p.tile_tokens, n = p.tok.n_tokens;
    const int64_t one = p.groups > 0 || p.max_tokens > n ? n : p.max_tokens;
    const int64_t pieces = (one < 1 ? 1 : one < step ? one : step) * p.group * (D / 4);
    const auto items_of = [&](int64_t runs) { return (n + runs * (step - 1)) / step * p.kv.kv_heads; };
    const int64_t prefixes = items_of(p.groups), items = (p.groups > 0 ? prefixes : 0) + items_of(p.tok.batch);
    AttendParams j = p;
    while ((int64_t)kJoinThreads << j.join_shift < pieces) ++j.join_shift;
    const bool halves = p.groups > 0 && prefixes << (j.join_shift + 1) <= blocks;
    if (halves) ++j.join_shift;
    const int64_t most = (items < p.workers ? items : p.workers) << j.join_shift;
    cfg.gridDim = dim3((unsigned)((most < blocks ? most : blocks) + p.tok.batch));
    e = halves ? cudaLaunchKernelEx(&cfg, attend_join_shared_kernel<T, D, 2>, j)
               : cudaLaunchKernelEx(&cfg, attend_join_shared_kernel<T, D, 1>, j);
  } else {
    cfg.gridDim = dim3((unsigned)(p.workers * kJoinBlocks + p.tok.batch));
    e = cudaLaunchKernelEx(&cfg, attend_join_kernel<T, D>, p);
  }
  if (!SH || p.groups == 0 || e != cudaSuccess) return e;
  const int64_t most = (int64_t)(p.max_tokens < p.tok.n_tokens ? p.max_tokens : p.tok.n_tokens) * p.q_heads * (D / 4);
  const int64_t room = (8 * p.workers + p.tok.batch - 1) / p.tok.batch, want = (most + kPairThreads - 1) / kPairThreads;
  cfg.gridDim = dim3((unsigned)p.tok.batch, (unsigned)(want < 1 ? 1 : want < room ? want : room));
  cfg.blockDim = dim3(kPairThreads);
  return cudaLaunchKernelEx(&cfg, attend_pair_kernel<T, D>, p);
}

template <bool SH>
cudaError_t launch(int dtype, int head_dim, const AttendParams& p, const CUtensorMap& kv, const CUtensorMap& q,
                   const CUtensorMap& pq, const CUtensorMap& rest, const CUtensorMap& rest_q,
                   cudaStream_t s) {
  if (dtype == TC_DT_BF16)
    return head_dim == 128 ? launch<Bf16, 128, SH>(p, kv, q, pq, rest, rest_q, s) : launch<Bf16, 64, SH>(p, kv, q, pq, rest, rest_q, s);
  return head_dim == 128 ? launch<F16, 128, SH>(p, kv, q, pq, rest, rest_q, s) : launch<F16, 64, SH>(p, kv, q, pq, rest, rest_q, s);
}

tc_status attend(const char* who, const tc_kv_t* kv, int32_t layer, const tc_tokens_t* tokens, const tc_attend_t* a,
                 const tc_shared_t* sh, void* workspace, int64_t workspace_bytes, int32_t* status, void* stream) {
  tc_status rc = kv_check(who, kv);
  if (rc == TC_OK) rc = kv_check_tokens(who, tokens, true);
  if (rc != TC_OK) return rc;
  if (!a || !status || layer < 0 || layer >= kv->layers || a->q_heads < 1 || a->max_tokens < 0 ||
      !tokens->page_table || tokens->table_width < 1 || !(a->scale == a->scale))
    return kv_fail(TC_ERR_INVALID_ARG, who, ": invalid arguments");
  if (a->q_heads % kv->kv_heads != 0 || a->q_heads / kv->kv_heads > 128)
    return kv_fail(TC_ERR_UNSUPPORTED, who,
                   ": q_heads must be a multiple of kv_heads, with at most 128 of them for each");
  if (a->tree && (a->tree_words < 1 || a->tree_words > TC_TREE_MAX_WORDS || a->max_tokens > 64 * a->tree_words))
    return kv_fail(TC_ERR_CAPACITY, who, ": a tree wants 1 to 4 words and at most 64 tokens a word");
  if (sh && (sh->groups < 1 || sh->groups > tokens->batch || !sh->cu_seqs || !sh->shared_lens))
    return kv_fail(TC_ERR_INVALID_ARG, who, ": there must be 1 to batch groups, with cu_seqs and shared_lens");
  int64_t need = 0;
  rc = sh ? tc_attend_shared_workspace(kv, tokens->n_tokens, a->q_heads, &need) : tc_attend_workspace(kv, &need);
  if (rc != TC_OK) return rc;
  if (!workspace || kv_misaligned(workspace, 16) || workspace_bytes < need)
    return kv_fail(TC_ERR_CAPACITY, who, ": the workspace is too small or not 16-byte aligned");
  const int64_t row = (int64_t)a->q_heads * kv->head_dim;
  if (tokens->n_tokens > 0 &&
      (!a->q || !a->out || kv_misaligned(a->q, 16) || kv_misaligned(a->out, 16) || a->q_stride % 8 != 0 ||
       a->out_stride % 8 != 0 || a->q_stride < row || a->out_stride < row))
    return kv_fail(TC_ERR_INVALID_ARG, who,
                   ": q and out must be 16-byte aligned, with row strides that are multiples of 8 and hold a row");
  KvDevice dev(kv->device);
  if (!dev.ok) return kv_fail(TC_ERR_CUDA, who, ": cannot use the cache's device");
  // Keys and values of the layer: [page][keys or values, head][slot][element],
  const KvView v = kv_view(kv, layer);
  const cuuint64_t d = (cuuint64_t)kv->head_dim, sz = (cuuint64_t)kv->page_size;
  // in pieces of 64 columns.  A copy brings a page's slots of one piece.
  const int halves = kv->head_dim / 64;
  const cuuint64_t kv_dims[5] = {64, sz, (cuuint64_t)halves, (cuuint64_t)2 * kv->kv_heads, (cuuint64_t)kv->pages};
  const cuuint64_t kv_strides[4] = {d * 2, 128, sz * d * 2, (cuuint64_t)2 * kv->kv_heads * sz * d * 2};
  const cuuint32_t kv_box[5] = {64, (cuuint32_t)kv->page_size, 1, 1, 1};
  const int group = a->q_heads / kv->kv_heads, tile_tokens = kTile / group;
  // Queries: rows (token, head of the group) of one M tile, at most max_tokens of them
  // (of a prefix: of all sequences that share it).
  const auto tokens_of = [&](int most) { return most < 1 ? 1 : most < tile_tokens ? most : tile_tokens; };
  const int q_tokens = tokens_of(a->max_tokens), pq_tokens = tokens_of(tokens->n_tokens);
  const bool none = tokens->n_tokens == 0;  // (no queries: the map is not used, any valid one does)
  const cuuint64_t q_dims[3] = {d, (cuuint64_t)(none ? group : a->q_heads), (cuuint64_t)(none ? 1 : tokens->n_tokens)};
  const cuuint64_t q_strides[2] = {d * 2, (cuuint64_t)(none ? row : a->q_stride) * 2};
  const cuuint32_t q_box[3] = {64, (cuuint32_t)group, (cuuint32_t)q_tokens};
  const cuuint32_t pq_box[3] = {64, (cuuint32_t)group, (cuuint32_t)pq_tokens};
  const cuuint32_t rest_box[5] = {64, (cuuint32_t)(kv->page_size < kRestTile ? kv->page_size : kRestTile), 1, 1, 1};
  const int rest_tokens = kRestRows / group < 1 ? 1 : q_tokens < kRestRows / group ? q_tokens : kRestRows / group;
  const cuuint32_t rest_q_box[3] = {64, (cuuint32_t)group, (cuuint32_t)rest_tokens};
  CUtensorMap map_kv, map_q, map_pq, map_rest, map_rest_q;
  if (!encode(&map_kv, kv->dtype, 5, v.base, kv_dims, kv_strides, kv_box) ||
      !encode(&map_q, kv->dtype, 3, none ? kv->pool : a->q, q_dims, q_strides, q_box) ||
      (sh && (!encode(&map_pq, kv->dtype, 3, none ? kv->pool : a->q, q_dims, q_strides, pq_box) ||
              !encode(&map_rest, kv->dtype, 5, v.base, kv_dims, kv_strides, rest_box) ||
              !encode(&map_rest_q, kv->dtype, 3, none ? kv->pool : a->q, q_dims, q_strides, rest_q_box))))
    return kv_fail(TC_ERR_UNSUPPORTED, who, ": the sizes or strides do not fit a tensor map");
  if (!sh) map_pq = map_rest_q = map_q, map_rest = map_kv;
  AttendParams p{};
  p.kv = v;
  p.tok = tokens_view(tokens);
  p.q_heads = a->q_heads;
  p.group = group;
  p.tile_tokens = tile_tokens;
  p.max_tokens = a->max_tokens;
  p.q_rows = group * q_tokens;
  p.prefix_q_rows = group * pq_tokens;
  p.rest_q_rows = group * rest_tokens;
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
  p.descs = reinterpret_cast<SharedSeg*>(ws);
  ws += (size_t)p.workers * sizeof(SharedSeg);
  p.errs = reinterpret_cast<int32_t*>(ws);
  if (sh) {
    p.cu_seqs = sh->cu_seqs;
    p.shared_lens = sh->shared_lens;
    // Contexts that are small together, whatever the lengths, are read sequence by sequence: sharing them saves less than
    // the joining takes, and what it saves is less the more rows a sequence has, as these share the reads and products of
    // a tile by themselves (the mean is what counts, so that a prompt among single tokens does not decide).  In us, shared
    // and not, rows of a sequence / MB: 4 / 16 21.6 and 19.1, 32 21.9 and 23.8 (four sequences), 42 36.9 and 34.8, 85 38.0
    // and 41.1 (64 of them); 10 / 65 26.5 and 26.1, 72 39.5 and 41.1; 18 / 72 45.3 and 41.6, 128 33.1 and 33.6; 48 / 135
    // 53.4 and 49.7, 252 48.4 and 50.4 (16 sequences; four take 41.8 and 47.8 and are not shared); 180 / 510 191 and 144.
    // The errors of their groups are found all the same.
    const int64_t rows_each = (int64_t)tokens->n_tokens * group / tokens->batch;
    const int64_t most = (int64_t)tokens->batch * tokens->table_width * kv->page_size * kv->kv_heads * kv->head_dim * 4;
    p.all_groups = sh->groups;
    p.groups = most <= kShareBytes + rows_each * kShareRowBytes ? 0 : sh->groups;
    const size_t rows = 2 * (size_t)tokens->n_tokens * a->q_heads;
    ws += ((size_t)p.workers * sizeof(int32_t) + 15) / 16 * 16;
    ws += (128 - (reinterpret_cast<uintptr_t>(ws) & 127)) & 127;
    p.row_o = reinterpret_cast<float*>(ws);
    p.row_ml = reinterpret_cast<float2*>(ws + rows * sizeof(float) * kv->head_dim);
    p.row_short = reinterpret_cast<int32_t*>(p.row_ml + rows);
    // With fewer items than SMs each has an SM in the main kernel anyway, and a launch less counts: four sequences of 3 to
    // 21 slots behind 32 19.9 us without, 21.4 with it.
    const int64_t items = (int64_t)tokens->batch * kv->kv_heads;
    p.rest_items = p.groups == 0 || items <= p.workers || items > INT32_MAX || group > kRestRows ? 0 : (int)items;
  }
  p.rest_wait_limit = a->wait_polls > 0 ? (int32_t)(a->wait_polls < 1 << 30 ? a->wait_polls : 1 << 30) : kWaitLimit;
  p.rest_withhold = a->withhold == 3 ? 2 : a->withhold != 0;
  const bool rest_only = sh && (a->withhold == 2 || a->withhold == 3);
  p.wait_limit = rest_only ? kWaitLimit : p.rest_wait_limit;
  p.withhold = !rest_only && a->withhold != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = sh ? launch<true>(kv->dtype, kv->head_dim, p, map_kv, map_q, map_pq, map_rest, map_rest_q, s)
                           : launch<false>(kv->dtype, kv->head_dim, p, map_kv, map_q, map_pq, map_rest, map_rest_q, s);
  return e == cudaSuccess ? TC_OK : kv_cuda_fail(e, sh ? "tc_attend_shared: " : "tc_attend: ");
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

extern "C" tc_status tc_attend_shared_workspace(const tc_kv_t* kv, int32_t n_tokens, int32_t q_heads, int64_t* bytes) {
  const tc_status rc = tc_attend_workspace(kv, bytes);
  if (rc != TC_OK) return rc;
  if (n_tokens < 0 || q_heads < 1)
    return kv_fail(TC_ERR_INVALID_ARG, "tc_attend_shared_workspace: n_tokens or q_heads out of range");
  *bytes += (int64_t)shared_bytes((int64_t)n_tokens * q_heads, kv->head_dim);
  return TC_OK;
}

extern "C" tc_status tc_attend(const tc_kv_t* kv, int32_t layer, const tc_tokens_t* tokens, const tc_attend_t* a,
                               void* workspace, int64_t workspace_bytes, int32_t* status, void* stream) {
  return attend("tc_attend", kv, layer, tokens, a, nullptr, workspace, workspace_bytes, status, stream);
}

extern "C" tc_status tc_attend_shared(const tc_kv_t* kv, int32_t layer, const tc_tokens_t* tokens,
                                      const tc_attend_t* a, const tc_shared_t* shared, void* workspace,
                                      int64_t workspace_bytes, int32_t* status, void* stream) {
  if (!shared) return kv_fail(TC_ERR_INVALID_ARG, "tc_attend_shared: shared is NULL");
  return attend("tc_attend_shared", kv, layer, tokens, a, shared, workspace, workspace_bytes, status, stream);
}
