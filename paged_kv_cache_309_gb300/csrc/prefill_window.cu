// prefill_window.cu -- causal varlen prefill attention over the paged cache with a
// sliding window and a few first tokens that stay visible (tcgen05, accumulators in
// tensor memory).
//
// What is computed: new token j of sequence b sits at position p = L_b - n_b + j
// and attends to tokens t <= p with t > p - window or t < num_sink; query head h
// uses kv head h / G.  fp32 online softmax in base 2, sums of weights in fp32.  Each weight is
// rounded to one bf16 for the second product, as in the plain prefill: as two terms (decode's
// way) it would take two products of the tensor core instead of one, a half more in all, where
// products are what bounds a long prompt.  It costs a relative error of 0.0022 instead of 0.0016.
//
// An item is two query tiles of 128 rows (128 / G consecutive new tokens x the G
// query heads of one kv head each) of one sequence; they share every key and value.
// Its steps of 64 keys run over the places (window.cuh) of the rows that the first tokens
// and its first row's window leave.  Windows make items short (a window of 250: five
// steps), so CTAs stay: one per SM walks items c, c + grid, ... of all sequences, and while
// an item's last steps are weighed and its rows written, the next one's queries, keys and
// values land and its first score products run.
//  * TMEM (512 columns): outputs O0, O1 (128 each) and for each query tile two score
//    buffers of 64, so that while the softmax works on step v, S(v + 1) is there or on
//    its way.  A step's weights (bf16 pairs) overwrite the first half of its scores.
//  * warps 0 and 3 load keys and values, four steps ahead (one warp for both came too late:
//    1680 us where two took 1300), warp 0 posts each step's row mask; warp 2 loads the
//    query tiles; all by TMA, 128-byte swizzled.
//  * one thread of warp 1 issues every product: O_i += P_i(v) V(v), S_i(v + 2) = Q_i K(v + 2)^T,
//    then the other query tile's.  Products of one thread run in order, so S_i(v + 2)
//    may overwrite P_i(v) without a wait between them.  The core holds a few products ahead,
//    about 100 cycles of work, so what this warp does besides must be short: the middle of
//    an item is a loop of its own, and barriers are asked before their answers matter.
//  * warps 4-7 and 8-11 do the softmax of query tiles 0 and 1, one thread per row.
// What bounds it (cycles of a step of both query tiles, on a long prompt): products 1240 alone
// (2 x (370 + 256): a score product of 64 keys reads as many bytes of shared memory as it has
// cycles), 1500 beside copies and hand-overs; the softmax warps' chain of scores, maximum,
// exponentials, weights and barriers 850 alone, 1250 and 400 of hand-overs where two
// warps of a quarter of the SM run in step: some 1700 in all.  Warps wait for
// instructions more than for anything else (1.8 warps an issue): loops are kept short.
// Measured (GPU time, perf/gpu_times.py; heads q / kv):
//  * 4 prompts of 8192, window 4096, 32 / 8: 1205 us back to back (1155 after a pause), 1.37
//    PFLOP/s over visible pairs (a CTA per item and products issued from a branch of one
//    lane: 1903);
//  * 8 chunks of 512 behind up to 6000, window 1024, 16 / 8: 45.5 us (73); its 256 items
//    take two rounds of the 152 SMs;
//  * 5 prompts of 1000 .. 6001, window 250, 16 / 2: 67 us (147): an item of five steps takes
//    14700 cycles, 4000 of them from its last weights to the next one's first (product, rows
//    read and written, first step), the other steps at an item's ends 2450 each;
//  * a few short rows: 9.5 us, a chain of lengths, block ids, copies and products.
// Slower: the two warps of a quarter kept apart by a barrier (1375), the next scores read before
// the weights are handed over (1360), both query tiles' products in one rolled body (1245),
// rows stored straight from registers (narrow window 75), next queries brought to L2 (no gain);
// before the loads were split, two issuing warps, one buffer of 128 keys, four softmax groups.
//
// Every wait is bounded (2 s); a timeout sets an error bit, drains what was issued and
// frees TMEM before the CTA exits.
#include <atomic>
#include <climits>

#include "tc_ops.cuh"
#include "window.cuh"

namespace pa_detail {
namespace {

using namespace pa;
using namespace tc;

constexpr int kD = 128;
constexpr int kM = 128;    // rows per query tile (tokens x heads)
constexpr int kStep = 64;  // keys per step
constexpr int kSlots = 4;  // of keys, and as many of values: step n of the CTA is in slot n % 4
constexpr int kThreads = 12 * 32;              // 4 role warps + 2 x 4 softmax warps
constexpr int kChunk = 128 * 128;              // 64 elements of 128 query rows: 16 KB
constexpr int kHalf = kStep * 128;             // 64 elements of a step's rows: 8 KB
constexpr int kQOff = 0;                       // query tile i: two chunks
constexpr int kSlotBytes = 2 * kHalf;
constexpr int kKOff = 2 * 2 * kChunk;
constexpr int kVOff = kKOff + kSlots * kSlotBytes;
constexpr int kStageOff = kVOff + kSlots * kSlotBytes;  // 32 half rows per softmax warp
constexpr int kStageBytes = 32 * 128;
constexpr int kBarOff = kStageOff + 8 * kStageBytes;
// Mask slot n % 8 is written again for step n + 8, whose keys need those of step n + 4 used; that
// score product comes after the output product of step n + 2, which needs the weights of
// both query tiles' step n + 2.
constexpr int kMaskSlots = 8;
// q_full, q_empty, pv_done, o_empty [2] each, s_full, p_full [2][2], k_full, k_empty, v_full,
// v_empty, drain
constexpr int kNumBars = 4 * 2 + 2 * 4 + 4 * kSlots + 1;
constexpr int kMaskOff = kBarOff + (kNumBars + 1) / 2 * 16;  // a 64-bit word per slot
constexpr int kMiscOff = kMaskOff + kMaskSlots * 8;
constexpr int kBytes = kMiscOff + 16;
constexpr int kAlloc = kBytes + 1024;
static_assert(kAlloc <= 227 * 1024, "shared memory");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 0;      // [0, 256): outputs O0, O1
constexpr uint32_t kSCol = 256;    // [256, 512): score buffer b of query tile i at + 128 i + 64 b
constexpr uint32_t kIdescS = instr_desc(kM, kStep, false);
constexpr uint32_t kIdescPV = instr_desc(kM, kD, true);
constexpr float kRescaleLog2 = 8.0f;
constexpr int kLog2Rows = 6;        // copies are of up to 64 rows
constexpr int kMaxItems = 1 << 24;  // (queries of 2^24 items are a terabyte)

struct Params {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k_cache;
  const __nv_bfloat16* v_cache;
  const int32_t* block_tables;
  const int32_t* cu_seqlens_q;
  const int32_t* context_lens;
  unsigned* err;
  int64_t num_blocks;
  int32_t num_seqs;
  int32_t total_tokens;
  int32_t max_q_len;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;
  int32_t tokens_per_tile;  // kM / group
  int32_t block_size;
  int32_t log2_bs;
  int32_t max_blocks_per_seq;
  int32_t window;
  int32_t num_sink;
  float scale_log2;
};

// 16 columns of this thread's TMEM lane, without waiting
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Waits for this thread's stores to TMEM, and tells whether a barrier's phase is complete: the
// two take their time side by side.
__device__ __forceinline__ bool wait_st_and_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred t;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 t, [%1], %2;\n\t"
      "tcgen05.wait::st.sync.aligned;\n\t"
      "selp.u32 %0, 1, 0, t;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// max of three, NaN if one of them is
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// ------------------------------------------------------------------ items --
struct Item {
  int b, g;      // sequence, kv head
  int q_row;     // the item's first row of q
  int ntok;      // its new tokens
  int nsteps;    // steps of 64 places (0: no row has a key)
  int nq;        // query tiles with a row
  int pos0;      // place of its first token
  WindowRange win;
};

// A warp's walk over items first, first + step, ...: items lie sequence by sequence, in a
// sequence the latest tokens first, kv heads fastest.  Lane l holds sequence
// chunk + l of the 32 in hand.
struct Walk {
  int next, base;  // next item; items before the chunk
  int chunk;
  int q0, n, avail, len;  // this lane's sequence: first row, new tokens, those with a row
  int incl;               // items of the chunk up to and with this lane's
  __device__ __forceinline__ void load(const Params& p, int lane) {
    const int b = chunk + lane;
    q0 = n = avail = len = 0;
    if (b < p.num_seqs) {
      q0 = __ldg(p.cu_seqlens_q + b);
      n = max(__ldg(p.cu_seqlens_q + b + 1) - q0, 0);
      len = max(__ldg(p.context_lens + b), 0);
      // (rows outside the array, and tokens past max_q_len, are not there)
      if (q0 >= 0) avail = max(min(min(n, p.max_q_len), p.total_tokens - q0), 0);
    }
    const int per = 2 * p.tokens_per_tile;
    // (sequences that share rows of q could add up to any number; the launch takes up to
    // kMaxItems, so sums of 32 sequences fit)
    incl = min((avail + per - 1) / per, kMaxItems / p.num_kv_heads) * p.num_kv_heads;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
  }
  __device__ __forceinline__ Walk(const Params& p, int first, int lane)
      : next(first), base(0), chunk(0) {
    load(p, lane);
  }
  __device__ __forceinline__ bool get(const Params& p, int step, int lane, Item& it) {
    for (;;) {
      const int all = __shfl_sync(0xffffffffu, incl, 31);
      if (next < base + all) break;
      base += all;
      chunk += 32;
      if (chunk >= p.num_seqs || base > kMaxItems) return false;
      load(p, lane);
    }
    const int at = next - base;
    next += step;
    const int l = __ffs(__ballot_sync(0xffffffffu, at < incl)) - 1;
    const int before = l == 0 ? 0 : __shfl_sync(0xffffffffu, incl, l - 1);
    const int end = __shfl_sync(0xffffffffu, incl, l);
    it.b = chunk + l;
    const int row0 = __shfl_sync(0xffffffffu, q0, l);
    const int count = __shfl_sync(0xffffffffu, n, l);
    const int rows = __shfl_sync(0xffffffffu, avail, l);
    int L = __shfl_sync(0xffffffffu, len, l);
    const int j = (end - 1 - at) / p.num_kv_heads;  // the item's pair of query tiles
    it.g = (at - before) % p.num_kv_heads;
    const int cap = p.max_blocks_per_seq * p.block_size;
    if (L > cap) {
      if (j == 0 && it.g == 0 && lane == 0) atomicOr(p.err, PA_DEVERR_CONTEXT_CLIPPED);
      L = cap;
    }
    const int first = 2 * j * p.tokens_per_tile;  // of the sequence's new tokens
    it.q_row = row0 + first;
    it.ntok = min(2 * p.tokens_per_tile, rows - first);
    it.nq = it.ntok > p.tokens_per_tile ? 2 : 1;
    it.pos0 = L - count + first;
    const int kend = min(L, it.pos0 + it.ntok);
    if (kend <= 0) {  // no row has a key (pos0 may be far below zero)
      it.win = WindowRange{0, 0, 0, 0};
    } else {
      it.win = window_range(kend, max(0, it.pos0 - p.window + 1), p.num_sink,
                            min(p.log2_bs, kLog2Rows));
      it.pos0 -= it.win.skip;
    }
    it.nsteps = (it.win.len + kStep - 1) / kStep;
    return true;
  }
};

// --------------------------------------------------------------- products --
// The issuing warp stays together and one lane's predicate guards each instruction: in a branch
// of one lane every operand would be moved to the uniform registers that these
// instructions read, at ~100 cycles a product.  Descriptors come as two words.
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a_tmem, uint32_t b,
                                       uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t one, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(one)
      : "memory");
}
// A score product: S = Q K^T over 64 keys, 8 k-steps of 16 over the 128 head elements, both
// operands K-major 128-byte swizzled (a k-step in a chunk is 32 bytes on).  While it is
// issued, three barriers are asked whether their phase of that parity is complete: beside the
// operands' reads of shared memory an answer takes 150 cycles and more.
struct Tests {
  uint32_t bar[3], parity[3], done[3];
};
__device__ __forceinline__ void score_product(uint32_t one, uint32_t d, uint32_t q, uint32_t k,
                                              uint32_t hi, uint32_t idesc, Tests& t) {
#define PA_KSTEP(qoff, koff, acc)                                         \
  "add.u32 a, %5, " qoff ";\n\tadd.u32 b, %6, " koff ";\n\t"             \
  "mov.b64 da, {a, %7};\n\tmov.b64 db, {b, %7};\n\t"                     \
  "@q tcgen05.mma.cta_group::1.kind::f16 [%4], da, db, %8, " acc ";\n\t"
  asm volatile(
      "{\n\t.reg .pred q, yes, no, t0, t1, t2;\n\t.reg .b32 a, b;\n\t.reg .b64 da, db;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 t0, [%9], %12;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 t1, [%10], %13;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 t2, [%11], %14;\n\t"
      "setp.ne.b32 q, %3, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\tsetp.ne.b32 no, 0, 0;\n\t"
      PA_KSTEP("0", "0", "no") PA_KSTEP("2", "2", "yes") PA_KSTEP("4", "4", "yes")
      PA_KSTEP("6", "6", "yes") PA_KSTEP("1024", "512", "yes") PA_KSTEP("1026", "514", "yes")
      PA_KSTEP("1028", "516", "yes") PA_KSTEP("1030", "518", "yes")
      "selp.u32 %0, 1, 0, t0;\n\tselp.u32 %1, 1, 0, t1;\n\tselp.u32 %2, 1, 0, t2;\n\t}"
      : "=r"(t.done[0]), "=r"(t.done[1]), "=r"(t.done[2])
      : "r"(one), "r"(d), "r"(q), "r"(k), "r"(hi), "r"(idesc), "r"(t.bar[0]), "r"(t.bar[1]),
        "r"(t.bar[2]), "r"(t.parity[0]), "r"(t.parity[1]), "r"(t.parity[2])
      : "memory");
#undef PA_KSTEP
}
// one lane of a warp that is together, the same one every time
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r));
  return r;
}

// ------------------------------------------------------------------ loads --
// A step's block pieces: lane i holds piece i % nbox: its block id (looked up a step before it is
// used), first row in the block, and rows that an item's query may see, as bits of the step.
struct Pieces {
  int bid, row, g;  // (g: the item's kv head)
  uint64_t seen;
};
__device__ __forceinline__ Pieces find_pieces(const Params& p, const Item& it, int place0,
                                              int log2_rpb, int lane) {
  Pieces x{-1, 0, it.g, 0};
  const int rpb = 1 << log2_rpb;
  const int start = (lane & ((kStep >> log2_rpb) - 1)) << log2_rpb;  // of the step's places
  const int first = it.win.row(place0 + start);
  const int rows = min(rpb, it.win.len - place0 - start);
  if (rows > 0) {
    x.bid = __ldg(p.block_tables + static_cast<int64_t>(it.b) * p.max_blocks_per_seq +
                  (first >> p.log2_bs));
    x.row = first & (p.block_size - 1);
    // (visible() from the row of bit 0, if this piece's run began there)
    x.seen = WindowRange::below(start + rows) & ~WindowRange::below(start) &
             it.win.visible(first - start, p.num_sink);
  }
  return x;
}
// The keys or values of one step; copy c is half c / nbox (64 head elements) of piece c % nbox.
__device__ __forceinline__ void load_step(const CUtensorMap* tm, int row, int g, uint8_t* dst,
                                          uint64_t* full, int log2_rpb, uint64_t pol, int lane) {
  const int nbox = kStep >> log2_rpb;
  const uint32_t there = __ballot_sync(0xffffffffu, lane < nbox && row >= 0);
  if (lane == 0)
    mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(there) << (log2_rpb + 8)));
  __syncwarp();
  if (lane < 2 * nbox && row >= 0) {
    const int half = lane >= nbox ? 1 : 0;
    tma_load_3d(dst + half * kHalf + ((lane & (nbox - 1)) << (log2_rpb + 7)), tm, 64 * half, g, row,
                full, pol);
  }
}

// ------------------------------------------------------- rows made again --
// A tile's product multiplies the values of a token that one row sees and another does not by that
// other row's weight 0, which is NaN for a value that is not finite.  Items with such rows are
// marked, and when all are done the softmax warps make the rows again that do not see some token
// of such values: the scan of an item's values finds the newest of these tokens and the oldest
// behind the first ones, and a row sees all of them where the newest is no newer than the row and the
// oldest not before its window.  (Such rows stay as they are.)  Tiles of 128 rows by
// mma.sync, 16 rows to a warp, over memory that keys, values and queries have left.  Elements that are
// not finite enter the product as 0; where a row sees one of them, whatever its weight, its
// output takes the infinity or NaN on: two more products of ones and zeros, of the elements
// +inf and -inf (NaN is both), say which.
// Measured on 4 prompts of 8192 (window 4096, 32 / 8 heads; 1.16 ms without): one infinite element
// 1.75 ms, one token of NaN 1.9, an infinite element in a first token 1.3, one in every 64th token
// (all rows are made again) 22 to 25, all values +inf 54, all NaN 3.8 (rows of NaN are done).
// Rows made again one by one took 214 ms for the one token.
constexpr int kAgainPitch = 256 + 16;             // bytes between rows: eight fall into all 32 banks
constexpr int kAgainKV = kM * kAgainPitch;        // behind the queries two buffers of keys and values
constexpr int kAgainBuffer = 2 * kStep * kAgainPitch;
// newest, oldest, and per buffer a stamp for every 16 keys: of the step that has such a value there
constexpr int kAgainMisc = kAgainKV + 2 * kAgainBuffer;
static_assert(kAgainMisc + 40 <= kStageOff, "inside the memory of queries, keys and values");
constexpr int kSoftmaxThreads = 8 * 32;

__device__ __forceinline__ void softmax_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
}
// the same, and whether every thread came with `x`
__device__ __forceinline__ bool softmax_all(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\t"
      "bar.red.and.pred b, 1, %2, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "n"(kSoftmaxThreads)
      : "memory");
  return r != 0;
}
// 16 bytes from global memory, or zeros, without waiting
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ bool not_finite(uint32_t pair) {
  return (pair & 0x7F80u) == 0x7F80u || (pair & 0x7F800000u) == 0x7F800000u;
}
// Of a pair of bf16: finite values (others 0); ones where it is +inf or NaN; -inf or NaN
__device__ __forceinline__ void apart(uint32_t pair, uint32_t& finite, uint32_t& up,
                                      uint32_t& down) {
  finite = pair;
  up = down = 0u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t x = (pair >> (16 * h)) & 0xFFFFu;
    if ((x & 0x7F80u) == 0x7F80u) {
      finite &= h ? 0x0000FFFFu : 0xFFFF0000u;
      if (x != 0xFF80u) up |= 0x3F80u << (16 * h);
      if (x != 0x7F80u) down |= 0x3F80u << (16 * h);
    }
  }
}
// one of 32 bits for an item, by its first row of q and out (in heads)
__device__ __forceinline__ unsigned item_bit(uint32_t first) {
  return 1u << ((first * 2654435761u) >> 27);
}
// A step's rows from the pieces that find_pieces gave (the same in every lane for one place)
struct StepRows {
  Pieces x;
  uint64_t seen;
  __device__ __forceinline__ StepRows(const Params& p, const Item& it, int v, int log2_rpb,
                                      int lane)
      : x(find_pieces(p, it, v * kStep, log2_rpb, lane)) {
    if (x.bid < 0 || static_cast<int64_t>(x.bid) >= p.num_blocks) x.seen = 0ull;
    const uint32_t lo = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(x.seen));
    const uint32_t hi = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(x.seen >> 32));
    seen = (static_cast<uint64_t>(hi) << 32) | lo;
  }
  // element offset of place r's row in the caches; called by whole warps
  __device__ __forceinline__ int64_t offset(const Params& p, int r, int log2_rpb) const {
    const int bid = __shfl_sync(0xffffffffu, x.bid, r >> log2_rpb);
    const int row = __shfl_sync(0xffffffffu, x.row, r >> log2_rpb);
    return ((static_cast<int64_t>(bid) * p.block_size + row + (r & ((1 << log2_rpb) - 1))) *
                p.num_kv_heads +
            x.g) *
           kD;
  }
};

// The rows of one query tile that do not see all of the tokens newest .. oldest
__device__ __noinline__ void tile_again(const Params& p, uint8_t* smem, const Item& it, int tile,
                                        int newest, int oldest, int& serial) {
  const int t = threadIdx.x - (kThreads - kSoftmaxThreads);
  const int warp = t >> 5, lane = t & 31;
  const int G = p.group, log2_rpb = min(p.log2_bs, kLog2Rows);
  const int tok0 = tile * p.tokens_per_tile;
  const int toks = min(p.tokens_per_tile, it.ntok - tok0);
  const uint32_t base = smem_u32(smem);
  volatile int* stamps = reinterpret_cast<volatile int*>(smem + kAgainMisc) + 2;
  const int c16 = lane & 15, half = lane >> 4;  // 16 lanes to a row of 256 bytes
  auto row_of = [&](int r) {  // element offset of tile row r in q and out
    return (static_cast<int64_t>(it.q_row + tok0 + r / G) * p.num_q_heads + it.g * G + r % G) * kD;
  };
#pragma unroll 1
  for (int r = 2 * warp + half; r < kM; r += 16) {
    const bool there = r / G < toks;
    copy16(base + r * kAgainPitch + 16 * c16, p.q + (there ? row_of(r) + 8 * c16 : 0), there);
  }
  // this warp's eight rows of a step's keys and values
  auto request = [&](int v, const StepRows& s) {
    const uint32_t dst = base + kAgainKV + (v & 1) * kAgainBuffer + 16 * c16;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 8 * warp + 2 * k + half;
      const int64_t at = s.offset(p, r, log2_rpb);
      const bool there = (s.seen >> r) & 1ull;
      copy16(dst + r * kAgainPitch, p.k_cache + (there ? at + 8 * c16 : 0), there);
      copy16(dst + (kStep + r) * kAgainPitch, p.v_cache + (there ? at + 8 * c16 : 0), there);
    }
  };
  // rows 16 warp + lane / 4 and eight more of the tile: this lane's
  const int gq = lane >> 2, tq = lane & 3;
  int pos[2];
  bool again[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = 16 * warp + gq + 8 * j;
    pos[j] = it.pos0 + tok0 + r / G;
    again[j] = r / G < toks && (newest > pos[j] || oldest <= pos[j] - p.window);
  }
  float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
  const int lo8 = lane & 7, hi8 = (lane >> 3) & 1;
  const uint32_t q_addr = base + (16 * warp + lo8 + 8 * hi8) * kAgainPitch + 16 * half;
  const uint32_t k_row = (lo8 + 8 * half) * kAgainPitch + 16 * hi8;
  const uint32_t v_row = (kStep + lo8 + 8 * hi8) * kAgainPitch + 16 * half;

  StepRows next(p, it, 0, log2_rpb, lane);
  uint64_t seen = next.seen;
  request(0, next);
  asm volatile("cp.async.commit_group;" ::: "memory");
  next = StepRows(p, it, 1, log2_rpb, lane);
#pragma unroll 1
  for (int v = 0; v < it.nsteps; ++v) {
    const uint64_t seen_now = seen;
    if (v + 1 < it.nsteps) {
      seen = next.seen;
      request(v + 1, next);
      next = StepRows(p, it, v + 2, log2_rpb, lane);
    }
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 1;" ::: "memory");
    const uint8_t* buf = smem + kAgainKV + (v & 1) * kAgainBuffer;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 8 * warp + 2 * k + half;
      const uint4 x = *reinterpret_cast<const uint4*>(buf + (kStep + r) * kAgainPitch + 16 * c16);
      bad |= not_finite(x.x) || not_finite(x.y) || not_finite(x.z) || not_finite(x.w);
    }
    volatile int* stamp = stamps + 4 * (serial & 1);
    ++serial;
    if (bad) stamp[warp >> 1] = serial;
    softmax_barrier();
    const uint32_t at = base + kAgainKV + (v & 1) * kAgainBuffer;
    float s[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      uint32_t a[4];
      ldsm_x4(q_addr + 32 * kk, a);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t b[4];
        ldsm_x4(at + k_row + 16 * n * kAgainPitch + 32 * kk, b);
        mma_bf16_16816(s[2 * n], a, b[0], b[1]);
        mma_bf16_16816(s[2 * n + 1], a, b[2], b[3]);
      }
    }
    // which of the step's places this lane's rows see (as in the first pass)
    const int k0 = v * kStep;
    uint64_t mw[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int low = pos[j] - p.window + 1;
      mw[j] = seen_now & WindowRange::below(pos[j] + 1 - k0) &
              (~WindowRange::below(low - k0) | WindowRange::below(p.num_sink - k0));
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 8 * n + 2 * tq + (i & 1);
        s[n][i] = (mw[i >> 1] >> c) & 1ull ? s[n][i] * p.scale_log2 : -INFINITY;
        mx[i >> 1] = fmaxf(mx[i >> 1], s[n][i]);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 1));
      mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 2));
      mx[j] = fmaxf(m[j], mx[j]);
      // (no key so far: m and mx are -inf, nothing to rescale)
      const float corr = mx[j] == m[j] ? 1.f : fast_exp2(m[j] - mx[j]);
      m[j] = mx[j];
      l[j] *= corr;
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        o[n][2 * j] *= corr;
        o[n][2 * j + 1] *= corr;
      }
      if (mx[j] == -INFINITY) mx[j] = 0.f;
    }
#pragma unroll
    for (int kk = 0; kk < kStep / 16; ++kk) {
      const bool special = stamp[kk] == serial;
      // weights of 16 keys, and ones where the row sees the key, as A operands
      uint32_t a[4], ones[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 2 * kk + (i >> 1), j = i & 1;
        const float e0 = fast_exp2(s[n][2 * j] - mx[j]), e1 = fast_exp2(s[n][2 * j + 1] - mx[j]);
        l[j] += e0 + e1;
        a[i] = pack_bf16x2(e0, e1);
        const uint32_t w = static_cast<uint32_t>(mw[j] >> (8 * n + 2 * tq));
        ones[i] = (w & 1u ? 0x3F80u : 0u) | (w & 2u ? 0x3F800000u : 0u);
      }
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        uint32_t b[4];
        ldsm_x4_trans(at + v_row + 16 * kk * kAgainPitch + 32 * n, b);
        if (special) {
          uint32_t up[4], down[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) apart(b[i], b[i], up[i], down[i]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float plus[4] = {0.f, 0.f, 0.f, 0.f}, minus[4] = {0.f, 0.f, 0.f, 0.f};
            mma_bf16_16816(plus, ones, up[2 * h], up[2 * h + 1]);
            mma_bf16_16816(minus, ones, down[2 * h], down[2 * h + 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (plus[i] > 0.f) o[2 * n + h][i] += INFINITY;
              if (minus[i] > 0.f) o[2 * n + h][i] -= INFINITY;
            }
          }
        }
        mma_bf16_16816(o[2 * n], a, b[0], b[1]);
        mma_bf16_16816(o[2 * n + 1], a, b[2], b[3]);
      }
    }
    // (the buffer is free for the step after the next; rows that are all NaN are done)
    bool done = true;
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) done &= o[n][i] != o[n][i] || !again[i >> 1];
    if (softmax_all(done)) break;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");  // (those of a step that was not taken)
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 1);
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 2);
    if (!again[j]) continue;
    const float inv = l[j] == 0.f ? 0.f : 1.f / l[j];
    __nv_bfloat16* dst = p.out + row_of(16 * warp + gq + 8 * j) + 2 * tq;
#pragma unroll
    for (int n = 0; n < 16; ++n)
      *reinterpret_cast<uint32_t*>(dst + 8 * n) =
          pack_bf16x2(o[n][2 * j] * inv, o[n][2 * j + 1] * inv);
  }
}

// The marked items of this CTA, by the softmax warps.  (No arguments but the kernel's: with more of
// them, or called before the CTA's last barrier, long prompts took 1 % and the smallest 5 %
// more where nothing was marked.)
__device__ __noinline__ void rows_again(const Params& p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int* flags = reinterpret_cast<const int*>(smem + kMiscOff + 8);
  if (threadIdx.x < kThreads - kSoftmaxThreads || flags[0] != 0) return;
  const unsigned marked = static_cast<unsigned>(flags[1]);
  const int t = threadIdx.x - (kThreads - kSoftmaxThreads);
  const int warp = t >> 5, lane = t & 31;
  const int log2_rpb = min(p.log2_bs, kLog2Rows);
  int* misc = reinterpret_cast<int*>(smem + kAgainMisc);
  int serial = 0;  // steps of all tiles so far, for the stamps
  if (t < 8) misc[2 + t] = 0;
  Walk walk(p, blockIdx.x, lane);
  Item it;
  while (walk.get(p, gridDim.x, lane, it)) {
    if (it.nsteps == 0 ||
        (marked & item_bit(static_cast<uint32_t>(it.q_row) * p.num_q_heads + it.g * p.group)) ==
            0u)
      continue;
    softmax_barrier();  // (misc of the item before is read)
    if (t == 0) {
      misc[0] = -1;
      misc[1] = INT_MAX;
    }
    softmax_barrier();
    int newest = -1, oldest = INT_MAX;  // places of tokens with values that are not finite
    for (int v = warp; v < it.nsteps; v += kSoftmaxThreads / 32) {
      const StepRows rows(p, it, v, log2_rpb, lane);
#pragma unroll 1
      for (int r0 = 0; r0 < kStep; r0 += 16) {
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = r0 + 2 * k + (lane >> 4);
          const int64_t at = rows.offset(p, r, log2_rpb);
          x[k] = make_uint4(0u, 0u, 0u, 0u);
          if ((rows.seen >> r) & 1ull)
            x[k] = __ldg(reinterpret_cast<const uint4*>(p.v_cache + at) + (lane & 15));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int place = v * kStep + r0 + 2 * k + (lane >> 4);
          if (not_finite(x[k].x) || not_finite(x[k].y) || not_finite(x[k].z) ||
              not_finite(x[k].w)) {
            newest = max(newest, place);
            if (place >= p.num_sink) oldest = min(oldest, place);
          }
        }
      }
    }
    newest = __reduce_max_sync(0xffffffffu, newest);
    oldest = __reduce_min_sync(0xffffffffu, oldest);
    if (lane == 0) {
      atomicMax(&misc[0], newest);
      atomicMin(&misc[1], oldest);
    }
    softmax_barrier();
    newest = *const_cast<volatile int*>(&misc[0]);
    oldest = *const_cast<volatile int*>(&misc[1]);
    for (int i = 0; i < it.nq; ++i) {
      const int first = it.pos0 + i * p.tokens_per_tile;
      const int last = it.pos0 + min((i + 1) * p.tokens_per_tile, it.ntok) - 1;
      if (newest > first || oldest <= last - p.window)
        tile_again(p, smem, it, i, newest, oldest, serial);
    }
  }
}

// A wait of the issuing warp that is not over at once.  A call: the loop in line at each of its
// waits cost 1% to 3%, as instructions between those that are needed.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, int* flags) {
  return mbar_wait_bounded(bar, parity, flags);
}

// kPositive: scale > 0, which goes into the exponentials' products; else scores are multiplied
// first (64 products a step; where they are not used their instructions alone cost 1% of a long
// prompt)
template <bool kPositive>
__global__ void __launch_bounds__(kThreads, 1)
    window_prefill_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const Params p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
  uint64_t* q_full = bars;                    // [2] query tile i landed
  uint64_t* q_empty = bars + 2;               // [2] its last score product done (commit)
  uint64_t* pv_done = bars + 4;               // [2] an output product into O_i done (commit)
  uint64_t* o_empty = bars + 6;               // [2] O_i read (4 warps)
  uint64_t* s_full = bars + 8;                // [2][2] scores of buffer b there (commit)
  uint64_t* p_full = bars + 12;               // [2][2] weights in buffer b (4 warps)
  uint64_t* k_full = bars + 16;               // [kSlots] keys landed
  uint64_t* k_empty = k_full + kSlots;        // [kSlots] their score products done (commit)
  uint64_t* v_full = k_empty + kSlots;        // [kSlots] values landed
  uint64_t* v_empty = v_full + kSlots;        // [kSlots] their output products done (commit)
  uint64_t* drain = v_empty + kSlots;         // every product done
  volatile uint64_t* step_mask =
      reinterpret_cast<volatile uint64_t*>(smem + kMaskOff);  // [kMaskSlots]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kMiscOff);
  int* flags = reinterpret_cast<int*>(smem + kMiscOff + 8);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int step = gridDim.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_empty[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(drain, 1);
    flags[0] = flags[1] = 0;
    mbar_init_fence();
  }
  if (warp == 1) {  // this warp owns the CTA's tensor memory
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __reduce_or_sync(0xffffffffu, *tmem_slot);
  volatile int* abort_flag = flags;
  uint32_t issued = 0;  // (warps 0, 3) steps whose keys, values are requested

  if (warp < 4) {
    bool ok = true;
    if (warp == 0 || warp == 3) {
      // ------------------------------------------- keys (warp 0), values (warp 3)
      const bool keys = warp == 0;
      const CUtensorMap* tm = keys ? &tm_k : &tm_v;
      uint64_t* full = keys ? k_full : v_full;
      uint64_t* empty = keys ? k_empty : v_empty;
      uint8_t* slots = smem + (keys ? kKOff : kVOff);
      Walk walk(p, blockIdx.x, lane);
      Item it;
      const uint64_t pol = l2_policy_evict_normal();
      const int log2_rpb = min(p.log2_bs, kLog2Rows);
      if (lane == 0) prefetch_tensormap(tm);
      bool have = true;
      int at = 0;
      it.nsteps = 0;
      // the next step's pieces, looked up before the wait for a slot
      auto next = [&]() {
        while (at == it.nsteps) {
          have = walk.get(p, step, lane, it);
          at = 0;
          if (!have) return Pieces{-1, 0, 0, 0};
        }
        return find_pieces(p, it, at++ * kStep, log2_rpb, lane);
      };
      Pieces x = next();
      while (have) {
        const Pieces now = x;
        x = next();
        const bool there =
            now.bid >= 0 && static_cast<int64_t>(now.bid) < p.num_blocks && now.seen != 0;
        const uint32_t n = issued;
        const uint32_t slot = n % kSlots;
        if (n >= kSlots) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded_long(&empty[slot], (n / kSlots - 1) & 1,
                                                              abort_flag));
          if (!ok) break;
        }
        if (keys) {
          const uint64_t seen = there ? now.seen : 0;
          const uint32_t w0 = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(seen));
          const uint32_t w1 = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(seen >> 32));
          // (read once the scores are there, which wait for the keys, asked for after this)
          if (lane == 0) step_mask[n % kMaskSlots] = (static_cast<uint64_t>(w1) << 32) | w0;
        }
        load_step(tm, there ? now.bid * p.block_size + now.row : -1, now.g,
                  slots + slot * kSlotBytes, &full[slot], log2_rpb, pol, lane);
        ++issued;
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------- queries
      Walk walk(p, blockIdx.x, lane);
      Item it;
      const uint64_t pol = l2_policy_evict_first();
      if (lane == 0) prefetch_tensormap(&tm_q);
      uint32_t count[2] = {0, 0};
      while (ok && walk.get(p, step, lane, it)) {
        if (it.nsteps == 0) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i >= it.nq) break;
          if (count[i] > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded_long(&q_empty[i], (count[i] - 1) & 1,
                                                                abort_flag));
            if (!ok) break;
          }
          if (lane == 0) {
            uint8_t* dst = smem + kQOff + i * 2 * kChunk;
            const int32_t row = it.q_row + i * p.tokens_per_tile;
            mbar_arrive_expect_tx(&q_full[i], 2 * kChunk);
            tma_load_3d(dst, &tm_q, 0, it.g * p.group, row, &q_full[i], pol);
            tma_load_3d(dst + kChunk, &tm_q, 64, it.g * p.group, row, &q_full[i], pol);
          }
          ++count[i];
        }
      }
      // the last copies are waited for before this warp ends, whoever gave up
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (count[i] > 0) mbar_wait_bounded_long(&q_full[i], (count[i] - 1) & 1, nullptr);
    } else if (warp == 1) {
      // ------------------------------------------------------------ products
      // Descriptors: the low words differ by (byte offset >> 4), the high words are
      // fixed, so that a product costs one addition.
      const uint64_t base = smem_desc(smem_u32(smem), 16, 1024);
      const uint32_t lo_kmajor = static_cast<uint32_t>(base);
      const uint32_t hi_word = static_cast<uint32_t>(base >> 32);
      // V is MN-major: leading offset = the next 64 elements
      const uint32_t lo_v = static_cast<uint32_t>(smem_desc(smem_u32(smem), kHalf, 1024));
      const uint32_t one = elect_one();
      auto wait = [&](uint64_t* bar, uint32_t n) {
        if (ok && !__all_sync(0xffffffffu, mbar_try_wait(bar, n & 1)))
          ok = __all_sync(0xffffffffu, wait_on(bar, n & 1, flags));
      };
      // A cursor over the steps of all items; scores run two steps ahead of outputs, so each
      // has its own.  (What a walk says comes by a reduction, whose result is known to
      // be the same in every lane.)
      struct Cursor {
        int step, nsteps, nq;  // of the item in hand; nsteps 0: no more
        uint32_t n;            // steps before it
        uint32_t steps[2];     // the same per query tile
        uint32_t items[2];     // items begun per query tile
      };
      Walk walk(p, blockIdx.x, lane);
      // the item after the scores' one as 4 steps + query tiles; 0: none, -1: not known yet
      int after = -1;
      auto look_ahead = [&]() {
        Item x;
        if (after >= 0) return;
        after = 0;
        while (after == 0 && walk.get(p, step, lane, x))
          if (x.nsteps > 0) after = __reduce_max_sync(0xffffffffu, 4 * x.nsteps + x.nq);
      };
      int begun[2] = {0, 0};  // items that the scores have come to and the outputs have not
      auto take = [&](Cursor& c, int item) {
        c.step = 0;
        c.nsteps = item >> 2;
        c.nq = item & 3;
      };
      Cursor sc{0, 0, 0, 0, {0, 0}, {0, 0}};
      auto next_scores = [&]() {
        look_ahead();
        take(sc, after);
        if (begun[0] == 0) {
          begun[0] = after;
        } else {
          begun[1] = after;
        }
        if (after > 0) after = -1;
      };
      auto advance_scores = [&]() {
        ++sc.n;
        if (++sc.step == sc.nsteps) next_scores();
      };
      Cursor pv = sc;
      auto next_outputs = [&]() {
        take(pv, begun[0]);
        begun[0] = begun[1];
        begun[1] = 0;
      };
      auto advance_outputs = [&]() {
        ++pv.n;
        if (++pv.step == pv.nsteps) next_outputs();
      };
      next_scores();
      next_outputs();
      // What is known of the barriers that come next (see Tests)
      Tests tests{};
      bool have_p[2] = {false, false}, have_k = false, have_v = false;
#pragma unroll
      for (int t = 0; t < 3; ++t) tests.bar[t] = smem_u32(drain);
      auto test_weights = [&](int i, uint32_t n) {
        tests.bar[0] = smem_u32(&p_full[2 * i + (n & 1)]);
        tests.parity[0] = (n >> 1) & 1;
      };
      auto test_loads = [&](uint32_t k, uint32_t v) {
        tests.bar[1] = smem_u32(&k_full[k % kSlots]);
        tests.parity[1] = (k / kSlots) & 1;
        tests.bar[2] = smem_u32(&v_full[v % kSlots]);
        tests.parity[2] = (v / kSlots) & 1;
      };
      // S_i of a step (the n-th) with the keys of slot k, into buffer n % 2
      auto score = [&](int i, uint32_t n, uint32_t k) {
        const uint32_t buf = n & 1;
        score_product(one, tmem + kSCol + 2 * kStep * i + kStep * buf,
                      lo_kmajor + (kQOff + i * 2 * kChunk) / 16,
                      lo_kmajor + (kKOff + (k % kSlots) * kSlotBytes) / 16, hi_word, kIdescS,
                      tests);
        commit(one, &s_full[2 * i + buf]);
      };
      // O_i += P_i V: 4 k-steps of 16 keys; P_i from TMEM (bf16 pairs, 8 columns per k-step), V
      // MN-major (stride offset: next 8 keys = 1 KB)
      auto output = [&](int i, uint32_t n, uint32_t v, bool add) {
        const uint32_t pc = tmem + kSCol + 2 * kStep * i + kStep * (n & 1);
        const uint32_t vd = lo_v + (kVOff + (v % kSlots) * kSlotBytes) / 16;
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          mma_ts(one, tmem + kOCol + kD * i, pc + 8 * kk, vd + kk * 2048 / 16, hi_word, kIdescPV,
                 add || kk > 0 ? 1u : 0u);
        commit(one, &pv_done[i]);
      };
      // the scores of cursor sc's step in query tile i
      auto next_score = [&](int i) {
        if (sc.step == 0) {
          wait(&q_full[i], sc.items[i]++);
          tc_fence_after();
        }
        if (!ok) return;
        score(i, sc.steps[i]++, sc.n);
        if (sc.step + 1 == sc.nsteps) commit(one, &q_empty[i]);
        if (i + 1 == sc.nq) commit(one, &k_empty[sc.n % kSlots]);
      };
      for (int ahead = 0; ahead < 2; ++ahead) {
        if (ok && sc.nsteps > 0) {
          wait(&k_full[sc.n % kSlots], sc.n / kSlots);
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (i < sc.nq) next_score(i);
          advance_scores();
        }
      }
      while (ok && pv.nsteps > 0) {
        // In the middle of an item, where neither cursor comes to its end, a step is this:
        if (pv.nq == 2 && pv.step > 0 && sc.step == pv.step + 2) {
          uint32_t k = sc.n, v = pv.n, n0 = pv.steps[0], n1 = pv.steps[1];
          const int steps = sc.nsteps - 1 - sc.step;
          for (int left = steps; ok && left > 0; --left) {
            if (!have_v) wait(&v_full[v % kSlots], v / kSlots);
            if (!have_k) wait(&k_full[k % kSlots], k / kSlots);
            if (!have_p[0]) wait(&p_full[n0 & 1], n0 >> 1);
            tc_fence_after();
            if (!ok) break;
            output(0, n0, v, true);
            test_weights(1, n1);
            score(0, n0, k);
            ++n0;
            if (!__all_sync(0xffffffffu, tests.done[0])) wait(&p_full[2 + (n1 & 1)], n1 >> 1);
            tc_fence_after();
            if (!ok) break;
            output(1, n1, v, true);
            commit(one, &v_empty[v % kSlots]);
            test_weights(0, n0);
            test_loads(k + 1, v + 1);
            score(1, n1, k);
            commit(one, &k_empty[k % kSlots]);
            ++n1, ++k, ++v;
            have_p[0] = __all_sync(0xffffffffu, tests.done[0]);
            have_k = __all_sync(0xffffffffu, tests.done[1]);
            have_v = __all_sync(0xffffffffu, tests.done[2]);
          }
          if (!ok) break;
          if (steps > 0) {
            sc.n = k, pv.n = v;
            sc.steps[0] = sc.steps[0] + (n0 - pv.steps[0]);
            sc.steps[1] = sc.steps[1] + (n1 - pv.steps[1]);
            pv.steps[0] = n0, pv.steps[1] = n1;
            sc.step += steps, pv.step += steps;
          }
        }
        if (!have_v) wait(&v_full[pv.n % kSlots], pv.n / kSlots);
        if (pv.step == 0) {
          look_ahead();  // (a wait follows in any case)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i < pv.nq) {
              if (pv.items[i] > 0) wait(&o_empty[i], pv.items[i] - 1);
              ++pv.items[i];
            }
          }
        }
        if (sc.nsteps > 0 && !have_k) wait(&k_full[sc.n % kSlots], sc.n / kSlots);
        have_k = have_v = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i < pv.nq) {
            const uint32_t n = pv.steps[i]++;
            if (!have_p[i]) wait(&p_full[2 * i + (n & 1)], n >> 1);
            have_p[i] = false;
            tc_fence_after();
            if (ok) {
              output(i, n, pv.n, pv.step > 0);
              if (i + 1 == pv.nq) commit(one, &v_empty[pv.n % kSlots]);
            }
          }
          if (i < sc.nq && ok) {
            const bool other = i == 0 && pv.nq == 2;
            test_weights(other ? 1 : 0, other ? pv.steps[1] : pv.steps[0]);
            test_loads(sc.n + 1, pv.n + 1);
            next_score(i);
            const bool there = __all_sync(0xffffffffu, tests.done[0]);
            if (other) {
              have_p[1] = there;
            } else {
              have_p[0] = there;
            }
            if (i + 1 == sc.nq) {
              have_k = __all_sync(0xffffffffu, tests.done[1]);
              have_v = __all_sync(0xffffffffu, tests.done[2]);
            }
          }
        }
        advance_outputs();
        if (sc.nsteps > 0) advance_scores();
      }
      __syncwarp();
      commit(one, drain);
      mbar_wait_bounded(drain, 0, nullptr);
      __syncwarp();
    }
    if (!__all_sync(0xffffffffu, ok) && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.err, PA_DEVERR_WAIT_TIMEOUT);
    }
  } else {
    // --------------------------------------------------------------- softmax
    const int qi = (warp - 4) >> 2;
    const int quad = warp & 3;
    const int row = 32 * quad + lane;  // = TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t s_addr = tmem + lane_addr + kSCol + 2 * kStep * qi;
    const uint32_t o_addr = tmem + lane_addr + kOCol + kD * qi;
    const int G = p.group;
    const int tok = qi * p.tokens_per_tile + row / G;  // the row's token among the item's
    const float sc = kPositive ? p.scale_log2 : 1.f;
    Walk walk(p, blockIdx.x, lane);
    Item it;
    bool scores = false;  // (of the next step are there)
    uint32_t u = 0, mine = 0;  // steps of the CTA before the item, of this query tile
    bool ok = true;
    bool have = walk.get(p, step, lane, it);
    while (ok && have) {
      if (qi >= it.nq) {
        u += it.nsteps;
        have = walk.get(p, step, lane, it);
        continue;
      }
      const bool rvalid = tok < it.ntok;
      const int pos = it.pos0 + tok;
      const int low = pos - p.window + 1;  // the row's window starts here
      const int64_t qrow = (static_cast<int64_t>(it.q_row + (rvalid ? tok : 0)) * p.num_q_heads +
                            it.g * G + row % G) *
                           kD;
      float m_run = -INFINITY, l_run = 0.f;
      for (int v = 0; v < it.nsteps; ++v, ++mine) {
        const uint32_t n = u + v;
        const uint32_t buf = mine & 1;
        if (!__all_sync(0xffffffffu, scores)) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s_full[2 * qi + buf], (mine >> 1) & 1,
                                                         abort_flag));
          if (!ok) break;
        }
        const uint64_t seen = step_mask[n % kMaskSlots];
        tc_fence_after();
        float s[kStep];
        const uint32_t sb = s_addr + kStep * buf;
        tc_ld32_nowait(sb, &s[0]);
        tc_ld32_nowait(sb + 32, &s[32]);
        tc_wait_ld();
        if constexpr (!kPositive) {
#pragma unroll
          for (int c = 0; c < kStep; ++c) s[c] *= p.scale_log2;
        }
        // places up to the row's own, from its window's first on or of first tokens
        // (places between the first tokens and the item's window are not in the mask)
        const int k0 = v * kStep;
        uint64_t mw = seen;
        if (k0 + kStep - 1 > pos || (k0 < low && k0 + kStep > p.num_sink))
          mw &= WindowRange::below(pos + 1 - k0) &
                (~WindowRange::below(low - k0) | WindowRange::below(p.num_sink - k0));
        if (!rvalid) mw = 0ull;
        if (mw != ~0ull) {
          const uint32_t w[2] = {static_cast<uint32_t>(mw), static_cast<uint32_t>(mw >> 32)};
#pragma unroll
          for (int c = 0; c < kStep; ++c)
            if (!((w[c >> 5] >> (c & 31)) & 1u)) s[c] = -INFINITY;
        }
        float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kStep; c += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) mq[i] = fmax3(mq[i], s[c + 2 * i], s[c + 2 * i + 1]);
        }
        const float mx_raw = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
        const float mx = kPositive ? mx_raw * p.scale_log2 : mx_raw;
        // lazy rescale; tcgen05.ld/st are warp-wide, so the warp rescales together when any
        // of its rows needs it (the others by 1), once the output product before is done
        const bool need = mx > m_run + kRescaleLog2;
        if (__any_sync(0xffffffffu, need)) {
          const float corr = need ? fast_exp2(m_run - mx) : 1.f;
          if (v > 0) {
            ok = __all_sync(0xffffffffu,
                            mbar_wait_bounded(&pv_done[qi], (mine - 1) & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kD; c += 32) {
              float o[32];
              tc_ld32(o_addr + c, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= corr;
              tc_st32u_nowait(o_addr + c, reinterpret_cast<const uint32_t*>(&o[0]));
            }
            tc_wait_st();
          }
          if (need) {
            l_run *= corr;
            m_run = mx;
          }
        }
        // weights 2^(s * scale - m) as bf16 pairs: the A operand of P.V_i, keys 2j, 2j + 1
        // in column j.  A masked score is -inf and 2^-inf = +0 (m is taken as 0 while the
        // row has seen no key, so no -inf + inf)
        const float2 sc2 = make_float2(sc, sc);
        const float mneg = m_run == -INFINITY ? 0.f : -m_run;
        const float2 mn2 = make_float2(mneg, mneg);
        float2 lq[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t pr[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 x = ffma2(make_float2(s[2 * i], s[2 * i + 1]), sc2, mn2);
          const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          lq[i & 1] = fadd2(lq[i & 1], e);
          pr[i] = pack_bf16x2(e.x, e.y);
          if (i == 15) st16(sb, pr);
        }
        st16(sb + 16, pr + 16);
        l_run += (lq[0].x + lq[0].y) + (lq[1].x + lq[1].y);
        // (tested meanwhile: the next step's scores)
        scores = wait_st_and_test(&s_full[2 * qi + (buf ^ 1)], ((mine + 1) >> 1) & 1);
        // keys without a cache row: zero their value rows (0 x NaN would poison P.V), by
        // query tile 0's threads (P.V_1(v) follows P.V_0(v)): (key row / 2, chunk row % 2)
        if (qi == 0 && seen != ~0ull) {
          const uint32_t slot = n % kSlots;
          ok = __all_sync(0xffffffffu,
                          mbar_wait_bounded(&v_full[slot], (n / kSlots) & 1, abort_flag));
          if (!ok) break;
          if (!((seen >> (row >> 1)) & 1ull)) {
            uint4* dst = reinterpret_cast<uint4*>(smem + kVOff + slot * kSlotBytes +
                                                  (row & 1) * kHalf + (row >> 1) * 128);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();  // generic writes before the tensor core reads them
        }
        // The wait for the item's last output product tells one phase from the next only, so the
        // product before it must be done by then: waited for while the last cannot begin.
        if (v > 0 && v + 1 == it.nsteps) {
          ok = __all_sync(0xffffffffu,
                          mbar_wait_bounded(&pv_done[qi], (mine - 1) & 1, abort_flag));
          if (!ok) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * qi + buf]);
      }
      if (!ok) break;
      u += it.nsteps;
      const bool none = it.nsteps == 0;
      have = walk.get(p, step, lane, it);  // (the next item, while the last product runs)
      if (none) {
        if (rvalid) {  // no key at all: a zero row
          uint4* dst = reinterpret_cast<uint4*>(p.out + qrow);
#pragma unroll
          for (int c = 0; c < kD / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      // ---- the item's end: this thread's output row
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&pv_done[qi], (mine - 1) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
      float o[kD];
#pragma unroll
      for (int c = 0; c < kD; c += 32) tc_ld32_nowait(o_addr + c, &o[c]);
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[qi]);
      float nan_max = -INFINITY;  // NaN where an element is
#pragma unroll
      for (int c = 0; c < kD; c += 2) nan_max = max3_nan(nan_max, o[c], o[c + 1]);
      const bool nan_row = nan_max != nan_max;
      // A thread's row is 256 bytes, far from the next one's: half rows go through shared
      // memory (16-byte unit c of row r at c ^ (r & 7)), and the warp stores four rows
      // (128-byte lines) at a time instead of 32 pieces of 16 bytes.
      uint8_t* stage = smem + kStageOff + (warp - 4) * kStageBytes;
      const int64_t out_row = rvalid ? qrow : -1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float* x = &o[64 * h + 8 * c];
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) =
              make_uint4(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv),
                         pack_bf16x2(x[4] * inv, x[5] * inv), pack_bf16x2(x[6] * inv, x[7] * inv));
        }
        __syncwarp();
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 4) {
          const int r = r0 + (lane >> 3), c = lane & 7;
          const int64_t to = __shfl_sync(0xffffffffu, out_row, r);
          const uint4 x = *reinterpret_cast<const uint4*>(stage + r * 128 + ((c ^ (r & 7)) << 4));
          if (to >= 0) *reinterpret_cast<uint4*>(p.out + to + 64 * h + 8 * c) = x;
        }
      }
      if (nan_row && rvalid && l_run == l_run)
        atomicOr(reinterpret_cast<unsigned*>(&flags[1]),
                 item_bit(static_cast<uint32_t>(qrow / kD) -
                          static_cast<uint32_t>(tok) * p.num_q_heads - row % G));
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.err, PA_DEVERR_WAIT_TIMEOUT);
    }
  }

  // ---- end: drain on error, free TMEM
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if ((warp == 0 || warp == 3) && lane == 0) {
      for (uint32_t t = issued > kSlots ? issued - kSlots : 0; t < issued; ++t)
        mbar_wait_bounded(&(warp == 0 ? k_full : v_full)[t % kSlots], (t / kSlots) & 1, nullptr);
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
  if (flags[1] != 0) rows_again(p);
}

// [T, H_Q, 128] bf16; box = 64 elements x G heads x 128 / G tokens: the 128 rows of a
// query tile, tokens slowest
bool make_q_map(CUtensorMap* map, const void* base, int64_t tokens, int32_t heads, int32_t group) {
  auto enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kD) * 2,
                                 static_cast<cuuint64_t>(kD) * 2 * heads};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(group),
                             static_cast<cuuint32_t>(kM / group)};
  const cuuint32_t es[3] = {1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kPositive>
pa_status launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                 const Params& p, unsigned grid, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_raised{0};
  if (!ensure_smem_limit(window_prefill_kernel<kPositive>, kAlloc, smem_raised)) return PA_ERR_CUDA;
  window_prefill_kernel<kPositive><<<grid, kThreads, kAlloc, stream>>>(mq, mk, mv, p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

pa_status launch_window_prefill(const WindowPrefillArgs& w, cudaStream_t stream) {
  const PrefillArgs& a = w.p;
  if (a.num_seqs == 0 || a.max_q_len == 0 || w.total_tokens == 0) return PA_OK;
  const int32_t G = a.num_q_heads / a.num_kv_heads;
  const int64_t rows = a.num_blocks * a.block_size;
  const int32_t box_rows = a.block_size < kStep ? a.block_size : kStep;
  CUtensorMap mq, mk, mv;
  if (!make_q_map(&mq, a.q, w.total_tokens, a.num_q_heads, G) ||
      !make_kv_map_swizzled(&mk, a.k_cache, rows, a.num_kv_heads, box_rows) ||
      !make_kv_map_swizzled(&mv, a.v_cache, rows, a.num_kv_heads, box_rows))
    return PA_ERR_CUDA;
  Params p;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k_cache = static_cast<const __nv_bfloat16*>(a.k_cache);
  p.v_cache = static_cast<const __nv_bfloat16*>(a.v_cache);
  p.block_tables = a.block_tables;
  p.cu_seqlens_q = a.cu_seqlens_q;
  p.context_lens = a.context_lens;
  p.err = a.error_word;
  p.num_blocks = a.num_blocks;
  p.num_seqs = a.num_seqs;
  p.total_tokens = static_cast<int32_t>(w.total_tokens);
  p.max_q_len = a.max_q_len;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = G;
  p.tokens_per_tile = kM / G;
  p.block_size = a.block_size;
  p.log2_bs = 0;
  while ((1 << p.log2_bs) < a.block_size) ++p.log2_bs;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.window = w.window;
  p.num_sink = w.num_sink;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  // one CTA per SM, no more than there can be items
  int64_t grid = num_sms_current_device();
  if (grid <= 0) grid = 148;
  const int64_t per = 2 * p.tokens_per_tile;
  const int64_t longest = a.max_q_len < w.total_tokens ? a.max_q_len : w.total_tokens;
  const int64_t most = (longest + per - 1) / per * a.num_seqs;
  if (most < grid && most * a.num_kv_heads < grid) grid = most * a.num_kv_heads;
  if ((w.total_tokens / per + a.num_seqs) * a.num_kv_heads > kMaxItems) return PA_ERR_UNSUPPORTED;
  return p.scale_log2 > 0.f ? launch<true>(mq, mk, mv, p, static_cast<unsigned>(grid), stream)
                            : launch<false>(mq, mk, mv, p, static_cast<unsigned>(grid), stream);
}

}  // namespace pa_detail
