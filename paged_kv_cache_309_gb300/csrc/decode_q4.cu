// decode_q4.cu -- paged GQA decode attention over a 4-bit cache.
//
// Rows are 80 bytes: 64 of codes, then four fp16 pairs (s, m), one per group u
// of 32 elements; an element stands for m + s c.
//
// Scores.  With S_u = sum_{d in u} q_d c_d and Q_u = sum_{d in u} q_d,
//     q . k = sum_u s_u S_u + m_u Q_u.
// A nibble at bits 0-3 (4-7) of a 16-bit half is, read as an fp16 number,
// the subnormal c 2^-24 (c 2^-20): one AND turns two nibbles of a code word
// into an fp16 pair, exactly, and the factors 2^24 and 16 go into the score
// scale and into q.  The products are exact and accumulate in fp32; s enters
// in fp32.  The minima's sum is one more product, the rows' (s, m) pairs
// times (0, Q_u), with Q_u as the sum of two fp16 numbers.
//
// Values.  ldmatrix.trans hands a lane the 16-bit units (four codes) of two
// tokens side by side, so one AND-OR per nibble makes the fp16 pair
// (64 + c) of both tokens (bits 4-7 of an fp16 in [64, 128) count units) and
// one fused multiply-add with (s, -64 s) the pair s c, rounded once.  The
// minima again cost one product: sum_t p_t m_t,u, with the (s, m) pairs of
// the rows as the matrix (rows 2u + 1 of its result).  The weights are held
// 2^7 above the running maximum's scale, so that fp16 carries them down to 2^-31 of it.
//
// Rows of 80 bytes need no swizzle: eight consecutive rows start in eight
// different groups of four banks (20 r mod 32).  The 160 bytes of two kv heads
// would start in four, so their boxes are 176 bytes wide (44 r mod 32; the last
// 16 bytes are the next head's or past the row, and unused): shared memory was
// 66% busy with 160.
//
// What bounds it: at 160 bytes per token and kv head HBM leaves an SM 440
// issue slots for 16 tokens, and the first form of this kernel needed 431 of
// them (0.54 of the copy rate at B = 8, 32K-128K).  So the element work is
// the forms above, 32 tokens share one vote on a new running maximum (the
// shuffles run only when a score beats the old one by 2^8), and the prologue
// and epilogue run once per piece of a balanced cut instead of once per short
// token range.  With 296 instructions for 16 tokens the copies alone take 137
// us there, the computation alone 137 and both together 143 (0.87 of the
// copy rate; B = 64, 512-4096: 41, 43 and 45; there a CTA spends 2 us on the
// cut and some 1.6 on the end of each piece).  The cut:
//   the sequences' units of 64 tokens lie end to end, every sequence start
//   charged kPieceCost units more; chunk c of C (C x H_KV CTAs fill the GPU
//   once) is the units whose cost lies in [c, c + 1) total / C.  A chunk
//   walks its pieces with the ring running on across them.  A sequence that
//   lies in one chunk is written directly; the pieces of one that does not
//   go to partial slots, which a second launch merges with one CTA per query
//   head (a single long sequence has up to 200 pieces; with the CTA that finished
//   last merging all its 16 query heads a scored call over 9001 tokens took 54
//   us, so 19).  Its CTAs are launched while this kernel runs and wait for its
//   end (programmatic dependent launch).
//
// Every mbarrier wait is bounded (2 s); after a timeout the error bit is
// set, the remaining pieces end empty, the copies in flight are waited for, and
// the CTA exits.
#include <atomic>
#include <type_traits>

#include "pa_internal.cuh"
#include "q4_cut.h"

namespace pa_detail {

using namespace pa;
using namespace decode;
using namespace q4cut;

namespace {

static_assert(kUnit == 64, "boxes are up to 64 rows, pieces start at multiples of them");
static_assert(kPartialFloats == kD, "a partial row is a head");
constexpr int kRow = 80;           // bytes of a cached row of one kv head
constexpr int kStageRows = 128;    // head rows per stage, 32 per consumer warp
constexpr float kLift = 7.0f;      // weights are 2^kLift (score - running maximum)
constexpr int kConsumers = kConsumerWarps * 32;

struct Q4Params {
  DecodeParams d;
  int32_t num_seqs;
  int32_t slots;  // partial slots per kv head
  int32_t* info;  // [H_KV / HP, B]: chunk of the first piece << 16 | pieces, 0 if not split
  bool whole;     // no partials: chunks begin at sequence starts
  int32_t log2_g;       // of the query heads per kv head
  int32_t pair_tokens;  // 1: the maps' rows are pairs of tokens (one kv head)
};

template <int NT, int HP>
struct Lay {
  // 16 heads (B = 8, 16K-64K, 4 kv heads): two CTAs with 168 registers and some
  // spills take 68 us, one without spills 77 (six stages: 78), three 90, two with
  // four stages 69
  static constexpr int kStages = 3;
  static constexpr int kCtasPerSm = NT == 1 ? 3 : 2;
  static constexpr int kTile = kStageRows / HP;        // tokens per stage
  static constexpr int kPitch = HP == 2 ? 176 : kRow;  // bytes of a token in a stage
  static constexpr int kTensorBytes = kTile * kPitch;
  static constexpr int kStageBytes = 2 * kTensorBytes;  // K rows, then V rows
  static constexpr int kHeads = NT * 8;
  // the join of a head's warps: 32 elements of every head of a warp at a time (more
  // where G is less than kHeads), then maxima and sums [warp][h]
  static constexpr int kRedOffset = kStages * kStageBytes;
  static constexpr int kRedFloats = kConsumerWarps * kHeads * 32;
  static constexpr int kStatOffset = kRedOffset + kRedFloats * 4;
  static constexpr int kStatFloats = 2 * kConsumerWarps * kHeads;
  static constexpr int kBarOffset = kStatOffset + kStatFloats * 4;
  static constexpr int kMaskOffset = kBarOffset + 2 * kStages * 8;  // four words per stage
  static constexpr int kSchedOffset = kMaskOffset + kStages * 16;   // five 64-bit words
  static constexpr int kFlagOffset = kSchedOffset + 40;
  static constexpr int kAlloc = kFlagOffset + 8 + 128;  // room to align the base to 128 bytes
  static_assert(kBarOffset % 8 == 0 && kMaskOffset % 16 == 0 && kSchedOffset % 8 == 0, "aligned");
  static_assert(kAlloc * kCtasPerSm + kCtasPerSm * 1024 <= 228 * 1024, "resident CTAs fit");
};

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// the low half of an fp16 pair in fp32
__device__ __forceinline__ float low_f32(uint32_t h) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
}
// (a & b) | c in one instruction (two constants in the expression make two)
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// 8x8 transpose of a 16-bit fragment across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
// a product that starts its sums
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void consumer_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
}

// ------------------------------------------------------------ the balanced cut --
// (the arithmetic and its invariants: q4_cut.h)
__device__ __forceinline__ int units_of(const DecodeParams& p, int b) {
  bool clipped;
  return units_of_len(effective_len(p, b, &clipped));
}

// Warp 0: the first unit of chunks c and c + 1.  sched: total, first unit of c,
// first unit of c + 1, then the first one's sequence and the units before that.
__device__ __forceinline__ void find_chunk(const Q4Params& q, int c, int chunks, int lane,
                                           int64_t* sched) {
  const DecodeParams& p = q.d;
  if (q.whole && chunks == q.num_seqs) {  // one sequence per chunk: nothing to cut
    bool clipped;
    const int n = units_of_len(effective_len(p, c, &clipped));
    if (clipped && blockIdx.x == 0 && lane == 0) atomicOr(p.err, PA_DEVERR_CONTEXT_CLIPPED);
    if (lane == 0) {
      sched[0] = 1;
      sched[1] = 0;
      sched[2] = n;
      sched[3] = c;
      sched[4] = 0;
    }
    return;
  }
  int64_t units = 0;
  bool any_clipped = false;
  int held[4];  // units of sequences lane, lane + 32, ...: the lengths are read in one round
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int b = lane + 32 * k;
    held[k] = 0;
    if (b < q.num_seqs) {
      bool clipped;
      held[k] = units_of_len(effective_len(p, b, &clipped));
      any_clipped |= clipped;
    }
    units += held[k];
  }
  for (int b = lane + 128; b < q.num_seqs; b += 32) {
    bool clipped;
    units += units_of_len(effective_len(p, b, &clipped));
    any_clipped |= clipped;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) units += __shfl_xor_sync(0xffffffffu, units, off);
  if (c == 0 && blockIdx.x == 0 && any_clipped) atomicOr(p.err, PA_DEVERR_CONTEXT_CLIPPED);
  const int64_t total = total_cost(units, q.num_seqs);
  const int64_t parts = parts_of(total, chunks);
  const int64_t x0 = chunk_begin_cost(c, total, parts);
  const int64_t x1 = chunk_begin_cost(c + 1, total, parts);
  int64_t g0 = units, g1 = units, pre0 = 0;
  int b0 = q.num_seqs;
  bool found0 = c >= parts, found1 = c + 1 >= parts;
  int64_t base = 0;
  for (int first = 0; first < q.num_seqs && !(found0 && found1); first += 32) {
    const int b = first + lane;
    const int n = first == 0    ? held[0]
                  : first == 32 ? held[1]
                  : first == 64 ? held[2]
                  : first == 96 ? held[3]
                  : b < q.num_seqs ? units_of(p, b)
                                   : 0;
    int64_t incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    const int64_t pre = base + incl - n;
    if (!found0) {
      const uint32_t hit = __ballot_sync(0xffffffffu, begins_in(x0, pre, n, b, q.whole));
      if (hit != 0u) {
        const int l = __ffs(hit) - 1;
        const int64_t at = begin_unit(x0, pre, b, q.whole);
        g0 = __shfl_sync(0xffffffffu, at, l);
        pre0 = __shfl_sync(0xffffffffu, pre, l);
        b0 = first + l;
        found0 = true;
      }
    }
    if (!found1) {
      const uint32_t hit = __ballot_sync(0xffffffffu, begins_in(x1, pre, n, b, q.whole));
      if (hit != 0u) {
        const int l = __ffs(hit) - 1;
        const int64_t at = begin_unit(x1, pre, b, q.whole);
        g1 = __shfl_sync(0xffffffffu, at, l);
        found1 = true;
      }
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) {
    sched[0] = total;
    sched[1] = g0;
    sched[2] = g1;
    sched[3] = b0;
    sched[4] = pre0;
  }
}

// A chunk's pieces in order.
struct Walk {
  int64_t t, end, pre;  // next unit, the chunk's end, units before sequence b
  int b;
  __device__ __forceinline__ explicit Walk(const int64_t* sched)
      : t(sched[1]), end(sched[2]), pre(sched[4]), b(static_cast<int>(sched[3])) {}
};
struct Piece {
  int b, tok_begin, tok_end;
  int64_t first, last;  // units of the whole sequence, counted over all sequences
};
__device__ __forceinline__ bool next_piece(const Q4Params& q, Walk& w, Piece& pc) {
  while (w.t < w.end) {
    bool clipped;
    const int L = effective_len(q.d, w.b, &clipped);
    const int n = units_of_len(L);
    if (n > 0) {
      const int64_t stop = min(w.end, w.pre + n);
      pc.b = w.b;
      pc.first = w.pre;
      pc.last = w.pre + n - 1;
      pc.tok_begin = static_cast<int>(w.t - w.pre) * kUnit;
      pc.tok_end = min(static_cast<int>(stop - w.pre) * kUnit, L);
      w.t = stop;
      w.pre += n;
      ++w.b;
      return true;
    }
    ++w.b;
  }
  return false;
}

// Merge of the split sequences' partials: one CTA per query head, for every
// gridDim.y-th sequence; weights 2^(lse - max).  Warp w takes pieces w, w + 8, ...
constexpr int kMergeWarps = 8;
template <int HP, bool kScored>
__global__ void __launch_bounds__(kMergeWarps * 32)
    merge_pieces_kernel(const __grid_constant__ Q4Params qp, int G, int chunks) {
  __shared__ float4 part[kMergeWarps][32];
  __shared__ float part_w[kMergeWarps];
  const DecodeParams& p = qp.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hq = blockIdx.x, g = hq / G;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (kScored) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int b = blockIdx.y; b < qp.num_seqs; b += gridDim.y) {
    const int32_t info = __ldcg(qp.info + static_cast<int64_t>(g / HP) * qp.num_seqs + b);
    if (info == 0) continue;
    const int c_first = info >> 16, n = info & 0xFFFF;
    const int start = start_slot_of(chunks, qp.num_seqs, b, c_first);
    const int64_t at = static_cast<int64_t>(g) * qp.slots * G + hq % G;
    const float* lse = p.ws_lse + at;
    const float* o = p.ws_o + at * kD;
    auto slot = [&](int i) -> int64_t {
      return static_cast<int64_t>(i == 0 ? start : c_first + i - 1) * G;
    };
    float M = -INFINITY;  // (a NaN lse is carried to the output)
    for (int i = lane; i < n; i += 32) M = max_nan(M, __ldcg(lse + slot(i)));
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, off));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float W = 0.f;
    if (M != -INFINITY) {
      for (int i0 = warp; i0 < n; i0 += 8 * kMergeWarps) {
        float4 v[8];
        float w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int i = i0 + k * kMergeWarps;
          if (i < n) {
            v[k] = __ldcg(reinterpret_cast<const float4*>(o + slot(i) * kD) + lane);
            w[k] = exp2f(__ldcg(lse + slot(i)) - M);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (i0 + k * kMergeWarps < n) {
            W += w[k];
            acc.x += w[k] * v[k].x;
            acc.y += w[k] * v[k].y;
            acc.z += w[k] * v[k].z;
            acc.w += w[k] * v[k].w;
          }
        }
      }
    }
    part[warp][lane] = acc;
    if (lane == 0) part_w[warp] = W;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int w = 1; w < kMergeWarps; ++w) {
        const float4 v = part[w][lane];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
        W += part_w[w];
      }
      const int64_t bh = static_cast<int64_t>(b) * p.num_q_heads + hq;
      if (kScored && lane == 0) p.final_lse[bh] = W == 0.f ? -INFINITY : M + log2f(W);
      const float inv = W == 0.f ? 0.f : 1.f / W;
      *reinterpret_cast<uint2*>(p.out + bh * kD + lane * 4) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    }
    __syncthreads();
  }
}

// NT: n-tiles of 8 query heads (G <= 8 -> 1, G = 16 -> 2); HP: kv heads per
// CTA; kScored: also store the scores and each query head's log2-sum-exp.
template <int NT, int HP, bool kScored>
__global__ void __launch_bounds__(kThreads, Lay<NT, HP>::kCtasPerSm)
    paged_decode_q4_kernel(const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ Q4Params qp, int G) {
  using L_ = Lay<NT, HP>;
  const DecodeParams& p = qp.d;
  constexpr int kStages = L_::kStages;
  constexpr int kTile = L_::kTile;
  constexpr int kPitch = L_::kPitch;
  constexpr int kTensorBytes = L_::kTensorBytes;
  constexpr int kHeadWarps = kConsumerWarps / HP;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L_::kBarOffset);
  uint64_t* empty = full + kStages;
  uint32_t* tile_mask = reinterpret_cast<uint32_t*>(smem + L_::kMaskOffset);
  int64_t* sched = reinterpret_cast<int64_t*>(smem + L_::kSchedOffset);
  int* abort_ptr = reinterpret_cast<int*>(smem + L_::kFlagOffset);

  // kv heads fastest in launch order: the CTAs of one chunk read neighbouring
  // rows at the same time
  const int g0 = blockIdx.x * HP;  // the CTA's first kv head
  const int c = blockIdx.y;
  const int chunks = gridDim.y;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int bs = p.block_size;

  if (warp == 0) find_chunk(qp, c, chunks, lane, sched);
  if (threadIdx.x == 32) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kConsumerWarps);
    }
    *abort_ptr = 0;
    mbar_init_fence();
  }
  __syncthreads();
  volatile int* abort_flag = abort_ptr;
  // (the merging CTAs may take their places; they wait for this kernel's end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t total = sched[0];
  const int parts = static_cast<int>(parts_of(total, chunks));

  if (warp == kConsumerWarps) {
    // ------------------------------------------------------------ producer
    const int rpb = bs < kUnit ? bs : kUnit;  // rows per box: pieces start at multiples of 64
    const int nbox = kTile / rpb;
    const uint64_t pol = l2_policy_evict_first();
    if (lane == 0) {
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
    Walk walk(sched);
    Piece pc;
    int u = 0;  // tiles issued
    bool ok = true;
    while (ok && next_piece(qp, walk, pc)) {
      const int32_t* bt = p.block_tables + static_cast<int64_t>(pc.b) * p.max_blocks_per_seq;
      // lane i < nbox: block id of box i of the tile at tok (-1 past the piece), read one
      // tile ahead of its issue
      auto tile_bid = [&](int tok) -> int {
        const int first = tok + lane * rpb;
        return (lane < nbox && first < pc.tok_end) ? __ldg(bt + (first >> p.log2_bs)) : -1;
      };
      int bid_next = tile_bid(pc.tok_begin);
      for (int tok = pc.tok_begin; tok < pc.tok_end; tok += kTile, ++u) {
        const int stage = u % kStages;
        const int bid = bid_next;
        bid_next = tile_bid(tok + kTile);
        if (u >= kStages) {
          const bool w_ok = mbar_wait_bounded(&empty[stage], ((u / kStages) - 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, w_ok)) {
            ok = false;
            break;
          }
        }
        const int first = tok + lane * rpb;
        const int rows = lane < nbox ? min(rpb, pc.tok_end - first) : 0;
        const bool valid = rows > 0 && bid >= 0 && static_cast<int64_t>(bid) < p.num_blocks;
        uint32_t words[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int lo = max(lane * rpb - 32 * w, 0), hi = min(lane * rpb + rows - 32 * w, 32);
          uint32_t bits = 0u;
          if (valid && hi > lo)
            bits = (hi >= 32 ? 0xFFFFFFFFu : ((1u << hi) - 1u)) & ~((1u << lo) - 1u);
          words[w] = __reduce_or_sync(0xffffffffu, bits);
        }
        const uint32_t vb = __ballot_sync(0xffffffffu, valid);
        if (lane == 0) {
          *reinterpret_cast<uint4*>(tile_mask + 4 * stage) =
              make_uint4(words[0], words[1], words[2], words[3]);
          mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(__popc(vb) * rpb * kPitch * 2));
        }
        __syncwarp();
        if (valid) {
          // (a cache of one head: two tokens make one 160-byte row of the map)
          const int32_t row = (bid * bs + (first & (bs - 1))) >> qp.pair_tokens;
          uint8_t* st = smem + stage * L_::kStageBytes + lane * rpb * kPitch;
          tma_load_2d(st, &tm_k, g0 * kRow, row, &full[stage], pol);
          tma_load_2d(st + kTensorBytes, &tm_v, g0 * kRow, row, &full[stage], pol);
        }
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.err, PA_DEVERR_WAIT_TIMEOUT);
    }
    // The last copies are waited for (bounded) before this warp ends, whoever gave up:
    // consumers whose wait ran out leave with copies in flight, and the CTA's shared
    // memory must not be handed on before those have landed.
    if (lane == 0) {
      for (int t = max(0, u - kStages); t < u; ++t)
        mbar_wait_bounded_long(&full[t % kStages], (t / kStages) & 1, nullptr);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  // sequences without tokens: zero rows (chunk c takes b = c mod C)
  for (int b = c; b < qp.num_seqs; b += chunks) {
    if (units_of(p, b) == 0) {
      const int64_t row = static_cast<int64_t>(b) * p.num_q_heads + g0 * G;
      for (int i = threadIdx.x; i < HP * G * (kD / 8); i += kConsumers)
        reinterpret_cast<uint4*>(p.out + row * kD)[i] = make_uint4(0u, 0u, 0u, 0u);
      if (kScored && threadIdx.x < HP * G) p.final_lse[row + threadIdx.x] = -INFINITY;
      if (!qp.whole && threadIdx.x == 0)
        qp.info[static_cast<int64_t>(blockIdx.x) * qp.num_seqs + b] = 0;
    }
  }

  const int gq = lane >> 2;  // mma groupID
  const int tq = lane & 3;   // thread in group
  // this warp's head and tokens of a tile
  const int g = g0 + warp / kHeadWarps;
  const int hq0 = g * G;
  const int t0 = 32 * (warp % kHeadWarps);
  const uint32_t base = static_cast<uint32_t>(t0 * kPitch + warp / kHeadWarps * kRow);
  // ldmatrix rows and 16-byte columns of this lane (K and V alike): rows
  // (lane & 15), column u + (lane >> 4); the (s, m) pairs: rows (lane & 15)
  const uint32_t frag = base + static_cast<uint32_t>((lane & 15) * kPitch + 16 * (lane >> 4));
  const uint32_t meta_frag = base + static_cast<uint32_t>((lane & 15) * kPitch + 64);
  // (s, m) rows read directly: K row gq, V row 2tq
  const uint32_t k_meta = base + static_cast<uint32_t>(gq * kPitch + 64);
  const uint32_t v_meta = base + static_cast<uint32_t>(2 * tq * kPitch + 64);
  const uint32_t smem_base = smem_u32(smem);
  uint32_t magic;  // fp16 pair (64, 64), kept in a register
  asm volatile("mov.u32 %0, 0x54005400;" : "=r"(magic));
  Walk walk(sched);
  Piece pc;
  int stage = 0;  // of the next tile
  uint32_t phase = 0u;
  bool ok = true;
  while (next_piece(qp, walk, pc)) {
    float o[8][NT][4];         // head elements 32u + 4gq + 2h (+1) of m-tile 2u + h
    float z[NT][4];            // sums of p s (even rows) and p m (odd rows) per group
    float m[NT][2], l[NT][2];  // m: running maximum - kLift
    // q as the B operand: for group u a lane (head gq of the n-tile) holds
    // elements 32u + 8tq + 0..7, paired as the nibbles of a code word are:
    // (0, 4), (1, 5)/16, (2, 6), (3, 7)/16, in fp16 after a power of two per
    // head that puts its largest |q| in [2^14, 2^15).  The minima's operand:
    // (0, Q_tq) in two fp16 terms after a power of two of its own.
    uint32_t qb[NT][4][4], qz[NT][2];
    float sscale[NT][2], zscale[NT][2];  // of heads 2tq, 2tq + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + gq;
      const uint4* qrow = reinterpret_cast<const uint4*>(
          p.q + (static_cast<int64_t>(pc.b) * p.num_q_heads + hq0 + (h < G ? h : 0)) * kD);
      float qv[4][8], qs[4];
      float qmax = 0.f, zmax = 0.f;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        to_f32(Vec8<bf16>{__ldg(qrow + 4 * v + tq)}, qv[v]);
        qs[v] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (h >= G) qv[v][e] = 0.f;
          qmax = fmaxf(qmax, fabsf(qv[v][e]));
          qs[v] += qv[v][e];
        }
        qs[v] += __shfl_xor_sync(0xffffffffu, qs[v], 1);
        qs[v] += __shfl_xor_sync(0xffffffffu, qs[v], 2);
        zmax = fmaxf(zmax, fabsf(qs[v]));
      }
      qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 1));
      qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 2));
      // 14 - floor(log2(x)) for finite x > 0
      auto lift = [](float x) -> int {
        return x > 0.f && x <= 3.0e38f
                   ? min(14 - (static_cast<int>((__float_as_uint(x) >> 23) & 0xFF) - 127), 126)
                   : 0;
      };
      const int e2 = lift(qmax), ez = lift(zmax);
      const float up = ldexpf(1.0f, e2);
      const float fs = p.scale_log2 * ldexpf(1.0f, 24 - e2), fz = p.scale_log2 * ldexpf(1.0f, -ez);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sscale[nt][j] = __shfl_sync(0xffffffffu, fs, 4 * (2 * tq + j));
        zscale[nt][j] = __shfl_sync(0xffffffffu, fz, 4 * (2 * tq + j));
      }
      const float zq = (tq == 0 ? qs[0] : tq == 1 ? qs[1] : tq == 2 ? qs[2] : qs[3]) *
                       ldexpf(1.0f, ez);
      const float zhi = __half2float(__float2half_rn(zq));
      qz[nt][0] = pack_f16x2(0.f, zhi);
      qz[nt][1] = pack_f16x2(0.f, zq - zhi);
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float f = (k & 1) ? up * 0.0625f : up;
          qb[nt][v][k] = pack_f16x2(qv[v][k] * f, qv[v][k + 4] * f);
        }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nt][j] = -INFINITY;
        l[nt][j] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[nt][i] = 0.f;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) o[mt][nt][i] = 0.f;
      }
    }

    // The warp's 32 tokens of a tile, two slices of 16.  kFull: every row is a token.
    auto tile = [&](auto full_tag, const int tok, const uint32_t st, const uint32_t mask32) {
      constexpr bool kFull = decltype(full_tag)::value;
      float s[2][NT][4];  // scores of rows gq (0, 1) and gq + 8 (2, 3), heads 2tq, 2tq + 1
      bool high = false;
#pragma unroll
      for (int sl = 0; sl < 2; ++sl) {
        const uint32_t kbase = st + sl * 16 * kPitch;
        // ---- S_u = codes . q, and the minima's sum
        float su[NT][4][4], zk[NT][4];
#pragma unroll
        for (int u2 = 0; u2 < 4; u2 += 2) {
          uint32_t r[4];  // (row gq, u2), (row gq + 8, u2), (row gq, u2 + 1), (row gq + 8, u2 + 1)
          ldsm_x4(kbase + frag + 16 * u2, r);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t lo = r[2 * i], hi = r[2 * i + 1];
            const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
            const uint32_t a0[4] = {lo & 0x000F000Fu, hi & 0x000F000Fu, lo & 0x00F000F0u,
                                    hi & 0x00F000F0u};
            const uint32_t a1[4] = {lo8 & 0x000F000Fu, hi8 & 0x000F000Fu, lo8 & 0x00F000F0u,
                                    hi8 & 0x00F000F0u};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16_first(su[nt][u2 + i], a0, qb[nt][u2 + i][0], qb[nt][u2 + i][1]);
              mma_f16_16816(su[nt][u2 + i], a1, qb[nt][u2 + i][2], qb[nt][u2 + i][3]);
            }
          }
        }
        {
          uint32_t r[4];  // (s, m) of group tq, rows gq and gq + 8
          ldsm_x4(kbase + meta_frag, r);
          const uint32_t a[4] = {r[0], r[1], r[0], r[1]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16_first(zk[nt], a, qz[nt][0], qz[nt][1]);
        }
        float ss[2][4];  // s_u of rows gq, gq + 8
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 w = lds128(kbase + k_meta + 8 * i * kPitch);
          ss[i][0] = low_f32(w.x);
          ss[i][1] = low_f32(w.y);
          ss[i][2] = low_f32(w.z);
          ss[i][3] = low_f32(w.w);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float a = ss[i >> 1][0] * su[nt][0][i];
#pragma unroll
            for (int v = 1; v < 4; ++v) a = fmaf(ss[i >> 1][v], su[nt][v][i], a);
            s[sl][nt][i] = fmaf(a, sscale[nt][i & 1], zk[nt][i] * zscale[nt][i & 1]);
          }
          if (!kFull) {
            const uint32_t mask16 = mask32 >> (16 * sl);
            if (!((mask16 >> gq) & 1u)) s[sl][nt][0] = s[sl][nt][1] = -INFINITY;
            if (!((mask16 >> (gq + 8)) & 1u)) s[sl][nt][2] = s[sl][nt][3] = -INFINITY;
          }
          if constexpr (kScored)
            store_scores(p, pc.b, g, G, tok + t0 + 16 * sl, gq,
                         pc.tok_end - tok - t0 - 16 * sl, nt * 8 + 2 * tq, s[sl][nt]);
        }
      }
      // ---- running maximum: moved when a score beats it by 2^kRescaleLog2 (always on
      // the first); whether any does is one vote
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          high |= fmaxf(fmaxf(s[0][nt][j], s[0][nt][j + 2]),
                        fmaxf(s[1][nt][j], s[1][nt][j + 2])) >
                  m[nt][j] + (kLift + kRescaleLog2);
      if (__any_sync(0xffffffffu, high)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx = fmaxf(fmaxf(s[0][nt][j], s[0][nt][j + 2]),
                             fmaxf(s[1][nt][j], s[1][nt][j + 2]));
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1)
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            if (mx > m[nt][j] + (kLift + kRescaleLog2)) {
              const float corr = exp2f(m[nt][j] - (mx - kLift));
              l[nt][j] *= corr;
              z[nt][j] *= corr;
              z[nt][j + 2] *= corr;
#pragma unroll
              for (int mt = 0; mt < 8; ++mt) {
                o[mt][nt][j] *= corr;
                o[mt][nt][j + 2] *= corr;
              }
              m[nt][j] = mx - kLift;
            }
          }
        }
      }
#pragma unroll
      for (int sl = 0; sl < 2; ++sl) {
        const uint32_t vbase = st + kTensorBytes + sl * 16 * kPitch;
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = ex2(s[sl][nt][i] - m[nt][i & 1]);
          if (!kFull) {  // (a head without a maximum yet: -inf - -inf)
            const uint32_t mask16 = mask32 >> (16 * sl);
            if (!((mask16 >> gq) & 1u)) e[0] = e[1] = 0.f;
            if (!((mask16 >> (gq + 8)) & 1u)) e[2] = e[3] = 0.f;
          }
          l[nt][0] += e[0] + e[2];
          l[nt][1] += e[1] + e[3];
          // (token, heads) pairs to the B operand's (tokens, head) pairs
          pb[nt][0] = transpose8(pack_f16x2(e[0], e[1]));
          pb[nt][1] = transpose8(pack_f16x2(e[2], e[3]));
        }
        // ---- sum p m (and p s): the rows' (s, m) pairs as a matrix
        {
          uint32_t r[4];
          ldsm_x4_trans(vbase + meta_frag, r);
          const uint32_t am[4] = {r[0], 0u, r[1], 0u};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16_16816(z[nt], am, pb[nt][0], pb[nt][1]);
        }
        // ---- O^T += (s c)^T . P^T
        uint32_t sv[2][4], sn[2][4];  // (s, s') and -64 (s, s') of tokens 2tq, 2tq + 1 (+ 8)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 x = lds128(vbase + v_meta + 8 * i * kPitch);
          const uint4 y = lds128(vbase + v_meta + (8 * i + 1) * kPitch);
          sv[i][0] = __byte_perm(x.x, y.x, 0x5410u);
          sv[i][1] = __byte_perm(x.y, y.y, 0x5410u);
          sv[i][2] = __byte_perm(x.z, y.z, 0x5410u);
          sv[i][3] = __byte_perm(x.w, y.w, 0x5410u);
#pragma unroll
          for (int v = 0; v < 4; ++v) sn[i][v] = hmul2(sv[i][v], 0xD400D400u);  // -64
        }
#pragma unroll
        for (int u2 = 0; u2 < 4; u2 += 2) {
          uint32_t r[4];  // (tokens 2tq, u2), (tokens 2tq + 8, u2), the same of u2 + 1
          ldsm_x4_trans(vbase + frag + 16 * u2, r);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int v = u2 + i;
            uint32_t x[2][4];  // s c of tokens 2tq.. (+8), element 32v + 4gq + k
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w = r[2 * i + j];
              x[j][0] = hfma2(and_or(w << 4, 0x00F000F0u, magic), sv[j][v], sn[j][v]);
              x[j][1] = hfma2(and_or(w, 0x00F000F0u, magic), sv[j][v], sn[j][v]);
              x[j][2] = hfma2(and_or(w >> 4, 0x00F000F0u, magic), sv[j][v], sn[j][v]);
              x[j][3] = hfma2(and_or(w >> 8, 0x00F000F0u, magic), sv[j][v], sn[j][v]);
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const uint32_t av[4] = {x[0][2 * hh], x[0][2 * hh + 1], x[1][2 * hh],
                                      x[1][2 * hh + 1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(o[2 * v + hh][nt], av, pb[nt][0], pb[nt][1]);
            }
          }
        }
      }
    };

    for (int tok = pc.tok_begin; ok && tok < pc.tok_end; tok += kTile) {
      const bool w_ok = mbar_wait_bounded(&full[stage], phase, abort_flag);
      if (!__all_sync(0xffffffffu, w_ok)) {
        ok = false;
        break;
      }
      const uint32_t mask32 = tile_mask[4 * stage + warp % kHeadWarps];
      const uint32_t st = smem_base + stage * L_::kStageBytes;
      if (mask32 == 0xFFFFFFFFu) {
        tile(std::true_type{}, tok, st, mask32);
      } else if (mask32 == 0u) {  // no token of the warp's is there
        if constexpr (kScored) {
          const float none[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int sl = 0; sl < 2; ++sl)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              store_scores(p, pc.b, g, G, tok + t0 + 16 * sl, gq,
                           pc.tok_end - tok - t0 - 16 * sl, nt * 8 + 2 * tq, none);
        }
      } else {
        // rows without a token: s = m = 0 makes their values 0 (the ring's
        // leftovers could be NaN, and 0 x NaN would poison the sums)
        if (!((mask32 >> lane) & 1u))
          *reinterpret_cast<uint4*>(smem + stage * L_::kStageBytes + kTensorBytes + base +
                                    lane * kPitch + 64) = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
        tile(std::false_type{}, tok, st, mask32);
        fence_proxy_async_smem();  // stores before the next TMA
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.err, PA_DEVERR_WAIT_TIMEOUT);
    }

    // ---- the accumulators of a head's warps joined in shared memory, as many
    // groups of 32 head elements at a time as the G heads leave room for
    constexpr int GH = L_::kHeads;
    float* red = reinterpret_cast<float*>(smem + L_::kRedOffset);  // [warp][G][32 vs]
    float* red_m = reinterpret_cast<float*>(smem + L_::kStatOffset);
    float* red_l = red_m + kConsumerWarps * GH;
    const int vs = min(4, GH >> qp.log2_g);  // groups per round
    const int lv = vs == 4 ? 2 : vs - 1;     // log2(vs)
    const int c_first = qp.whole ? c : chunk_of(pc.first, pc.b, total, parts);
    const int c_last = qp.whole ? c : chunk_of(pc.last, pc.b, total, parts);
    const int slot = slot_of_piece(chunks, qp.num_seqs, pc.b, c_first, c);
    if (!qp.whole && c == c_first && threadIdx.x == 0)
      qp.info[static_cast<int64_t>(blockIdx.x) * qp.num_seqs + pc.b] =
          info_of(c_first, c_last);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = l[nt][j];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (gq == 0) {
          red_m[warp * GH + nt * 8 + 2 * tq + j] = m[nt][j];
          red_l[warp * GH + nt * 8 + 2 * tq + j] = x;
        }
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      // (a barrier has passed since the last reads of this memory)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int h = nt * 8 + 2 * tq + j;
          const float zu = __shfl_sync(0xffffffffu, z[nt][j], 4 * (2 * v + 1) + tq);
          if (h < G)
            *reinterpret_cast<float4*>(red + ((warp << qp.log2_g) + h) * (32 << lv) +
                                       32 * (v & (vs - 1)) + 4 * gq) =
                make_float4(o[2 * v][nt][j] + zu, o[2 * v][nt][j + 2] + zu,
                            o[2 * v + 1][nt][j] + zu, o[2 * v + 1][nt][j + 2] + zu);
        }
      }
      if ((v + 1) & (vs - 1)) continue;  // the pass holds more groups
      consumer_barrier();
      for (int i = threadIdx.x; i < (HP * 8 << lv) << qp.log2_g; i += kConsumers) {
        const int hh = i >> (3 + lv);  // of the CTA's query heads
        const int head = hh >> qp.log2_g, h = hh & (G - 1);
        const int e0 = (i & ((8 << lv) - 1)) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kHeadWarps; ++w)
          M = fmaxf(M, red_m[(head * kHeadWarps + w) * GH + h]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float Ls = 0.f;
#pragma unroll
        for (int w = 0; w < kHeadWarps; ++w) {
          const int wi = head * kHeadWarps + w;
          const float wt = M == -INFINITY ? 0.f : exp2f(red_m[wi * GH + h] - M);
          const float lw = red_l[wi * GH + h];
          // (a warp of NaN scores only has no maximum: its sum is NaN all the same)
          Ls += lw * (lw != lw ? 1.f : wt);
          const float4 x =
              *reinterpret_cast<const float4*>(red + ((wi << qp.log2_g) + h) * (32 << lv) + e0);
          acc.x += wt * x.x;
          acc.y += wt * x.y;
          acc.z += wt * x.z;
          acc.w += wt * x.w;
        }
        const float inv = Ls == 0.f ? 0.f : 1.f / Ls;  // NaN stays NaN
        acc.x *= inv;
        acc.y *= inv;
        acc.z *= inv;
        acc.w *= inv;
        const int e = 32 * (v & ~(vs - 1)) + e0;
        if (c_first == c_last) {
          const int64_t row = static_cast<int64_t>(pc.b) * p.num_q_heads + g0 * G + hh;
          *reinterpret_cast<uint2*>(p.out + row * kD + e) =
              make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
          if (kScored && e == 0) p.final_lse[row] = Ls == 0.f ? -INFINITY : M + log2f(Ls);
        } else {
          const int64_t row = (static_cast<int64_t>(g0 + head) * qp.slots + slot) * G + h;
          *reinterpret_cast<float4*>(p.ws_o + row * kD + e) = acc;
          if (e == 0) p.ws_lse[row] = Ls == 0.f ? -INFINITY : M + log2f(Ls);
        }
      }
      consumer_barrier();
    }
  }
}

template <int NT, int HP, bool kScored>
pa_status launch_q4(const CUtensorMap& mk, const CUtensorMap& mv, Q4Params q, int G,
                    int num_splits, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_raised{0};
  auto kern = paged_decode_q4_kernel<NT, HP, kScored>;
  if (!ensure_smem_limit(kern, Lay<NT, HP>::kAlloc, smem_raised)) return PA_ERR_CUDA;
  int sms = num_sms_current_device();
  if (sms <= 0) sms = 148;
  const int32_t heads = q.d.num_kv_heads, seqs = q.num_seqs;
  const Launch l = launch_of(static_cast<int64_t>(sms) * Lay<NT, HP>::kCtasPerSm / (heads / HP),
                             seqs, num_splits, heads, G);
  const int32_t chunks = l.chunks;
  q.whole = l.whole;
  q.slots = l.slots;
  q.info = reinterpret_cast<int32_t*>(q.d.ws_o + l.info_float);
  const dim3 grid(static_cast<unsigned>(heads / HP), static_cast<unsigned>(chunks));
  kern<<<grid, kThreads, Lay<NT, HP>::kAlloc, stream>>>(mk, mv, q, G);
  if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
  if (q.whole || chunks == 1) return PA_OK;  // no sequence is split
  const dim3 merge_grid(static_cast<unsigned>(heads * G),
                        static_cast<unsigned>(seqs < 256 ? seqs : 256));
  return launch_dependent(merge_pieces_kernel<HP, kScored>, merge_grid, kMergeWarps * 32, stream, q,
                          G, chunks);
}

}  // namespace

pa_status launch_paged_decode_q4(const DecodeArgs& a, cudaStream_t stream) {
  if (a.num_seqs == 0) return PA_OK;
  if (a.num_seqs > 65535) return PA_ERR_UNSUPPORTED;
  const int32_t G = a.num_q_heads / a.num_kv_heads;
  // Two kv heads per CTA where their number is even: a token's rows of both
  // are 160 contiguous bytes, and a copy's rate is per row, not per byte
  // (rows of 80 bytes alone: 0.89 of the copy rate with nothing computed, 160: 0.98).
  // A single kv head: two tokens' rows are one 160-byte row of the map.
  const bool paired = a.num_kv_heads % 2 == 0, single = a.num_kv_heads == 1;
  const int64_t rows = a.num_blocks * a.block_size >> (single ? 1 : 0);
  const int32_t box_rows = (a.block_size < kUnit ? a.block_size : kUnit) >> (single ? 1 : 0);
  const int32_t row_bytes = kRow * a.num_kv_heads * (single ? 2 : 1);
  const int32_t box_bytes = paired ? Lay<1, 2>::kPitch : kRow * (single ? 2 : 1);
  CUtensorMap mk, mv;
  if (!make_row_map(&mk, a.k_cache, rows, row_bytes, box_bytes, box_rows) ||
      !make_row_map(&mv, a.v_cache, rows, row_bytes, box_bytes, box_rows))
    return PA_ERR_CUDA;
  Q4Params q{};
  q.d = make_decode_params(a);
  q.num_seqs = a.num_seqs;
  q.pair_tokens = single ? 1 : 0;
  while ((1 << q.log2_g) < G) ++q.log2_g;
  const int n = a.plan.num_splits;
  const bool scored = a.scores != nullptr;
  if (G <= 8) {
    if (paired)
      return scored ? launch_q4<1, 2, true>(mk, mv, q, G, n, stream)
                    : launch_q4<1, 2, false>(mk, mv, q, G, n, stream);
    return scored ? launch_q4<1, 1, true>(mk, mv, q, G, n, stream)
                  : launch_q4<1, 1, false>(mk, mv, q, G, n, stream);
  }
  if (paired)
    return scored ? launch_q4<2, 2, true>(mk, mv, q, G, n, stream)
                  : launch_q4<2, 2, false>(mk, mv, q, G, n, stream);
  return scored ? launch_q4<2, 1, true>(mk, mv, q, G, n, stream)
                : launch_q4<2, 1, false>(mk, mv, q, G, n, stream);
}

}  // namespace pa_detail
