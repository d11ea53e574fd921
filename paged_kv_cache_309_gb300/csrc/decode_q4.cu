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
// different groups of four banks (20 r mod 32).
//
// What bounds it: at 160 bytes per token and kv head HBM leaves an SM 440
// issue slots for 16 tokens, and the first form of this kernel needed 431 of
// them (0.54 of the copy rate at B = 8, 32K-128K).  So the element work is
// the forms above, a new running maximum is looked for by a vote (the
// shuffles run only when a score beats the old one by 2^8), and the prologue
// and epilogue, which cost as much as 40 tokens, run once per piece of a
// balanced cut instead of once per short token range:
//   the sequences' units of 64 tokens lie end to end, every sequence start
//   charged kPieceCost units more; chunk c of C (C x H_KV CTAs fill the GPU
//   once) is the units whose cost lies in [c, c + 1) total / C.  A chunk
//   walks its pieces with the ring running on across them.  A sequence that
//   lies in one chunk is written directly; the pieces of one that does not
//   go to partial slots, and the last of them to finish merges them.
//
// Every mbarrier wait is bounded (2 s); after a timeout the error bit is
// set, the remaining pieces end empty (so the counts complete), the copies in
// flight are waited for, and the CTA exits.
#include <atomic>
#include <type_traits>

#include "decode_common.cuh"

namespace pa_detail {
namespace {

constexpr int kUnit = 64;          // tokens per unit of the cut (boxes are up to 64 rows)
constexpr int kTile = 128;         // tokens per stage, 32 per consumer warp
constexpr int kRow = 80;           // bytes of a cached row
constexpr int kTensorBytes = kTile * kRow;
constexpr float kLift = 7.0f;      // weights are 2^kLift (score - running maximum)
constexpr int kPieceCost = 1;      // units charged for a sequence's start
constexpr int kConsumers = kConsumerWarps * 32;

struct Q4Params {
  DecodeParams d;
  int32_t num_seqs;
  int32_t slots;  // partial slots per kv head
  bool whole;     // no partials: chunks begin at sequence starts
};

template <int NT>
struct Lay {
  static constexpr int kStages = 3;
  static constexpr int kCtasPerSm = NT == 1 ? 3 : 2;
  static constexpr int kStageBytes = 2 * kTensorBytes;  // K rows, then V rows
  static constexpr int kHeads = NT * 8;
  // the join of the four warps, 64 head elements at a time: [warp][h][64], then
  // maxima and sums [warp][h], weights [warp][h], totals [h][2]
  static constexpr int kRedOffset = kStages * kStageBytes;
  static constexpr int kRedFloats = kConsumerWarps * kHeads * 64;
  static constexpr int kStatOffset = kRedOffset + kRedFloats * 4;
  static constexpr int kStatFloats = 3 * kConsumerWarps * kHeads + 2 * kHeads;
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
// Units of 64 tokens lie end to end in sequence order; unit t (counted over
// all sequences) of sequence b sits at cost t + kPieceCost (b + 1), the line is
// total = units + kPieceCost B long, and its chunk is floor(cost parts / total)
// with parts = min(C, total): a step of one unit moves at most one chunk on, so
// no chunk inside a sequence's span is empty.
__device__ __forceinline__ int chunk_of(int64_t t, int b, int64_t total, int parts) {
  return static_cast<int>((t + static_cast<int64_t>(kPieceCost) * (b + 1)) * parts / total);
}

__device__ __forceinline__ int units_of(const DecodeParams& p, int b) {
  bool clipped;
  return (effective_len(p, b, &clipped) + kUnit - 1) / kUnit;
}

// Warp 0: the first unit of chunks c and c + 1.  sched: total, first unit of c,
// first unit of c + 1, then the first one's sequence and the units before that.
__device__ __forceinline__ void find_chunk(const Q4Params& q, int c, int chunks, int lane,
                                           int64_t* sched) {
  const DecodeParams& p = q.d;
  int64_t units = 0;
  bool any_clipped = false;
  for (int b = lane; b < q.num_seqs; b += 32) {
    bool clipped;
    units += (effective_len(p, b, &clipped) + kUnit - 1) / kUnit;
    any_clipped |= clipped;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) units += __shfl_xor_sync(0xffffffffu, units, off);
  if (c == 0 && blockIdx.x == 0 && any_clipped) atomicOr(p.err, PA_DEVERR_CONTEXT_CLIPPED);
  const int64_t total = units + static_cast<int64_t>(kPieceCost) * q.num_seqs;
  const int64_t parts = min(total, static_cast<int64_t>(chunks));
  // chunk k begins at the first unit whose cost reaches ceil(k total / parts)
  const int64_t x0 = (c * total + parts - 1) / parts;
  const int64_t x1 = ((c + 1) * total + parts - 1) / parts;
  int64_t g0 = units, g1 = units, pre0 = 0;
  int b0 = q.num_seqs;
  bool found0 = c >= parts, found1 = c + 1 >= parts;
  int64_t base = 0;
  for (int first = 0; first < q.num_seqs && !(found0 && found1); first += 32) {
    const int b = first + lane;
    const int n = b < q.num_seqs ? units_of(p, b) : 0;
    int64_t incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    const int64_t pre = base + incl - n;
    // the cost that decides: of the sequence's last unit (some unit reaches x), or of
    // its first when sequences stay whole
    const int64_t cost = pre + (q.whole ? 0 : n - 1) + static_cast<int64_t>(kPieceCost) * (b + 1);
    const int64_t charge = static_cast<int64_t>(kPieceCost) * (b + 1);
    if (!found0) {
      const uint32_t hit = __ballot_sync(0xffffffffu, n > 0 && cost >= x0);
      if (hit != 0u) {
        const int l = __ffs(hit) - 1;
        const int64_t at = q.whole ? pre : max(x0 - charge, pre);
        g0 = __shfl_sync(0xffffffffu, at, l);
        pre0 = __shfl_sync(0xffffffffu, pre, l);
        b0 = first + l;
        found0 = true;
      }
    }
    if (!found1) {
      const uint32_t hit = __ballot_sync(0xffffffffu, n > 0 && cost >= x1);
      if (hit != 0u) {
        const int l = __ffs(hit) - 1;
        const int64_t at = q.whole ? pre : max(x1 - charge, pre);
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
    const int n = (L + kUnit - 1) / kUnit;
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

// Merge of one query head's n partials by one warp (the first in start_slot, the others
// in slots first_slot, first_slot + 1, ...): weights 2^(lse - max).
template <bool kScored>
__device__ __forceinline__ void merge_pieces(const DecodeParams& p, int64_t bh, const float* lse,
                                             const float* o, int G, int start_slot, int first_slot,
                                             int n, int lane) {
  auto slot = [&](int i) -> int64_t {
    return static_cast<int64_t>(i == 0 ? start_slot : first_slot + i - 1) * G;
  };
  float M = -INFINITY;  // (a NaN lse is carried to the output)
  for (int i = lane; i < n; i += 32) M = max_nan(M, __ldcg(lse + slot(i)));
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, off));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float W = 0.f;
  if (M != -INFINITY) {
    for (int i0 = 0; i0 < n; i0 += 32) {
      const float wl = i0 + lane < n ? exp2f(__ldcg(lse + slot(i0 + lane)) - M) : 0.f;
      const int cnt = min(32, n - i0);
      for (int k0 = 0; k0 < cnt; k0 += 8) {
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          v[k] = k0 + k < cnt
                     ? __ldcg(reinterpret_cast<const float4*>(o + slot(i0 + k0 + k) * kD) + lane)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float w = __shfl_sync(0xffffffffu, wl, (k0 + k) & 31);
          if (k0 + k < cnt) {
            W += w;
            acc.x += w * v[k].x;
            acc.y += w * v[k].y;
            acc.z += w * v[k].z;
            acc.w += w * v[k].w;
          }
        }
      }
    }
  }
  if (kScored && lane == 0) p.final_lse[bh] = W == 0.f ? -INFINITY : M + log2f(W);
  const float inv = W == 0.f ? 0.f : 1.f / W;
  *reinterpret_cast<uint2*>(p.out + bh * kD + lane * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

// NT: n-tiles of 8 query heads (G <= 8 -> 1, G = 16 -> 2); kScored: also
// store the scores and each query head's log2-sum-exp.
template <int NT, bool kScored>
__global__ void __launch_bounds__(kThreads, Lay<NT>::kCtasPerSm)
    paged_decode_q4_kernel(const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ Q4Params qp, int G) {
  using L_ = Lay<NT>;
  const DecodeParams& p = qp.d;
  constexpr int kStages = L_::kStages;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L_::kBarOffset);
  uint64_t* empty = full + kStages;
  uint32_t* tile_mask = reinterpret_cast<uint32_t*>(smem + L_::kMaskOffset);
  int64_t* sched = reinterpret_cast<int64_t*>(smem + L_::kSchedOffset);
  int* abort_ptr = reinterpret_cast<int*>(smem + L_::kFlagOffset);
  int* last_flag = abort_ptr + 1;

  // kv heads fastest in launch order: the CTAs of one chunk read neighbouring
  // rows at the same time
  const int g = blockIdx.x;
  const int c = blockIdx.y;
  const int chunks = gridDim.y;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int bs = p.block_size;
  const int hq0 = g * G;

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
  const int64_t total = sched[0];
  const int parts = static_cast<int>(min(total, static_cast<int64_t>(chunks)));

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
          mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(__popc(vb) * rpb * kRow * 2));
        }
        __syncwarp();
        if (valid) {
          const int32_t row = bid * bs + (first & (bs - 1));
          uint8_t* st = smem + stage * L_::kStageBytes + lane * rpb * kRow;
          tma_load_3d(st, &tm_k, 0, g, row, &full[stage], pol);
          tma_load_3d(st + kTensorBytes, &tm_v, 0, g, row, &full[stage], pol);
        }
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.err, PA_DEVERR_WAIT_TIMEOUT);
    }
    // copies in flight at an early end are waited for (bounded) before the CTA exits
    if (!ok && lane == 0) {
      for (int t = max(0, u - kStages); t < u; ++t)
        mbar_wait_bounded(&full[t % kStages], (t / kStages) & 1, nullptr);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  // sequences without tokens: zero rows (chunk c takes b = c mod C)
  for (int b = c; b < qp.num_seqs; b += chunks) {
    if (units_of(p, b) == 0) {
      for (int i = threadIdx.x; i < G * (kD / 8); i += kConsumers)
        reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(b) * p.num_q_heads + hq0) * kD)[i] =
            make_uint4(0u, 0u, 0u, 0u);
      if (kScored && threadIdx.x < G)
        p.final_lse[static_cast<int64_t>(b) * p.num_q_heads + hq0 + threadIdx.x] = -INFINITY;
    }
  }

  const int gq = lane >> 2;  // mma groupID
  const int tq = lane & 3;   // thread in group
  // ldmatrix rows and 16-byte columns of this lane (K and V alike): rows
  // (lane & 15), column u + (lane >> 4); the (s, m) pairs: rows (lane & 15)
  const uint32_t frag = static_cast<uint32_t>((32 * warp + (lane & 15)) * kRow + 16 * (lane >> 4));
  const uint32_t meta_frag = static_cast<uint32_t>((32 * warp + (lane & 15)) * kRow + 64);
  // (s, m) rows read directly: K row gq, V row 2tq
  const uint32_t k_meta = static_cast<uint32_t>((32 * warp + gq) * kRow + 64);
  const uint32_t v_meta = static_cast<uint32_t>(kTensorBytes + (32 * warp + 2 * tq) * kRow + 64);
  const uint32_t smem_base = smem_u32(smem);
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

    // One 16-token slice of a tile (sl 0 or 1).  kFull: every row is a token.
    auto slice = [&](auto full_tag, const int sl, const int tok, const uint32_t st,
                     const uint32_t mask32) {
      constexpr bool kFull = decltype(full_tag)::value;
      const int r0 = 32 * warp + 16 * sl;
      const uint32_t mask16 = (mask32 >> (16 * sl)) & 0xFFFFu;
      if (!kFull && mask16 == 0u) {  // no token of the slice is there
        if constexpr (kScored) {
          const float none[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            store_scores(p, pc.b, g, G, tok + r0, gq, pc.tok_end - tok - r0, nt * 8 + 2 * tq,
                         none);
        }
        return;
      }
      const uint32_t kbase = st + sl * 16 * kRow;
      const uint32_t kaddr = kbase + frag;
      const uint32_t vaddr = kaddr + kTensorBytes;
      // ---- S_u = codes . q, and the minima's sum
      float su[NT][4][4], zk[NT][4];
#pragma unroll
      for (int u2 = 0; u2 < 4; u2 += 2) {
        uint32_t r[4];  // (row gq, u2), (row gq + 8, u2), (row gq, u2 + 1), (row gq + 8, u2 + 1)
        ldsm_x4(kaddr + 16 * u2, r);
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
        const uint4 w = lds128(kbase + k_meta + 8 * i * kRow);
        ss[i][0] = low_f32(w.x);
        ss[i][1] = low_f32(w.y);
        ss[i][2] = low_f32(w.z);
        ss[i][3] = low_f32(w.w);
      }
      const bool v0 = kFull || ((mask16 >> gq) & 1u);        // token r0 + gq
      const bool v1 = kFull || ((mask16 >> (gq + 8)) & 1u);  // token r0 + gq + 8
      // ---- scores relative to the running maximum (first: to -inf, so +inf)
      float a[NT][4], sr[NT][4];
      bool high = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[nt][i] = ss[i >> 1][0] * su[nt][0][i];
#pragma unroll
          for (int v = 1; v < 4; ++v) a[nt][i] = fmaf(ss[i >> 1][v], su[nt][v][i], a[nt][i]);
          sr[nt][i] = fmaf(a[nt][i], sscale[nt][i & 1],
                           fmaf(zk[nt][i], zscale[nt][i & 1], -m[nt][i & 1]));
        }
        if (!v0) sr[nt][0] = sr[nt][1] = -INFINITY;
        if (!v1) sr[nt][2] = sr[nt][3] = -INFINITY;
        high |= fmaxf(fmaxf(sr[nt][0], sr[nt][1]), fmaxf(sr[nt][2], sr[nt][3])) >
                kLift + kRescaleLog2;
      }
      if (kScored || __any_sync(0xffffffffu, high)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float s[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s[i] = fmaf(a[nt][i], sscale[nt][i & 1], zk[nt][i] * zscale[nt][i & 1]);
          if (!v0) s[0] = s[1] = -INFINITY;
          if (!v1) s[2] = s[3] = -INFINITY;
          if constexpr (kScored)
            store_scores(p, pc.b, g, G, tok + r0, gq, pc.tok_end - tok - r0, nt * 8 + 2 * tq, s);
          if (kScored && !__any_sync(0xffffffffu, high)) continue;
          float mx[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
#pragma unroll
          for (int off = 4; off <= 16; off <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], off));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], off));
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (mx[j] > m[nt][j] + (kLift + kRescaleLog2)) {  // always on the first
              const float corr = exp2f(m[nt][j] - (mx[j] - kLift));
              l[nt][j] *= corr;
              z[nt][j] *= corr;
              z[nt][j + 2] *= corr;
#pragma unroll
              for (int mt = 0; mt < 8; ++mt) {
                o[mt][nt][j] *= corr;
                o[mt][nt][j + 2] *= corr;
              }
              m[nt][j] = mx[j] - kLift;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) sr[nt][i] = s[i] - m[nt][i & 1];
          if (!v0) sr[nt][0] = sr[nt][1] = -INFINITY;
          if (!v1) sr[nt][2] = sr[nt][3] = -INFINITY;
        }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float p0 = ex2(sr[nt][0]), p1 = ex2(sr[nt][1]);
        const float p2 = ex2(sr[nt][2]), p3 = ex2(sr[nt][3]);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        // (token, heads) pairs to the B operand's (tokens, head) pairs
        pb[nt][0] = transpose8(pack_f16x2(p0, p1));
        pb[nt][1] = transpose8(pack_f16x2(p2, p3));
      }
      // ---- sum p m (and p s): the rows' (s, m) pairs as a matrix
      {
        uint32_t r[4];
        ldsm_x4_trans(kbase + kTensorBytes + meta_frag, r);
        const uint32_t am[4] = {r[0], 0u, r[1], 0u};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(z[nt], am, pb[nt][0], pb[nt][1]);
      }
      // ---- O^T += (s c)^T . P^T
      uint32_t sv[2][4], sn[2][4];  // (s, s') and -64 (s, s') of tokens 2tq, 2tq + 1 (+ 8)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 x = lds128(kbase + v_meta + 8 * i * kRow);
        const uint4 y = lds128(kbase + v_meta + (8 * i + 1) * kRow);
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
        ldsm_x4_trans(vaddr + 16 * u2, r);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int v = u2 + i;
          uint32_t x[2][4];  // s c of tokens 2tq.. (+8), element 32v + 4gq + k
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w = r[2 * i + j];
            x[j][0] = hfma2(((w << 4) & 0x00F000F0u) | 0x54005400u, sv[j][v], sn[j][v]);
            x[j][1] = hfma2((w & 0x00F000F0u) | 0x54005400u, sv[j][v], sn[j][v]);
            x[j][2] = hfma2(((w >> 4) & 0x00F000F0u) | 0x54005400u, sv[j][v], sn[j][v]);
            x[j][3] = hfma2(((w >> 8) & 0x00F000F0u) | 0x54005400u, sv[j][v], sn[j][v]);
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
    };

    for (int tok = pc.tok_begin; ok && tok < pc.tok_end; tok += kTile) {
      const bool w_ok = mbar_wait_bounded(&full[stage], phase, abort_flag);
      if (!__all_sync(0xffffffffu, w_ok)) {
        ok = false;
        break;
      }
      const uint32_t mask32 = tile_mask[4 * stage + warp];
      const uint32_t st = smem_base + stage * L_::kStageBytes;
      if (mask32 == 0xFFFFFFFFu) {
        slice(std::true_type{}, 0, tok, st, mask32);
        slice(std::true_type{}, 1, tok, st, mask32);
      } else {
        // rows without a token: s = m = 0 makes their values 0 (the ring's
        // leftovers could be NaN, and 0 x NaN would poison the sums)
        if (!((mask32 >> lane) & 1u))
          *reinterpret_cast<uint4*>(smem + stage * L_::kStageBytes + kTensorBytes +
                                    (32 * warp + lane) * kRow + 64) = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
#pragma unroll 1
        for (int sl = 0; sl < 2; ++sl) slice(std::false_type{}, sl, tok, st, mask32);
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

    // ---- the four warps' (maximum, sum, accumulator) joined in shared memory
    constexpr int GH = L_::kHeads;
    float* red = reinterpret_cast<float*>(smem + L_::kRedOffset);  // [warp][h][64]
    float* red_m = reinterpret_cast<float*>(smem + L_::kStatOffset);
    float* red_l = red_m + kConsumerWarps * GH;
    float* red_w = red_l + kConsumerWarps * GH;
    float* fin = red_w + kConsumerWarps * GH;
    const int c_first = qp.whole ? c : chunk_of(pc.first, pc.b, total, parts);
    const int c_last = qp.whole ? c : chunk_of(pc.last, pc.b, total, parts);
    // partial slot: c - 1 for a piece that goes on from chunk c - 1; for a
    // sequence's first piece one of its own behind those
    const int start_slot = chunks - 1 + (qp.num_seqs <= chunks - 1 ? pc.b : c_first);
    const int slot = c == c_first ? start_slot : c - 1;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      // (a barrier has passed since the last reads of this memory)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int h = nt * 8 + 2 * tq + j;
          if (half == 0) {
            float lv = l[nt][j];
            lv += __shfl_xor_sync(0xffffffffu, lv, 4);
            lv += __shfl_xor_sync(0xffffffffu, lv, 8);
            lv += __shfl_xor_sync(0xffffffffu, lv, 16);
            if (gq == 0) {
              red_m[warp * GH + h] = m[nt][j];
              red_l[warp * GH + h] = lv;
            }
          }
#pragma unroll
          for (int v = 2 * half; v < 2 * half + 2; ++v) {
            const float zu = __shfl_sync(0xffffffffu, z[nt][j], 4 * (2 * v + 1) + tq);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              float* dst = red + (warp * GH + h) * 64 + 32 * (v & 1) + 4 * gq + 2 * hh;
              *reinterpret_cast<float2*>(dst) =
                  make_float2(o[2 * v + hh][nt][j] + zu, o[2 * v + hh][nt][j + 2] + zu);
            }
          }
        }
      }
      consumer_barrier();
      if (half == 0) {
        if (threadIdx.x < G) {
          const int h = threadIdx.x;
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kConsumerWarps; ++w) M = fmaxf(M, red_m[w * GH + h]);
          float Ls = 0.f;
#pragma unroll
          for (int w = 0; w < kConsumerWarps; ++w) {
            const float wt = (M == -INFINITY) ? 0.f : exp2f(red_m[w * GH + h] - M);
            red_w[w * GH + h] = wt;
            // (a warp of NaN scores only has no maximum: its sum is NaN all the same)
            Ls += red_l[w * GH + h] * (red_l[w * GH + h] != red_l[w * GH + h] ? 1.f : wt);
          }
          fin[2 * h] = M;
          fin[2 * h + 1] = Ls;
        }
        consumer_barrier();
      }
      for (int i = threadIdx.x; i < G * 16; i += kConsumers) {
        const int h = i >> 4;
        const int e0 = (i & 15) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kConsumerWarps; ++w) {
          const float wt = red_w[w * GH + h];
          const float4 v = *reinterpret_cast<const float4*>(red + (w * GH + h) * 64 + e0);
          acc.x += wt * v.x;
          acc.y += wt * v.y;
          acc.z += wt * v.z;
          acc.w += wt * v.w;
        }
        const float Ls = fin[2 * h + 1];
        const float inv = Ls == 0.f ? 0.f : 1.f / Ls;  // NaN stays NaN
        acc.x *= inv;
        acc.y *= inv;
        acc.z *= inv;
        acc.w *= inv;
        const float lse = Ls == 0.f ? -INFINITY : fin[2 * h] + log2f(Ls);
        const int e = 64 * half + e0;
        if (c_first == c_last) {
          const int64_t row = static_cast<int64_t>(pc.b) * p.num_q_heads + hq0 + h;
          *reinterpret_cast<uint2*>(p.out + row * kD + e) =
              make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
          if (kScored && e == 0) p.final_lse[row] = lse;
        } else {
          const int64_t row = (static_cast<int64_t>(g) * qp.slots + slot) * G + h;
          *reinterpret_cast<float4*>(p.ws_o + row * kD + e) = acc;
          if (e == 0) p.ws_lse[row] = lse;
        }
      }
      consumer_barrier();
    }
    if (c_first != c_last) {
      // the piece that completes the count merges the sequence's pieces and
      // returns the counter to zero
      if (threadIdx.x == 0) {
        __threadfence();
        unsigned* ctr = p.counters + static_cast<int64_t>(pc.b) * p.num_kv_heads + g;
        const bool last = atomicAdd(ctr, 1u) + 1u == static_cast<unsigned>(c_last - c_first + 1);
        if (last) {
          atomicExch(ctr, 0u);
          __threadfence();
        }
        *last_flag = last ? 1 : 0;
      }
      consumer_barrier();
      if (*last_flag) {
        const int64_t at = static_cast<int64_t>(g) * qp.slots * G;
        for (int h = warp; h < G; h += kConsumerWarps)
          merge_pieces<kScored>(p, static_cast<int64_t>(pc.b) * p.num_q_heads + hq0 + h,
                                p.ws_lse + at + h, p.ws_o + (at + h) * kD, G, start_slot, c_first,
                                c_last - c_first + 1, lane);
      }
    }
  }
}

template <int NT, bool kScored>
pa_status launch_q4(const CUtensorMap& mk, const CUtensorMap& mv, Q4Params q, int G,
                    int num_splits, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_raised{0};
  auto kern = paged_decode_q4_kernel<NT, kScored>;
  if (!ensure_smem_limit(kern, Lay<NT>::kAlloc, smem_raised)) return PA_ERR_CUDA;
  // one wave of CTAs, as far as the workspace's partial rows (num_seqs * num_splits
  // per query head) hold what the cut can leave: a piece behind every inner chunk
  // boundary and a first piece for every sequence that crosses one
  int sms = num_sms_current_device();
  if (sms <= 0) sms = 148;
  int64_t chunks = static_cast<int64_t>(sms) * Lay<NT>::kCtasPerSm / q.d.num_kv_heads;
  const int64_t seqs = q.num_seqs, rows = seqs * num_splits;
  q.whole = num_splits == 1;
  if (q.whole) {
    if (chunks > seqs) chunks = seqs;
  } else if (chunks - 1 + (seqs < chunks - 1 ? seqs : chunks - 1) > rows) {
    chunks = seqs < rows - seqs ? rows - seqs + 1 : rows / 2 + 1;
  }
  if (chunks > 65535) chunks = 65535;
  if (chunks < 1) chunks = 1;
  q.slots = static_cast<int32_t>(chunks - 1 + (seqs < chunks - 1 ? seqs : chunks - 1));
  const dim3 grid(static_cast<unsigned>(q.d.num_kv_heads), static_cast<unsigned>(chunks));
  kern<<<grid, kThreads, Lay<NT>::kAlloc, stream>>>(mk, mv, q, G);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

pa_status launch_paged_decode_q4(const DecodeArgs& a, cudaStream_t stream) {
  if (a.num_seqs == 0) return PA_OK;
  if (a.num_seqs > 65535) return PA_ERR_UNSUPPORTED;
  const int32_t G = a.num_q_heads / a.num_kv_heads;
  const int64_t rows = a.num_blocks * a.block_size;
  const int32_t box_rows = a.block_size < kUnit ? a.block_size : kUnit;
  CUtensorMap mk, mv;
  if (!make_kv_map_q4(&mk, a.k_cache, rows, a.num_kv_heads, box_rows) ||
      !make_kv_map_q4(&mv, a.v_cache, rows, a.num_kv_heads, box_rows))
    return PA_ERR_CUDA;
  Q4Params q{};
  q.d = make_decode_params(a);
  q.num_seqs = a.num_seqs;
  const int n = a.plan.num_splits;
  if (a.scores != nullptr)
    return G <= 8 ? launch_q4<1, true>(mk, mv, q, G, n, stream)
                  : launch_q4<2, true>(mk, mv, q, G, n, stream);
  return G <= 8 ? launch_q4<1, false>(mk, mv, q, G, n, stream)
                : launch_q4<2, false>(mk, mv, q, G, n, stream);
}

}  // namespace pa_detail
