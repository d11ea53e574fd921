// decode_window.cu -- paged GQA decode attention with a sliding window and a few first
// tokens that stay visible, over bf16 and e4m3 caches.
//
// The query of a sequence of L tokens sees t >= L - window and t < num_sink.  The rows that
// this leaves are one range of places (window.cuh): pieces of a block's rows with first
// tokens, then those from the window's start on; what a piece holds besides is
// masked.  Blocks between are neither looked up nor read.
//
// What bounds it: HBM (G flops a byte over bf16).  A window makes contexts short and alike, so a
// CTA for each (sequence, kv head, range) would spend its time on prologues, epilogues and a
// last wave that does not fill the GPU.  The cut is the 4-bit decode's instead
// (q4_cut.h, decode_pieces.cuh): one wave of CTAs (two per SM), each with an equal share of all
// sequences' units of 64 places, walking its pieces with the copy ring running on
// across them; sequences that lie in one chunk are written directly, the
// others' pieces are merged by a second, dependent launch.  Where that would take longer than
// whole sequences to a CTA, nothing is cut (window_cut.h).
//
// Per tile a producer warp looks up blocks and issues TMA copies (128-byte swizzled);
// four consumer warps take 16 (bf16, tiles of 64) or 32 (e4m3, tiles of 128) places each:
// S^T = K Q^T, an fp32 softmax in base 2 whose running maximum moves only when a score beats it
// by 2^8 (one vote), O^T += V^T P^T, all mma.sync m16n8k16.  bf16 weights are carried as two
// bf16 terms; e4m3 codes go to fp16 (exact), q after a power of two and weights in
// fp16, 2^7 above the running maximum's scale so that they keep 11 bits down to 2^-21 of it.
//
// Measured (GPU time of both launches, perf/gpu_times.py):
//  * 64 sequences of 512 .. 4096 tokens, window 1024, 8 kv heads, bf16: 45.9 us for 258 MB
//    (a CTA per sequence, head and range of places: 86.8);
//  * 8 of 32768 .. 131072, window 16384, 8 kv heads: 84.4 us for 539 MB, 6.4 TB/s (127.8);
//  * e4m3, 64 of 512 .. 8192, window 2000, 4 kv heads, whole sequences: 22.7 us for
//    122 MB (cut and merged 33.4; a CTA per range 55.4).  Three or four CTAs an SM
//    changed nothing;
//  * the smallest call is a chain of launch, lengths, block ids, first copy and the join
//    of four warps: 3.9 us.
// A merge by whichever CTA came last instead of a second launch gained nothing.
//
// Every mbarrier wait is bounded (2 s); after a timeout the error bit is set, the
// remaining pieces end empty, the copies in flight are waited for, and the CTA exits.
#include <atomic>
#include <type_traits>

#include "decode_pieces.cuh"
#include "window.cuh"

namespace pa_detail {

using namespace pa;
using namespace decode;
using namespace pieces;
using namespace windowcut;

namespace {

static_assert(kHeaderBytes == kWorkspaceHeader, "one header for all workspaces");
constexpr int kLog2Rows = 6;  // copies are of up to 64 rows
// A running maximum before the first score: finite, so that a score of -inf (a masked place, or an
// infinite key) has the weight 2^(-inf - m) = 0 then too.
constexpr float kNoMaximum = -3.402823466e38f;

__device__ __forceinline__ WindowRange range_of(const PieceParams& q, int b, bool* clipped) {
  const DecodeParams& p = q.d;
  int L = max(__ldg(p.context_lens + b), 0);
  const int64_t cap = min(static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size,
                          static_cast<int64_t>(q.max_len));
  *clipped = L > cap;
  if (*clipped) L = static_cast<int>(cap);
  return window_range(L, max(0, L - q.window), q.num_sink, min(p.log2_bs, kLog2Rows));
}
struct WindowRows {
  static __device__ __forceinline__ int len(const PieceParams& q, int b, bool* clipped) {
    return range_of(q, b, clipped).len;
  }
};

template <int NT, bool kFp8>
struct Lay {
  static constexpr int kStages = 3;
  static constexpr int kSlices = kFp8 ? 2 : 1;         // of 16 places per warp and tile
  static constexpr int kTile = kConsumerWarps * 16 * kSlices;
  static constexpr int kRowBytes = kFp8 ? 128 : 256;
  static constexpr int kHalf = kTile * 128;            // 128 bytes of every row
  static constexpr int kVOffset = kTile * kRowBytes;
  static constexpr int kStageBytes = 2 * kVOffset;
  static constexpr int kHeads = NT * 8;
  // the join of a head's warps: kRound head elements of every head of a warp at a time, rows
  // padded by four floats (a warp's stores then fall into 32 banks)
  static constexpr int kRound = NT == 1 ? 64 : 32;
  static constexpr int kPitch = kRound + 4;
  static constexpr int kRedOffset = kStages * kStageBytes;
  static constexpr int kRedFloats = kConsumerWarps * kHeads * kPitch;
  static constexpr int kStatOffset = kRedOffset + kRedFloats * 4;
  static constexpr int kBarOffset = kStatOffset + 2 * kConsumerWarps * kHeads * 4;
  static constexpr int kMaskOffset = kBarOffset + 2 * kStages * 8;  // four words per stage
  static constexpr int kSchedOffset = kMaskOffset + kStages * 16;   // five 64-bit words
  static constexpr int kFlagOffset = kSchedOffset + 40;
  static constexpr int kAlloc = kFlagOffset + 8 + 1024;  // room to align the base to 1 KB
  static constexpr float kLift = kFp8 ? 7.0f : 0.0f;     // weights are 2^kLift (score - maximum)
  static_assert(kBarOffset % 8 == 0 && kMaskOffset % 16 == 0 && kSchedOffset % 8 == 0, "aligned");
  static_assert((kAlloc + 1024) * kCtasPerSm <= 228 * 1024, "resident CTAs fit");
};

// What the pieces of one (sequence, query head) come to: weights 2^(lse - max), by one warp (lane:
// four head elements).  `slot(i)`: place of piece i; partials are read through L2.
template <int kAhead, typename Slot>
__device__ __forceinline__ void merge_row(const DecodeParams& p, int64_t bh, int n, int lane,
                                          const Slot& slot) {
  float M = -INFINITY;  // (a NaN lse is carried to the output)
  for (int i = lane; i < n; i += 32) M = max_nan(M, __ldcg(p.ws_lse + slot(i)));
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, off));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float W = 0.f;
  if (M != -INFINITY) {
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      float4 v[kAhead];
      float w[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (i0 + k < n) {
          const int64_t at = slot(i0 + k);
          v[k] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + at * kD) + lane);
          w[k] = exp2f(__ldcg(p.ws_lse + at) - M);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (i0 + k < n) {
          W += w[k];
          acc.x += w[k] * v[k].x;
          acc.y += w[k] * v[k].y;
          acc.z += w[k] * v[k].z;
          acc.w += w[k] * v[k].w;
        }
      }
    }
  }
  const float inv = W == 0.f ? 0.f : 1.f / W;
  *reinterpret_cast<uint2*>(p.out + bh * kD + lane * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

// The second launch: a warp per (split sequence, query head); a CTA looks at 32
// sequences a time and takes every gridDim.y-th.
constexpr int kMergeThreads = 128;
__global__ void __launch_bounds__(kMergeThreads)
    merge_split_kernel(const __grid_constant__ PieceParams qp, int G, int chunks) {
  const DecodeParams& p = qp.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hq = blockIdx.x * (kMergeThreads / 32) + warp;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (hq >= p.num_q_heads) return;
  const int g = hq / G;
  for (int first = blockIdx.y; first < qp.num_seqs; first += 32 * gridDim.y) {
    const int mine = first + lane * gridDim.y;
    const int32_t info =
        mine < qp.num_seqs ? __ldcg(qp.info + static_cast<int64_t>(g) * qp.num_seqs + mine) : 0;
    for (uint32_t todo = __ballot_sync(0xffffffffu, info != 0); todo != 0u; todo &= todo - 1u) {
      const int l = __ffs(todo) - 1;
      const int32_t x = __shfl_sync(0xffffffffu, info, l);
      const int b = first + l * gridDim.y, c_first = x >> 16;
      merge_row<8>(p, static_cast<int64_t>(b) * p.num_q_heads + hq, x & 0xFFFF, lane, [&](int i) {
        return (static_cast<int64_t>(g) * qp.slots +
                slot_of_piece(chunks, qp.num_seqs, b, c_first, c_first + i)) *
                   G +
               hq % G;
      });
    }
  }
}

template <int NT, bool kFp8>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    window_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ PieceParams qp, int G) {
  using L_ = Lay<NT, kFp8>;
  const DecodeParams& p = qp.d;
  constexpr int kStages = L_::kStages, kTile = L_::kTile, kSlices = L_::kSlices;
  constexpr float kLift = L_::kLift;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  // 1 KB-aligned base (the 128-byte swizzle pattern repeats every 1 KB)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L_::kBarOffset);
  uint64_t* empty = full + kStages;
  uint32_t* tile_mask = reinterpret_cast<uint32_t*>(smem + L_::kMaskOffset);
  int64_t* sched = reinterpret_cast<int64_t*>(smem + L_::kSchedOffset);
  int* abort_ptr = reinterpret_cast<int*>(smem + L_::kFlagOffset);

  // kv heads fastest in launch order: the CTAs of one chunk read neighbouring rows at
  // the same time
  const int g = blockIdx.x;
  const int c = blockIdx.y;
  const int chunks = gridDim.y;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int bs = p.block_size;

  if (warp == 0) find_chunk<WindowRows>(qp, c, chunks, lane, sched);
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
    const int rpb = 1 << min(p.log2_bs, kLog2Rows);
    const int nbox = kTile / rpb;
    const int start = lane * rpb;  // of the tile's places
    const uint64_t pol = l2_policy_evict_first();
    if (lane == 0) {
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
    Walk walk(sched);
    Piece pc;
    int u = 0;  // tiles issued
    bool ok = true;
    while (ok && next_piece<WindowRows>(qp, walk, pc)) {
      const int32_t* bt = p.block_tables + static_cast<int64_t>(pc.b) * p.max_blocks_per_seq;
      bool clipped;
      const WindowRange win = range_of(qp, pc.b, &clipped);
      // lane i < nbox: block id of box i of the tile at `at` (-1 past the piece), read one
      // tile ahead of its issue
      auto tile_bid = [&](int at) -> int {
        const int first = at + start;
        return lane < nbox && first < pc.tok_end ? __ldg(bt + (win.row(first) >> p.log2_bs)) : -1;
      };
      int bid_next = tile_bid(pc.tok_begin);
      for (int at = pc.tok_begin; at < pc.tok_end; at += kTile, ++u) {
        const int stage = u % kStages;
        const int bid = bid_next;
        bid_next = tile_bid(at + kTile);
        if (u >= kStages) {
          const bool w_ok = mbar_wait_bounded(&empty[stage], ((u / kStages) - 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, w_ok)) {
            ok = false;
            break;
          }
        }
        const int first = win.row(at + start);
        const int rows = lane < nbox ? min(rpb, pc.tok_end - at - start) : 0;
        uint64_t seen = 0ull;  // of the box's rows
        if (rows > 0 && bid >= 0 && static_cast<int64_t>(bid) < p.num_blocks)
          seen = WindowRange::below(rows) & win.visible(first, qp.num_sink);
        const bool valid = seen != 0ull;
        // the box's rows as bits of the tile, a word for each consumer warp
        uint32_t words[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int shift = start - 16 * kSlices * w;
          const uint64_t bits = shift >= 64 || shift <= -64 ? 0ull
                                : shift >= 0                ? seen << shift
                                                            : seen >> -shift;
          words[w] = __reduce_or_sync(0xffffffffu,
                                      static_cast<uint32_t>(bits & ((1ull << (16 * kSlices)) - 1)));
        }
        const uint32_t vb = __ballot_sync(0xffffffffu, valid);
        if (lane == 0) {
          *reinterpret_cast<uint4*>(tile_mask + 4 * stage) =
              make_uint4(words[0], words[1], words[2], words[3]);
          mbar_arrive_expect_tx(&full[stage],
                                static_cast<uint32_t>(__popc(vb) * rpb * L_::kRowBytes * 2));
        }
        __syncwarp();
        if (valid) {
          const int32_t row = bid * bs + (first & (bs - 1));
          uint8_t* st = smem + stage * L_::kStageBytes + start * 128;
          tma_load_3d(st, &tm_k, 0, g, row, &full[stage], pol);
          if (!kFp8) tma_load_3d(st + L_::kHalf, &tm_k, 64, g, row, &full[stage], pol);
          tma_load_3d(st + L_::kVOffset, &tm_v, 0, g, row, &full[stage], pol);
          if (!kFp8)
            tma_load_3d(st + L_::kVOffset + L_::kHalf, &tm_v, 64, g, row, &full[stage], pol);
        }
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.err, PA_DEVERR_WAIT_TIMEOUT);
    }
    // The last copies are waited for (bounded) before this warp ends, whoever gave up: the
    // CTA's shared memory must not be handed on before they have landed.
    if (lane == 0) {
      for (int t = max(0, u - kStages); t < u; ++t)
        mbar_wait_bounded_long(&full[t % kStages], (t / kStages) & 1, nullptr);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int hq0 = g * G;
  // sequences without tokens: zero rows (chunk c takes b = c mod C)
  for (int b = c; b < qp.num_seqs; b += chunks) {
    if (units_of<WindowRows>(qp, b) == 0) {
      const int64_t row = static_cast<int64_t>(b) * p.num_q_heads + hq0;
      for (int i = threadIdx.x; i < G * (kD / 8); i += kConsumers)
        reinterpret_cast<uint4*>(p.out + row * kD)[i] = make_uint4(0u, 0u, 0u, 0u);
      if (!qp.whole && threadIdx.x == 0)
        qp.info[static_cast<int64_t>(g) * qp.num_seqs + b] = 0;
    }
  }

  const int gq = lane >> 2;  // mma groupID
  const int tq = lane & 3;   // thread in group
  const int r0 = warp * 16 * kSlices;  // this warp's places of a tile
  // ldmatrix rows of this lane (16-byte unit u of row r sits at u ^ (r & 7))
  const int sw = lane & 7;
  const uint32_t k_row = static_cast<uint32_t>((r0 + (lane & 15)) * 128);
  const uint32_t v_row =
      kFp8 ? k_row : static_cast<uint32_t>((r0 + (lane & 7) + 8 * (lane >> 4)) * 128);
  const int hi16 = lane >> 4;
  const int v_hi = (lane >> 3) & 1;
  const uint32_t smem_base = smem_u32(smem);
  const float v_scale = kFp8 && p.v_scale != nullptr ? __ldg(p.v_scale) : 1.f;
  const float k_scale = kFp8 && p.k_scale != nullptr ? __ldg(p.k_scale) : 1.f;

  Walk walk(sched);
  Piece pc;
  int stage = 0;  // of the next tile
  uint32_t phase = 0u;
  bool ok = true;
  while (next_piece<WindowRows>(qp, walk, pc)) {
    float o[8][NT][4];
    float m[NT][2], l[NT][2];  // m: running maximum - kLift
    // q as the B operand.  bf16: b0 = q[head gq][16kk + 2tq .. + 1], b1 = [.. + 8].  e4m3: the
    // k index of every 16-wide step is permuted to match how K arrives (below): b0 =
    // q[16kk + 4tq .. + 1], b1 = q[16kk + 4tq + 2 .. + 3], in fp16 after a power of two
    // that puts the piece's largest |q| in [2^14, 2^15) (undone in the score scale).
    uint32_t qb[NT][8][2];
    float score_scale = p.scale_log2;
    {
      float qmax = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = nt * 8 + gq;
        const uint32_t* qrow = reinterpret_cast<const uint32_t*>(
            p.q + (static_cast<int64_t>(pc.b) * p.num_q_heads + hq0 + (h < G ? h : 0)) * kD);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          if constexpr (kFp8) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(qrow + 8 * kk + 2 * tq));
            qb[nt][kk][0] = h < G ? w.x : 0u;
            qb[nt][kk][1] = h < G ? w.y : 0u;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              qmax = fmaxf(qmax, fmaxf(fabsf(__uint_as_float(qb[nt][kk][i] << 16)),
                                       fabsf(__uint_as_float(qb[nt][kk][i] & 0xFFFF0000u))));
          } else {
            qb[nt][kk][0] = h < G ? __ldg(qrow + 8 * kk + tq) : 0u;
            qb[nt][kk][1] = h < G ? __ldg(qrow + 8 * kk + tq + 4) : 0u;
          }
        }
      }
      if constexpr (kFp8) {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
          qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, off));
        // 2^e with e = 14 - floor(log2(qmax)); finite non-zero q only
        int e = 0;
        if (qmax > 0.f && qmax <= 3.0e38f)
          e = min(14 - (static_cast<int>((__float_as_uint(qmax) >> 23) & 0xFF) - 127), 126);
        const float up = ldexpf(1.0f, e);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t w = qb[nt][kk][i];
              qb[nt][kk][i] =
                  pack_f16x2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
            }
        score_scale = p.scale_log2 * k_scale * ldexpf(1.0f, -e);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nt][j] = kNoMaximum;
        l[nt][j] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.f;
    }

    // The warp's places of a tile.  kFull: every one is visible.
    auto tile = [&](auto full_tag, const uint32_t st, const uint32_t mask) {
      constexpr bool kFull = decltype(full_tag)::value;
      float s[kSlices][NT][4];  // scores of rows gq (0, 1) and gq + 8 (2, 3), heads 2tq, 2tq + 1
      bool high = false;
#pragma unroll
      for (int sl = 0; sl < kSlices; ++sl) {
        const uint32_t kbase = st + sl * 16 * 128 + k_row;
        float s0[NT][4], s1[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s0[nt][i] = s1[nt][i] = 0.f;
        if constexpr (kFp8) {
          // One ldmatrix.x4 over 32 bytes of 16 rows (byte pairs as b16) gives each lane four
          // consecutive codes per row and 16-byte group: row gq in r[0] / r[2], row
          // gq + 8 in r[1] / r[3].  In a 16-wide k-step the codes 4tq .. 4tq + 3 serve as
          // k = 2tq, 2tq + 1, 2tq + 8, 2tq + 9 -- the permutation q's fragments use.
#pragma unroll
          for (int k2 = 0; k2 < 4; ++k2) {
            uint32_t r[4];
            ldsm_x4(kbase + ((static_cast<uint32_t>(2 * k2 + hi16) ^ sw) << 4), r);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t a[4];
              e4m3x4_to_f16x2x2(r[2 * half], a[0], a[2]);
              e4m3x4_to_f16x2x2(r[2 * half + 1], a[1], a[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(half ? s1[nt] : s0[nt], a, qb[nt][2 * k2 + half][0],
                              qb[nt][2 * k2 + half][1]);
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            uint32_t a[4];
            ldsm_x4(kbase + (kk >> 2) * L_::kHalf +
                        ((static_cast<uint32_t>(((2 * kk) & 7) + hi16) ^ sw) << 4),
                    a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_bf16_16816((kk & 1) ? s1[nt] : s0[nt], a, qb[nt][kk][0], qb[nt][kk][1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 4; ++i) s[sl][nt][i] = (s0[nt][i] + s1[nt][i]) * score_scale;
          if (!kFull) {
            const uint32_t m16 = mask >> (16 * sl);
            if (!((m16 >> gq) & 1u)) s[sl][nt][0] = s[sl][nt][1] = -INFINITY;
            if (!((m16 >> (gq + 8)) & 1u)) s[sl][nt][2] = s[sl][nt][3] = -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
            high |= fmaxf(s[sl][nt][j], s[sl][nt][j + 2]) > m[nt][j] + (kLift + kRescaleLog2);
        }
      }
      // ---- running maximum: moved when a score beats it by 2^kRescaleLog2 (always on the
      // first); whether any does is one vote
      if (__any_sync(0xffffffffu, high)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
#pragma unroll
            for (int sl = 1; sl < kSlices; ++sl)
              mx = fmaxf(mx, fmaxf(s[sl][nt][j], s[sl][nt][j + 2]));
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1)
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            if (mx > m[nt][j] + (kLift + kRescaleLog2)) {
              const float corr = exp2f(m[nt][j] - (mx - kLift));
              l[nt][j] *= corr;
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
      for (int sl = 0; sl < kSlices; ++sl) {
        const uint32_t vbase = st + L_::kVOffset + sl * 16 * 128 + v_row;
        uint32_t pb[NT][2];
        [[maybe_unused]] uint32_t pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = ex2(s[sl][nt][i] - m[nt][i & 1]);
          l[nt][0] += e[0] + e[2];
          l[nt][1] += e[1] + e[3];
          // (place, heads) pairs to the B operand's (places, head) pairs
          if constexpr (kFp8) {
            pb[nt][0] = transpose8(pack_f16x2(e[0], e[1]));
            pb[nt][1] = transpose8(pack_f16x2(e[2], e[3]));
          } else {
            // hi = bf16(p), lo = bf16(p - hi): together about 16 bits of each weight
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t hi = pack_bf16x2(e[2 * i], e[2 * i + 1]);
              pb[nt][i] = transpose8(hi);
              pl[nt][i] = transpose8(pack_bf16x2(e[2 * i] - __uint_as_float(hi << 16),
                                                 e[2 * i + 1] - __uint_as_float(hi & 0xFFFF0000u)));
            }
          }
        }
        // ---- O^T += V^T . P^T
        if constexpr (kFp8) {
          // ldmatrix.trans of byte pairs gives lane (gq, tq), for places 2tq, 2tq + 1 (+ 8 in
          // r[1], r[3]), the codes of head elements 2gq and 2gq + 1 of a 16-element unit: A
          // row gq of an m-tile carries element 16mt + 2gq, row gq + 8 the one after it.
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t r[4];
            ldsm_x4_trans(vbase + ((static_cast<uint32_t>(2 * j + hi16) ^ sw) << 4), r);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t a[4];
              e4m3x4_to_f16x2x2(__byte_perm(r[2 * h], 0u, 0x3120u), a[0], a[1]);
              e4m3x4_to_f16x2x2(__byte_perm(r[2 * h + 1], 0u, 0x3120u), a[2], a[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(o[2 * j + h][nt], a, pb[nt][0], pb[nt][1]);
            }
          }
        } else {
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            uint32_t a[4];
            ldsm_x4_trans(vbase + (mt >> 2) * L_::kHalf +
                              ((static_cast<uint32_t>(((2 * mt) & 7) + v_hi) ^ sw) << 4),
                          a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_bf16_16816(o[mt][nt], a, pb[nt][0], pb[nt][1]);
              mma_bf16_16816(o[mt][nt], a, pl[nt][0], pl[nt][1]);
            }
          }
        }
      }
    };

    constexpr uint32_t kAll = kSlices == 2 ? 0xFFFFFFFFu : 0xFFFFu;
    for (int at = pc.tok_begin; ok && at < pc.tok_end; at += kTile) {
      const bool w_ok = mbar_wait_bounded(&full[stage], phase, abort_flag);
      if (!__all_sync(0xffffffffu, w_ok)) {
        ok = false;
        break;
      }
      const uint32_t mask = tile_mask[4 * stage + warp];
      const uint32_t st = smem_base + stage * L_::kStageBytes;
      if (mask == kAll) {
        tile(std::true_type{}, st, mask);
      } else if (mask != 0u) {
        // rows that are not seen: zero their values (they or the ring's leftovers could be
        // NaN, and 0 x NaN would poison the sums)
        uint8_t* vrow0 = smem + stage * L_::kStageBytes + L_::kVOffset + r0 * 128;
        constexpr int kUnits = L_::kRowBytes / 16;
        for (int i = lane; i < 16 * kSlices * kUnits; i += 32) {
          const int r = i / kUnits, unit = i % kUnits;
          if (!((mask >> r) & 1u))
            *reinterpret_cast<uint4*>(vrow0 + (unit >> 3) * L_::kHalf + r * 128 + (unit & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
        tile(std::false_type{}, st, mask);
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

    // ---- the accumulators of the four warps joined in shared memory, kRound head
    // elements at a time
    constexpr int GH = L_::kHeads, kRound = L_::kRound, kPitch = L_::kPitch;
    float* red = reinterpret_cast<float*>(smem + L_::kRedOffset);  // [warp][GH][kPitch]
    float* red_m = reinterpret_cast<float*>(smem + L_::kStatOffset);
    float* red_l = red_m + kConsumerWarps * GH;
    const int c_first = qp.whole ? c : chunk_of(pc.first, pc.b, total, parts);
    const int c_last = qp.whole ? c : chunk_of(pc.last, pc.b, total, parts);
    const int slot = slot_of_piece(chunks, qp.num_seqs, pc.b, c_first, c);
    if (!qp.whole && c == c_first && threadIdx.x == 0)
      qp.info[static_cast<int64_t>(g) * qp.num_seqs + pc.b] = info_of(c_first, c_last);
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
    for (int v = 0; v < kD / kRound; ++v) {
      // (a barrier has passed since the last reads of this memory)
#pragma unroll
      for (int mt = 0; mt < kRound / 16; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int h = nt * 8 + 2 * tq + j;
            float* dst = red + (warp * GH + h) * kPitch + 16 * mt;
            const float x = o[v * (kRound / 16) + mt][nt][j];
            const float y = o[v * (kRound / 16) + mt][nt][j + 2];
            if (h < G) {
              if (kFp8) {
                *reinterpret_cast<float2*>(dst + 2 * gq) = make_float2(x, y);
              } else {
                dst[gq] = x;
                dst[gq + 8] = y;
              }
            }
          }
        }
      }
      consumer_barrier();
      for (int i = threadIdx.x; i < G * (kRound / 4); i += kConsumers) {
        const int h = i / (kRound / 4);
        const int e0 = (i % (kRound / 4)) * 4;
        float M = kNoMaximum;
#pragma unroll
        for (int w = 0; w < kConsumerWarps; ++w) M = fmaxf(M, red_m[w * GH + h]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float Ls = 0.f;
#pragma unroll
        for (int w = 0; w < kConsumerWarps; ++w) {
          const float wt = exp2f(red_m[w * GH + h] - M);
          // (a warp of NaN scores only has no maximum and a sum of NaN, which stays)
          Ls += red_l[w * GH + h] * wt;
          const float4 x = *reinterpret_cast<const float4*>(red + (w * GH + h) * kPitch + e0);
          acc.x += wt * x.x;
          acc.y += wt * x.y;
          acc.z += wt * x.z;
          acc.w += wt * x.w;
        }
        const float inv = Ls == 0.f ? 0.f : v_scale / Ls;  // NaN stays NaN
        acc.x *= inv;
        acc.y *= inv;
        acc.z *= inv;
        acc.w *= inv;
        const int e = kRound * v + e0;
        if (c_first == c_last) {
          const int64_t row = static_cast<int64_t>(pc.b) * p.num_q_heads + hq0 + h;
          *reinterpret_cast<uint2*>(p.out + row * kD + e) =
              make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        } else {
          const int64_t row = (static_cast<int64_t>(g) * qp.slots + slot) * G + h;
          *reinterpret_cast<float4*>(p.ws_o + row * kD + e) = acc;
          if (e == 0) p.ws_lse[row] = Ls == 0.f ? -INFINITY : M + log2f(Ls);
        }
      }
      consumer_barrier();
    }
  }
}

WindowPlan plan_of(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t window,
                   int32_t num_sink, int32_t max_context_len, bool e4m3) {
  const int sms = num_sms_current_device();
  return window_plan(sms > 0 ? sms : 148, num_seqs, num_q_heads, num_kv_heads, window, num_sink,
                     max_context_len, e4m3);
}

template <int NT, bool kFp8>
pa_status launch(const CUtensorMap& mk, const CUtensorMap& mv, const PieceParams& q, int G,
                 int chunks, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_raised{0};
  auto kern = window_decode_kernel<NT, kFp8>;
  if (!ensure_smem_limit(kern, Lay<NT, kFp8>::kAlloc, smem_raised)) return PA_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>(q.d.num_kv_heads), static_cast<unsigned>(chunks));
  kern<<<grid, kThreads, Lay<NT, kFp8>::kAlloc, stream>>>(mk, mv, q, G);
  if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
  if (q.whole) return PA_OK;  // no sequence is split
  // Pieces per sequence are about chunks / num_seqs and two at its ends: a warp merges few, the
  // eight warps of a CTA many (one sequence of 18 pieces: 8.3 us in all, 12.7 with a warp;
  // 64 sequences of two: 46 us with warps, 47 with CTAs).
  if (chunks > 4 * q.num_seqs) {
    const dim3 merge_grid(static_cast<unsigned>(q.d.num_q_heads),
                          static_cast<unsigned>(q.num_seqs < 256 ? q.num_seqs : 256));
    return launch_dependent(merge_pieces_kernel<1, false>, merge_grid, kMergeWarps * 32, stream, q,
                            G, chunks);
  }
  constexpr int kWarps = kMergeThreads / 32;
  const dim3 merge_grid(static_cast<unsigned>((q.d.num_q_heads + kWarps - 1) / kWarps),
                        static_cast<unsigned>(q.num_seqs < 128 ? q.num_seqs : 128));
  return launch_dependent(merge_split_kernel, merge_grid, kMergeThreads, stream, q, G, chunks);
}

}  // namespace

size_t window_decode_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                     int32_t window, int32_t num_sink, int32_t max_context_len) {
  // (the size does not depend on the cache's type)
  return plan_of(num_seqs, num_q_heads, num_kv_heads, window, num_sink, max_context_len, false)
      .bytes;
}

pa_status launch_window_decode(const DecodeArgs& a, int32_t window, int32_t num_sink,
                               int32_t max_context_len, cudaStream_t stream) {
  if (a.num_seqs == 0) return PA_OK;
  if (a.num_seqs > 65535) return PA_ERR_UNSUPPORTED;
  const int32_t G = a.num_q_heads / a.num_kv_heads;
  const int64_t rows = a.num_blocks * a.block_size;
  const int32_t box_rows = a.block_size < 64 ? a.block_size : 64;
  const bool fp8 = a.cache_dtype == PA_FP8_E4M3;
  CUtensorMap mk, mv;
  const auto make = fp8 ? make_kv_map_fp8 : make_kv_map_swizzled;
  if (!make(&mk, a.k_cache, rows, a.num_kv_heads, box_rows) ||
      !make(&mv, a.v_cache, rows, a.num_kv_heads, box_rows))
    return PA_ERR_CUDA;
  const WindowPlan w = plan_of(a.num_seqs, a.num_q_heads, a.num_kv_heads, window, num_sink,
                               max_context_len, fp8);
  PieceParams q{};
  q.d = make_decode_params(a);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  q.d.ws_lse = reinterpret_cast<float*>(ws + w.lse_offset);
  q.d.ws_o = reinterpret_cast<float*>(ws + w.o_offset);
  q.info = reinterpret_cast<int32_t*>(ws + w.info_offset);
  q.num_seqs = a.num_seqs;
  q.slots = w.slots;
  q.whole = w.whole;
  q.window = window;
  q.num_sink = num_sink;
  q.max_len = max_context_len;
  if (G == 16)
    return fp8 ? launch<2, true>(mk, mv, q, G, w.chunks, stream)
               : launch<2, false>(mk, mv, q, G, w.chunks, stream);
  return fp8 ? launch<1, true>(mk, mv, q, G, w.chunks, stream)
             : launch<1, false>(mk, mv, q, G, w.chunks, stream);
}

}  // namespace pa_detail
