// decode_q4.cu -- paged GQA decode attention over a 4-bit cache.
//
// The split scheme, pipeline and merge of decode.cu (one CTA per kv head,
// token range and sequence; a producer warp feeding a shared-memory ring by
// TMA; four consumer warps with an online softmax each; the last CTA merges
// the ranges) over rows of 80 bytes: 64 of codes, then four fp16 pairs
// (s, m), one per group u of 32 elements; an element stands for m + s c.
//
// Scores.  With S_u = sum_{d in u} q_d c_d and Q_u = sum_{d in u} q_d,
//     q . k = sum_u s_u S_u + m_u Q_u.
// A nibble at bits 0-3 (4-7) of a 16-bit half is, read as an fp16 number,
// the subnormal c 2^-24 (c 2^-20): one AND turns two nibbles of a code word
// into an fp16 pair, exactly, and the factors 2^24 and 16 go into the score
// scale and into q.  The products are exact and accumulate in fp32; s and m
// enter in fp32.
//
// Values.  ldmatrix.trans hands a lane the 16-bit units (four codes) of two
// tokens side by side, so one AND-OR per nibble makes the fp16 pair
// (64 + c) of both tokens (bits 4-7 of an fp16 in [64, 128) count units) and
// one fused multiply-add with (s, -64 s) the pair s c, rounded once.  The
// minima need no element work: sum_t p_t m_t,u is one more product, with the
// (s, m) pairs of the rows themselves as the matrix (rows 2u + 1 of its
// result).  The weights are held 2^7 above the running maximum's scale, so
// that fp16 carries them down to 2^-31 of it.
//
// Rows of 80 bytes need no swizzle: eight consecutive rows start in eight
// different groups of four banks (20 r mod 32).
#include <atomic>

#include "decode_common.cuh"

namespace pa_detail {
namespace {

constexpr int kTile = 128;         // tokens per stage, 32 per consumer warp
constexpr int kRow = 80;           // bytes of a cached row
constexpr int kTensorBytes = kTile * kRow;
constexpr float kLift = 7.0f;      // weights are 2^kLift (score - running maximum)

struct Lay {
  static constexpr int kStages = 3;
  static constexpr int kStageBytes = 2 * kTensorBytes;  // K rows, then V rows
  static constexpr int kBarOffset = kStages * kStageBytes;
  static constexpr int kMaskOffset = kBarOffset + 2 * kStages * 8;  // four words per stage
  static constexpr int kFlagOffset = kMaskOffset + kStages * 16;
  static constexpr int kAlloc = kFlagOffset + 16 + 128;  // room to align the base to 128 bytes
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
// the two halves of an fp16 pair in fp32
__device__ __forceinline__ float2 pair_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// 8x8 transpose of a 16-bit fragment across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}

// NT: n-tiles of 8 query heads (G <= 8 -> 1, G = 16 -> 2); kScored: also
// store the scores and each query head's log2-sum-exp.
template <int NT, bool kScored>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
    paged_decode_split_q4_kernel(const __grid_constant__ CUtensorMap tm_k,
                                 const __grid_constant__ CUtensorMap tm_v, const DecodeParams p,
                                 int G) {
  constexpr int kStages = Lay::kStages;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::kBarOffset);
  uint64_t* empty = full + kStages;
  uint32_t* tile_mask = reinterpret_cast<uint32_t*>(smem + Lay::kMaskOffset);
  int* abort_ptr = reinterpret_cast<int*>(smem + Lay::kFlagOffset);

  // kv heads fastest in launch order: the CTAs of one (sequence, range) read
  // neighbouring rows at the same time
  const int g = blockIdx.x;
  const int split = blockIdx.y;
  const int b = blockIdx.z;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int bs = p.block_size;
  const int hq0 = g * G;

  bool clipped;
  const int L = effective_len(p, b, &clipped);
  if (clipped && split == 0 && g == 0 && threadIdx.x == 0)
    atomicOr(p.err, PA_DEVERR_CONTEXT_CLIPPED);
  const int tok_begin = split * p.tokens_per_split;
  const int tok_end = min(tok_begin + p.tokens_per_split, L);
  if (tok_begin >= tok_end) {
    if (split == 0) {  // only when L == 0: a zero row per head
      for (int i = threadIdx.x; i < G * (kD / 8); i += kThreads)
        reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(b) * p.num_q_heads + hq0) * kD)[i] =
            make_uint4(0u, 0u, 0u, 0u);
      if (kScored && threadIdx.x < G)
        p.final_lse[static_cast<int64_t>(b) * p.num_q_heads + hq0 + threadIdx.x] = -INFINITY;
    }
    return;
  }
  const int ntiles = (tok_end - tok_begin + kTile - 1) / kTile;

  if (threadIdx.x == 0) {
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

  const int gq = lane >> 2;  // mma groupID
  const int tq = lane & 3;   // thread in group
  float o[8][NT][4];         // head elements 32u + 4gq + 2h (+1) of m-tile 2u + h
  float z[NT][4];            // sums of p s (even rows) and p m (odd rows) per group
  float m[NT][2], l[NT][2];  // m: running maximum - kLift
  int issued = 0;

  if (warp == kConsumerWarps) {
    // ------------------------------------------------------------ producer
    const int rpb = bs < 64 ? bs : 64;  // rows per box: token ranges start at multiples of 64
    const int nbox = kTile / rpb;
    const uint64_t pol = l2_policy_evict_first();
    if (lane == 0) {
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
    const int32_t* bt = p.block_tables + static_cast<int64_t>(b) * p.max_blocks_per_seq;
    // lane i < nbox: block id of box i of tile t (-1 past the range), read one tile ahead
    auto tile_bid = [&](int t) -> int {
      const int first = tok_begin + t * kTile + lane * rpb;
      return (t < ntiles && lane < nbox && first < tok_end) ? __ldg(bt + (first >> p.log2_bs))
                                                            : -1;
    };
    int bid_next = tile_bid(0);
    bool ok = true;
    for (int t = 0; t < ntiles; ++t) {
      const int stage = t % kStages;
      const int bid = bid_next;
      bid_next = tile_bid(t + 1);
      if (t >= kStages) {
        const bool w_ok = mbar_wait_bounded(&empty[stage], ((t / kStages) - 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, w_ok)) {
          ok = false;
          break;
        }
      }
      const int first = tok_begin + t * kTile + lane * rpb;
      const int rows = lane < nbox ? min(rpb, tok_end - first) : 0;
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
        uint8_t* st = smem + stage * Lay::kStageBytes + lane * rpb * kRow;
        tma_load_3d(st, &tm_k, 0, g, row, &full[stage], pol);
        tma_load_3d(st + kTensorBytes, &tm_v, 0, g, row, &full[stage], pol);
      }
      issued = t + 1;
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.err, PA_DEVERR_WAIT_TIMEOUT);
    }
  } else {
    // ------------------------------------------------------------ consumers
    // q as the B operand: for group u a lane (head gq of the n-tile) holds
    // elements 32u + 8tq + 0..7, paired as the nibbles of a code word are:
    // (0, 4), (1, 5)/16, (2, 6), (3, 7)/16, in fp16 after a power of two per
    // head that puts its largest |q| in [2^14, 2^15).
    uint32_t qb[NT][4][4];
    float qsum[NT][4][2];      // scale_log2 Q_u of heads 2tq, 2tq + 1
    float sscale[NT][2];       // scale_log2 2^(24 - e) of heads 2tq, 2tq + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + gq;
      const uint4* qrow = reinterpret_cast<const uint4*>(
          p.q + (static_cast<int64_t>(b) * p.num_q_heads + hq0 + (h < G ? h : 0)) * kD);
      float qv[4][8];
      float qmax = 0.f;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        to_f32(Vec8<bf16>{__ldg(qrow + 4 * u + tq)}, qv[u]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (h >= G) qv[u][e] = 0.f;
          qmax = fmaxf(qmax, fabsf(qv[u][e]));
        }
      }
      qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 1));
      qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 2));
      int e2 = 0;
      if (qmax > 0.f && qmax <= 3.0e38f)
        e2 = min(14 - (static_cast<int>((__float_as_uint(qmax) >> 23) & 0xFF) - 127), 126);
      const float up = ldexpf(1.0f, e2);
      const float fs = p.scale_log2 * ldexpf(1.0f, 24 - e2);
#pragma unroll
      for (int j = 0; j < 2; ++j) sscale[nt][j] = __shfl_sync(0xffffffffu, fs, 4 * (2 * tq + j));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += qv[u][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= p.scale_log2;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          qsum[nt][u][j] = __shfl_sync(0xffffffffu, sum, 4 * (2 * tq + j));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float f = (k & 1) ? up * 0.0625f : up;
          qb[nt][u][k] = pack_f16x2(qv[u][k] * f, qv[u][k + 4] * f);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nt][j] = -INFINITY;
        l[nt][j] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        z[nt][c] = 0.f;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) o[mt][nt][c] = 0.f;
      }
    }
    // ldmatrix rows and 16-byte columns of this lane (K and V alike): rows
    // (lane & 15), column u + (lane >> 4)
    const uint32_t frag = static_cast<uint32_t>((32 * warp + (lane & 15)) * kRow + 16 * (lane >> 4));
    const uint32_t smem_base = smem_u32(smem);

    bool ok = true;
    for (int t = 0; t < ntiles; ++t) {
      const int stage = t % kStages;
      const bool w_ok = mbar_wait_bounded(&full[stage], (t / kStages) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, w_ok)) {
        ok = false;
        break;
      }
      const uint32_t mask32 = tile_mask[4 * stage + warp];
      uint8_t* st_k = smem + stage * Lay::kStageBytes;
      uint8_t* st_v = st_k + kTensorBytes;
      bool smem_written = false;
#pragma unroll 1
      for (int sl = 0; sl < 2; ++sl) {
        const uint32_t mask16 = (mask32 >> (16 * sl)) & 0xFFFFu;
        const int r0 = 32 * warp + 16 * sl;
        const int tok0 = tok_begin + t * kTile + r0;
        if (mask16 == 0u) {  // no token of the slice is there
          if constexpr (kScored) {
            const float none[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              store_scores(p, b, g, G, tok0, gq, tok_end - tok0, nt * 8 + 2 * tq, none);
          }
          continue;
        }
        if (mask16 != 0xFFFFu) {
          // rows without a token: s = m = 0 makes their values 0 (the ring's
          // leftovers could be NaN, and 0 x NaN would poison the sums)
          if (lane < 16 && !((mask16 >> lane) & 1u))
            *reinterpret_cast<uint4*>(st_v + (r0 + lane) * kRow + 64) = make_uint4(0u, 0u, 0u, 0u);
          smem_written = true;
          __syncwarp();
        }
        const uint32_t kaddr = smem_base + stage * Lay::kStageBytes + frag + sl * 16 * kRow;
        const uint32_t vaddr = kaddr + kTensorBytes;
        // ---- S_u = codes . q, one accumulator per group
        float su[NT][4][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int c = 0; c < 4; ++c) su[nt][u][c] = 0.f;
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
              mma_f16_16816(su[nt][u2 + i], a0, qb[nt][u2 + i][0], qb[nt][u2 + i][1]);
              mma_f16_16816(su[nt][u2 + i], a1, qb[nt][u2 + i][2], qb[nt][u2 + i][3]);
            }
          }
        }
        // ---- scores: sum_u s_u S_u and m_u Q_u in fp32
        float ss[2][4], mm[2][4];  // rows gq, gq + 8
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(st_k + (r0 + gq + 8 * i) * kRow + 64);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float2 f = pair_f32(ww[u]);
            ss[i][u] = f.x;
            mm[i][u] = f.y;
          }
        }
        const bool v0 = (mask16 >> gq) & 1u;        // token r0 + gq
        const bool v1 = (mask16 >> (gq + 8)) & 1u;  // token r0 + gq + 8
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float s[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float a = 0.f, q = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              a = fmaf(ss[c >> 1][u], su[nt][u][c], a);
              q = fmaf(mm[c >> 1][u], qsum[nt][u][c & 1], q);
            }
            s[c] = fmaf(a, sscale[nt][c & 1], q);
          }
          if (!v0) s[0] = s[1] = -INFINITY;
          if (!v1) s[2] = s[3] = -INFINITY;
          if constexpr (kScored)
            store_scores(p, b, g, G, tok0, gq, tok_end - tok0, nt * 8 + 2 * tq, s);
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
          const float p0 = v0 ? exp2f(s[0] - m[nt][0]) : 0.f;
          const float p1 = v0 ? exp2f(s[1] - m[nt][1]) : 0.f;
          const float p2 = v1 ? exp2f(s[2] - m[nt][0]) : 0.f;
          const float p3 = v1 ? exp2f(s[3] - m[nt][1]) : 0.f;
          l[nt][0] += p0 + p2;
          l[nt][1] += p1 + p3;
          // (token, heads) pairs to the B operand's (tokens, head) pairs
          pb[nt][0] = transpose8(pack_f16x2(p0, p1));
          pb[nt][1] = transpose8(pack_f16x2(p2, p3));
        }
        // ---- sum p m (and p s): the rows' (s, m) pairs as a matrix
        {
          uint32_t r[4];
          ldsm_x4_trans(vaddr - 16 * (lane >> 4) + 64, r);  // rows r0 + (lane & 15)
          const uint32_t a[4] = {r[0], 0u, r[1], 0u};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16_16816(z[nt], a, pb[nt][0], pb[nt][1]);
        }
        // ---- O^T += (s c)^T . P^T
        uint32_t sv[2][4], sn[2][4];  // (s, s') and -64 (s, s') of tokens 2tq, 2tq + 1 (+ 8)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* row = st_v + (r0 + 2 * tq + 8 * i) * kRow + 64;
          const uint4 x = *reinterpret_cast<const uint4*>(row);
          const uint4 y = *reinterpret_cast<const uint4*>(row + kRow);
          sv[i][0] = __byte_perm(x.x, y.x, 0x5410u);
          sv[i][1] = __byte_perm(x.y, y.y, 0x5410u);
          sv[i][2] = __byte_perm(x.z, y.z, 0x5410u);
          sv[i][3] = __byte_perm(x.w, y.w, 0x5410u);
#pragma unroll
          for (int u = 0; u < 4; ++u) sn[i][u] = hmul2(sv[i][u], 0xD400D400u);  // -64
        }
#pragma unroll
        for (int u2 = 0; u2 < 4; u2 += 2) {
          uint32_t r[4];  // (tokens 2tq, u2), (tokens 2tq + 8, u2), the same of u2 + 1
          ldsm_x4_trans(vaddr + 16 * u2, r);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int u = u2 + i;
            uint32_t x[2][4];  // s c of tokens 2tq.. (+8), element 32u + 4gq + k
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w = r[2 * i + j];
              x[j][0] = hfma2(((w << 4) & 0x00F000F0u) | 0x54005400u, sv[j][u], sn[j][u]);
              x[j][1] = hfma2((w & 0x00F000F0u) | 0x54005400u, sv[j][u], sn[j][u]);
              x[j][2] = hfma2(((w >> 4) & 0x00F000F0u) | 0x54005400u, sv[j][u], sn[j][u]);
              x[j][3] = hfma2(((w >> 8) & 0x00F000F0u) | 0x54005400u, sv[j][u], sn[j][u]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a[4] = {x[0][2 * h], x[0][2 * h + 1], x[1][2 * h], x[1][2 * h + 1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(o[2 * u + h][nt], a, pb[nt][0], pb[nt][1]);
            }
          }
        }
      }
      if (smem_written) fence_proxy_async_smem();  // ordinary stores before the next TMA
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) atomicOr(p.err, PA_DEVERR_WAIT_TIMEOUT);
    }
  }

  __syncthreads();
  if (*abort_flag) {
    // wait (bounded) for copies already in flight, then leave an empty
    // partial so that the split count below still completes
    if (warp == kConsumerWarps && lane == 0) {
      for (int t = max(0, issued - kStages); t < issued; ++t)
        mbar_wait_bounded(&full[t % kStages], (t / kStages) & 1, nullptr);
    }
    if (p.num_splits > 1 && threadIdx.x < G)
      p.ws_lse[(static_cast<int64_t>(b) * p.num_q_heads + hq0 + threadIdx.x) * p.num_splits +
               split] = -INFINITY;
  } else {
    // ---- the four warps' (maximum, sum, accumulator) joined in shared memory
    constexpr int GH = NT * 8;
    float* red = reinterpret_cast<float*>(smem);            // [warp][h][d]
    float* red_m = red + kConsumerWarps * GH * kD;          // [warp][h]
    float* red_l = red_m + kConsumerWarps * GH;
    float* red_w = red_l + kConsumerWarps * GH;
    float* fin = red_w + kConsumerWarps * GH;               // [h][2]
    static_assert((kConsumerWarps * GH * (kD + 3) + 2 * GH) * 4 <= Lay::kBarOffset,
                  "the join fits the ring");
    if (warp < kConsumerWarps) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float lv = l[nt][j];
          lv += __shfl_xor_sync(0xffffffffu, lv, 4);
          lv += __shfl_xor_sync(0xffffffffu, lv, 8);
          lv += __shfl_xor_sync(0xffffffffu, lv, 16);
          const int h = nt * 8 + 2 * tq + j;
          if (gq == 0) {
            red_m[warp * GH + h] = m[nt][j];
            red_l[warp * GH + h] = lv;
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float zu = __shfl_sync(0xffffffffu, z[nt][j], 4 * (2 * u + 1) + tq);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              float* dst = red + (warp * GH + h) * kD + 32 * u + 4 * gq + 2 * hh;
              dst[0] = o[2 * u + hh][nt][j] + zu;
              dst[1] = o[2 * u + hh][nt][j + 2] + zu;
            }
          }
        }
      }
    }
    __syncthreads();
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
        Ls += red_l[w * GH + h] * wt;
      }
      fin[2 * h] = M;
      fin[2 * h + 1] = Ls;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * (kD / 4); i += kThreads) {
      const int h = i / (kD / 4);
      const int e0 = (i % (kD / 4)) * 4;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kConsumerWarps; ++w) {
        const float wt = red_w[w * GH + h];
        const float4 v = *reinterpret_cast<const float4*>(red + (w * GH + h) * kD + e0);
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
      const int64_t row = static_cast<int64_t>(b) * p.num_q_heads + hq0 + h;
      if (p.num_splits == 1) {
        *reinterpret_cast<uint2*>(p.out + row * kD + e0) =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        if (kScored && e0 == 0)
          p.final_lse[row] = Ls == 0.f ? -INFINITY : fin[2 * h] + log2f(Ls);
      } else {
        const int64_t slot = row * p.num_splits + split;
        *reinterpret_cast<float4*>(p.ws_o + slot * kD + e0) = acc;
        if (e0 == 0) p.ws_lse[slot] = Ls == 0.f ? -INFINITY : fin[2 * h] + log2f(Ls);
      }
    }
  }
  if (p.num_splits == 1) return;
  count_and_merge<kScored>(p, b, g, hq0, G, L, abort_ptr + 1, warp, lane);
}

template <int NT, bool kScored>
pa_status launch_split_q4(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeParams& p,
                          dim3 grid, int G, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_raised{0};
  auto kern = paged_decode_split_q4_kernel<NT, kScored>;
  if (!ensure_smem_limit(kern, Lay::kAlloc, smem_raised)) return PA_ERR_CUDA;
  kern<<<grid, kThreads, Lay::kAlloc, stream>>>(mk, mv, p, G);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

pa_status launch_paged_decode_q4(const DecodeArgs& a, cudaStream_t stream) {
  if (a.num_seqs == 0) return PA_OK;
  if (a.plan.num_splits > 65535 || a.num_seqs > 65535) return PA_ERR_UNSUPPORTED;
  const int32_t G = a.num_q_heads / a.num_kv_heads;
  const int64_t rows = a.num_blocks * a.block_size;
  const int32_t box_rows = a.block_size < 64 ? a.block_size : 64;
  CUtensorMap mk, mv;
  if (!make_kv_map_q4(&mk, a.k_cache, rows, a.num_kv_heads, box_rows) ||
      !make_kv_map_q4(&mv, a.v_cache, rows, a.num_kv_heads, box_rows))
    return PA_ERR_CUDA;
  const DecodeParams p = make_decode_params(a);
  const dim3 grid(static_cast<unsigned>(a.num_kv_heads), static_cast<unsigned>(a.plan.num_splits),
                  static_cast<unsigned>(a.num_seqs));
  if (a.scores != nullptr)
    return G <= 8 ? launch_split_q4<1, true>(mk, mv, p, grid, G, stream)
                  : launch_split_q4<2, true>(mk, mv, p, grid, G, stream);
  return G <= 8 ? launch_split_q4<1, false>(mk, mv, p, grid, G, stream)
                : launch_split_q4<2, false>(mk, mv, p, grid, G, stream);
}

}  // namespace pa_detail
