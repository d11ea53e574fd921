// decode_pieces.cuh -- what the decode kernels with a balanced cut share (decode_q4.cu,
// decode_window.cu): finding a chunk's pieces, walking them, and the merge of sequences that were
// split over chunks.
#pragma once

#include "pa_internal.cuh"
#include "q4_cut.h"

namespace pa_detail {
namespace pieces {

using namespace pa;
using namespace decode;
using namespace q4cut;

static_assert(kUnit == 64, "boxes are up to 64 rows, pieces start at multiples of them");
static_assert(kPartialFloats == kD, "a partial row is a head");
constexpr int kConsumers = kConsumerWarps * 32;

struct PieceParams {
  DecodeParams d;
  int32_t num_seqs;
  int32_t slots;  // partial slots per kv head
  int32_t* info;  // [H_KV / HP, B]: chunk of the first piece << 16 | pieces, 0 if not split
  bool whole;     // no partials: chunks begin at sequence starts
  // the rows of a context that a window leaves (window 0: all of them)
  int32_t window, num_sink, max_len;
};

// `Rows::len`: how many rows of sequence b are attended to, and whether its length was clipped
struct WholeContext {
  static __device__ __forceinline__ int len(const PieceParams& q, int b, bool* clipped) {
    return effective_len(q.d, b, clipped);
  }
};

__device__ __forceinline__ void consumer_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
}

// 8x8 transpose of a 16-bit fragment across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
// ------------------------------------------------------------ the balanced cut --
// (the arithmetic and its invariants: q4_cut.h)
template <typename Rows>
__device__ __forceinline__ int units_of(const PieceParams& q, int b) {
  bool clipped;
  return units_of_len(Rows::len(q, b, &clipped));
}

// Warp 0: the first unit of chunks c and c + 1.  sched: total, first unit of c,
// first unit of c + 1, then the first one's sequence and the units before that.
template <typename Rows>
__device__ __forceinline__ void find_chunk(const PieceParams& q, int c, int chunks, int lane,
                                           int64_t* sched) {
  const DecodeParams& p = q.d;
  if (q.whole && chunks == q.num_seqs) {  // one sequence per chunk: nothing to cut
    bool clipped;
    const int n = units_of_len(Rows::len(q, c, &clipped));
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
      held[k] = units_of_len(Rows::len(q, b, &clipped));
      any_clipped |= clipped;
    }
    units += held[k];
  }
  for (int b = lane + 128; b < q.num_seqs; b += 32) {
    bool clipped;
    units += units_of_len(Rows::len(q, b, &clipped));
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
                  : b < q.num_seqs ? units_of<Rows>(q, b)
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
template <typename Rows>
__device__ __forceinline__ bool next_piece(const PieceParams& q, Walk& w, Piece& pc) {
  while (w.t < w.end) {
    bool clipped;
    const int L = Rows::len(q, w.b, &clipped);
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
    merge_pieces_kernel(const __grid_constant__ PieceParams qp, int G, int chunks) {
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

}  // namespace pieces
}  // namespace pa_detail
