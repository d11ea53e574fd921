// decode_common.cuh -- what the paged decode attention kernels share: their
// parameters, the clipped context length, and the merge of the splits by the
// last CTA of each (sequence, kv head).
#pragma once

#include "pa_internal.cuh"

namespace pa_detail {

using namespace pa;

constexpr int kD = 128;                 // head size handled by the decode kernels
constexpr int kConsumerWarps = 4;
constexpr int kThreads = (kConsumerWarps + 1) * 32;
constexpr float kRescaleLog2 = 8.0f;    // lazy-rescale threshold (base-2 units)
constexpr size_t kWorkspaceHeader = 256;  // error word + padding

struct DecodeParams {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* ws_lse;
  float* ws_o;
  unsigned* counters;  // [B, H_KV] split arrivals, zero between calls
  unsigned* err;
  int64_t num_blocks;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t block_size;
  int32_t log2_bs;
  int32_t max_blocks_per_seq;
  int32_t num_splits;
  int32_t tokens_per_split;
  float scale_log2;
  const float* k_scale;  // quantised cache: code * k_scale is the value (else null)
  const float* v_scale;
  // fused decode step (else null): each sequence's newest K/V row
  // [B, H_KV, d] bf16, written at slot_mapping[b] before it is attended to
  const __nv_bfloat16* new_k;
  const __nv_bfloat16* new_v;
  const int64_t* slot_mapping;
  void* k_cache;
  void* v_cache;
  // accumulated attention weights (else null): the scores in base 2, -inf
  // where there is no token, [B, H_KV, score_len, G]; and each query head's
  // log2-sum-exp [B, H_Q]
  float* scores;
  float* final_lse;
  int64_t score_len;
};


// context length used by both kernels: clipped to the plan and the table
__device__ __forceinline__ int effective_len(const DecodeParams& p, int b, bool* clipped) {
  int L = __ldg(p.context_lens + b);
  L = L < 0 ? 0 : L;
  const int64_t cap = min(static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size,
                          static_cast<int64_t>(p.num_splits) * p.tokens_per_split);
  *clipped = static_cast<int64_t>(L) > cap;
  return *clipped ? static_cast<int>(cap) : L;
}

// Scores of one 16-token slice, from the accumulator layout of the score
// products: this lane holds tokens row and row + 8 of heads h, h + 1 (s[0],
// s[1] and s[2], s[3]).  Rows at or past `rows` belong to another range.
__device__ __forceinline__ void store_scores(const DecodeParams& p, int b, int g, int G, int tok0,
                                             int row, int rows, int h, const float (&s)[4]) {
  if (h >= G) return;
  float* dst =
      p.scores +
      ((static_cast<int64_t>(b) * p.num_kv_heads + g) * p.score_len + tok0 + row) * G + h;
#pragma unroll
  for (int i = 0; i < 2; ++i, dst += 8 * G) {
    if (row + 8 * i >= rows) break;
    if (G == 1) {
      dst[0] = s[2 * i];
    } else {  // G and h are even
      *reinterpret_cast<float2*>(dst) = make_float2(s[2 * i], s[2 * i + 1]);
    }
  }
}

// The parameters of a call (workspace split up, scale in base 2).
DecodeParams make_decode_params(const DecodeArgs& a);

// Merge of one (sequence, query head) by one warp: weights 2^(lse_s - max)
// over the n splits that hold tokens, out = sum_s w_s o_s / sum_s w_s,
// rounded to bf16.  Partials are read through L2 (__ldcg): other CTAs wrote
// them during this launch.
template <bool kScored>
__device__ __forceinline__ void merge_splits_warp(const DecodeParams& p, int64_t bh, int n,
                                                  int lane) {
  const float* lse = p.ws_lse + bh * p.num_splits;
  const float* o = p.ws_o + bh * p.num_splits * kD;
  float M = -INFINITY;
  // (a NaN lse, of a split whose sum is NaN, is carried to the output)
  for (int s = lane; s < n; s += 32) M = max_nan(M, __ldcg(lse + s));
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, off));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float W = 0.f;
  if (M != -INFINITY) {
    for (int s0 = 0; s0 < n; s0 += 32) {
      const int my = s0 + lane;
      const float wl = my < n ? exp2f(__ldcg(lse + my) - M) : 0.f;
      const int cnt = min(32, n - s0);
      int k = 0;
      for (; k + 8 <= cnt; k += 8) {
        float4 v[8];
        float w[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          v[u] = __ldcg(reinterpret_cast<const float4*>(o + static_cast<int64_t>(s0 + k + u) * kD) +
                        lane);
          w[u] = __shfl_sync(0xffffffffu, wl, k + u);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          W += w[u];
          acc.x += w[u] * v[u].x;
          acc.y += w[u] * v[u].y;
          acc.z += w[u] * v[u].z;
          acc.w += w[u] * v[u].w;
        }
      }
      for (; k < cnt; ++k) {
        const float4 v =
            __ldcg(reinterpret_cast<const float4*>(o + static_cast<int64_t>(s0 + k) * kD) + lane);
        const float w = __shfl_sync(0xffffffffu, wl, k);
        W += w;
        acc.x += w * v.x;
        acc.y += w * v.y;
        acc.z += w * v.z;
        acc.w += w * v.w;
      }
    }
  }
  if (kScored && lane == 0) p.final_lse[bh] = W == 0.f ? -INFINITY : M + log2f(W);
  const float inv = W > 0.f ? 1.f / W : 0.f;
  *reinterpret_cast<uint2*>(p.out + bh * kD + lane * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

// Counts this CTA's partial in its (sequence, kv head)'s counter; the CTA that
// completes the count merges the splits of its G query heads and returns the
// counter to zero.  Every thread of the CTA calls it; last_flag: one int of
// shared memory nothing else uses.
template <bool kScored>
__device__ __forceinline__ void count_and_merge(const DecodeParams& p, int b, int g, int hq0, int G,
                                                int L, int* last_flag, int warp, int lane) {
  __syncthreads();  // every partial of this CTA is written
  const int n_valid = (L + p.tokens_per_split - 1) / p.tokens_per_split;
  if (threadIdx.x == 0) {
    __threadfence();
    unsigned* ctr = p.counters + static_cast<int64_t>(b) * p.num_kv_heads + g;
    const unsigned prev = atomicAdd(ctr, 1u);
    const bool last = prev + 1u == static_cast<unsigned>(n_valid);
    if (last) {
      atomicExch(ctr, 0u);
      __threadfence();
    }
    *last_flag = last ? 1 : 0;
  }
  __syncthreads();
  if (*last_flag) {
    for (int h = warp; h < G; h += kThreads / 32)
      merge_splits_warp<kScored>(p, static_cast<int64_t>(b) * p.num_q_heads + hq0 + h, n_valid, lane);
  }
}

}  // namespace pa_detail
