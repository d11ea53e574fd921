// decode_scored.cu -- decode attention that adds up each cached token's
// attention weight.
//
// A token's weight needs its sequence's final log-sum-exp, which no CTA knows
// while it holds the scores.  So the split kernels store the scores as they
// go (fp32, G per token and kv head, beside 160 to 512 bytes of K/V read) and
// the merge stores each head's log2-sum-exp; this second launch forms
//     sums_out[b, g, t] = (t >= L - num_new ? 0 : sums_in[b, g, t])
//                         + sum_h 2^(score[b, g, t, h] - lse[b, h])
// in a fixed order (no atomics).
#include "decode_common.cuh"

namespace pa_detail {
namespace {

constexpr int kSumThreads = 256;

struct SumsParams {
  float* out;
  const float* in;
  int32_t sums_len;
  int32_t num_new;
};

template <int G>
__global__ void __launch_bounds__(kSumThreads) add_weights_kernel(const DecodeParams p,
                                                                  const SumsParams w) {
  const int g = blockIdx.y, b = blockIdx.z;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores and sums of logs are there
  bool clipped;
  const int L = effective_len(p, b, &clipped);
  const int t = blockIdx.x * kSumThreads + threadIdx.x;
  if (t >= min(L, w.sums_len)) return;
  const float* lse = p.final_lse + static_cast<int64_t>(b) * p.num_q_heads + g * G;
  const float* s = p.scores +
                   ((static_cast<int64_t>(b) * p.num_kv_heads + g) * p.score_len + t) * G;
  float v[G];
  if constexpr (G % 4 == 0) {
#pragma unroll
    for (int h = 0; h < G; h += 4) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(s + h));
      v[h] = x.x;
      v[h + 1] = x.y;
      v[h + 2] = x.z;
      v[h + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int h = 0; h < G; ++h) v[h] = __ldcs(s + h);
  }
  float weight = 0.f;
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const float m = __ldcg(lse + h);
    weight += m == -INFINITY ? 0.f : exp2f(v[h] - m);  // -inf: no token is there
  }
  const int64_t at = (static_cast<int64_t>(b) * p.num_kv_heads + g) * w.sums_len + t;
  const float old = t >= L - w.num_new ? 0.f : w.in[at];
  w.out[at] = old + weight;
}

template <int G>
pa_status launch_add(const DecodeParams& p, const SumsParams& w, int32_t num_seqs, int64_t tokens,
                     cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((tokens + kSumThreads - 1) / kSumThreads),
                  static_cast<unsigned>(p.num_kv_heads), static_cast<unsigned>(num_seqs));
  return launch_dependent(add_weights_kernel<G>, grid, kSumThreads, stream, p, w);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// Workspace: [decode workspace, padded] [log2-sum-exp: B*H_Q f32, padded]
//            [scores: B*H_Q*(splits * tokens per split) f32].
size_t scored_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                              int32_t head_size, const DecodePlan& plan) {
  const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads;
  return align256(decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_size, plan)) +
         align256(rows * sizeof(float)) +
         rows * plan.num_splits * static_cast<size_t>(plan.tokens_per_split) * sizeof(float);
}

pa_status launch_paged_decode_scored(DecodeArgs a, float* sums_out, const float* sums_in,
                                     int32_t sums_len, int32_t num_new, cudaStream_t stream) {
  if (a.num_seqs == 0) return PA_OK;
  if (a.num_kv_heads > 65535 || a.num_seqs > 65535) return PA_ERR_UNSUPPORTED;
  uint8_t* at = static_cast<uint8_t*>(a.workspace) +
                align256(decode_workspace_bytes(a.num_seqs, a.num_q_heads, a.num_kv_heads,
                                                a.head_size, a.plan));
  a.final_lse = reinterpret_cast<float*>(at);
  a.scores = reinterpret_cast<float*>(
      at + align256(static_cast<size_t>(a.num_seqs) * a.num_q_heads * sizeof(float)));
  const pa_status st = a.cache_dtype == PA_Q4 ? launch_paged_decode_q4(a, stream)
                                              : launch_paged_decode(a, stream);
  if (st != PA_OK) return st;
  const DecodeParams p = make_decode_params(a);
  const SumsParams w{sums_out, sums_in, sums_len, num_new};
  const int64_t tokens = p.score_len < sums_len ? p.score_len : sums_len;
  switch (a.num_q_heads / a.num_kv_heads) {
    case 1: return launch_add<1>(p, w, a.num_seqs, tokens, stream);
    case 2: return launch_add<2>(p, w, a.num_seqs, tokens, stream);
    case 4: return launch_add<4>(p, w, a.num_seqs, tokens, stream);
    case 8: return launch_add<8>(p, w, a.num_seqs, tokens, stream);
    case 16: return launch_add<16>(p, w, a.num_seqs, tokens, stream);
  }
  return PA_ERR_UNSUPPORTED;
}

}  // namespace pa_detail
