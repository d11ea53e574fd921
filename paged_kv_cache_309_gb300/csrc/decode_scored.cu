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
#include "pa_internal.cuh"

namespace pa_detail {

using namespace pa;
using namespace decode;

namespace {

constexpr int kSumThreads = 256;
constexpr int kSumLoads = 8;  // 16-byte score loads in flight per thread

struct SumsParams {
  float* out;
  const float* in;
  int32_t sums_len;
  int32_t num_new;
  bool wide;  // rows of sums on 16-byte boundaries
};

// A 16-byte load holds 4 / G tokens' scores (G <= 4) or a quarter to a half of
// one token's (G = 16, 8).  A CTA takes kSumThreads * kSumLoads loads' worth of
// tokens of one (sequence, kv head): one token per thread, a CTA for every
// 256 tokens, spent its time waiting for the lengths and sums of logs
// (B = 8, 32K-128K, G = 4: 126 us; so: 27-29 us from DRAM, 105 MB read).
template <int G>
__global__ void __launch_bounds__(kSumThreads) add_weights_kernel(const DecodeParams p,
                                                                  const SumsParams w) {
  constexpr int kV = G < 4 ? 4 / G : 1;   // tokens per step of a thread
  constexpr int kL = G < 4 ? 1 : G / 4;   // loads per step
  constexpr int kSteps = kSumLoads / kL;
  const int g = blockIdx.y, b = blockIdx.z;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores and sums of logs are there
  // A wait that ran out in the launches before left tokens without a score (their
  // places hold an earlier call's): the sums stay as they were, all of them, so that
  // the call can be repeated.  The caller clears the word.
  const unsigned err = __ldcg(p.err);
  bool clipped;
  const int L = effective_len(p, b, &clipped);
  if (err & PA_DEVERR_WAIT_TIMEOUT) return;
  const int end = min(L, w.sums_len);
  const int64_t row = static_cast<int64_t>(b) * p.num_kv_heads + g;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kSumThreads * kSteps * kV);
  if (first >= end) return;
  const float* scores = p.scores + row * p.score_len * G;
  const int t0 = static_cast<int>(first) + threadIdx.x * kV;
  float4 v[kSteps][kL];
  float old[kSteps][kV];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int t = t0 + i * kSumThreads * kV;
    if (t < end) {
#pragma unroll
      for (int k = 0; k < kL; ++k)  // (rows of scores are 64 tokens long at least)
        v[i][k] = __ldcs(reinterpret_cast<const float4*>(scores + static_cast<int64_t>(t) * G) + k);
      const float* in = w.in + row * w.sums_len + t;
      if (kV > 1 && w.wide && t + kV <= end) {
        if constexpr (kV == 4) {
          const float4 x = *reinterpret_cast<const float4*>(in);
          old[i][0] = x.x;
          old[i][1] = x.y;
          old[i][2] = x.z;
          old[i][3] = x.w;
        } else if constexpr (kV == 2) {
          const float2 x = *reinterpret_cast<const float2*>(in);
          old[i][0] = x.x;
          old[i][1] = x.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j) old[i][j] = t + j < end ? in[j] : 0.f;
      }
    }
  }
  float lse[G];
#pragma unroll
  for (int h = 0; h < G; ++h)
    lse[h] = __ldcg(p.final_lse + static_cast<int64_t>(b) * p.num_q_heads + g * G + h);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int t = t0 + i * kSumThreads * kV;
    if (t >= end) break;
    float s[4 * kL];
#pragma unroll
    for (int k = 0; k < kL; ++k) {
      s[4 * k] = v[i][k].x;
      s[4 * k + 1] = v[i][k].y;
      s[4 * k + 2] = v[i][k].z;
      s[4 * k + 3] = v[i][k].w;
    }
    float sum[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      float weight = 0.f;
#pragma unroll
      for (int h = 0; h < G; ++h)  // (a sum of logs of -inf: no token is there)
        weight += lse[h] == -INFINITY ? 0.f : exp2f(s[j * G + h] - lse[h]);
      sum[j] = (t + j >= L - w.num_new ? 0.f : old[i][j]) + weight;
    }
    float* out = w.out + row * w.sums_len + t;
    if (kV > 1 && w.wide && t + kV <= end) {
      if constexpr (kV == 4)
        *reinterpret_cast<float4*>(out) = make_float4(sum[0], sum[1], sum[2], sum[3]);
      else if constexpr (kV == 2)
        *reinterpret_cast<float2*>(out) = make_float2(sum[0], sum[1]);
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (t + j < end) out[j] = sum[j];
    }
  }
}

template <int G>
pa_status launch_add(const DecodeParams& p, const SumsParams& w, int32_t num_seqs, int64_t tokens,
                     cudaStream_t stream) {
  constexpr int64_t kPerCta = static_cast<int64_t>(kSumThreads) * kSumLoads * 4 / G;
  const dim3 grid(static_cast<unsigned>((tokens + kPerCta - 1) / kPerCta),
                  static_cast<unsigned>(p.num_kv_heads), static_cast<unsigned>(num_seqs));
  return launch_dependent(add_weights_kernel<G>, grid, kSumThreads, stream, p, w);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// The decode workspace, with room for its split counters even where the plan has
// one range and no counters: they have to be zero when a later call with a
// longer max_context_len (or a decode call with another plan) finds them.
size_t decode_part_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                         int32_t head_size, const DecodePlan& plan) {
  const size_t bytes =
      decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_size, plan);
  const size_t counters =
      kWorkspaceHeader + static_cast<size_t>(num_seqs) * num_kv_heads * sizeof(unsigned);
  return align256(bytes > counters ? bytes : counters);
}

}  // namespace

// Workspace: [decode workspace, padded] [log2-sum-exp: B*H_Q f32, padded]
//            [scores: B*H_Q*(splits * tokens per split) f32].
size_t scored_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                              int32_t head_size, const DecodePlan& plan) {
  const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads;
  return decode_part_bytes(num_seqs, num_q_heads, num_kv_heads, head_size, plan) +
         align256(rows * sizeof(float)) +
         rows * plan.num_splits * static_cast<size_t>(plan.tokens_per_split) * sizeof(float);
}

pa_status launch_paged_decode_scored(DecodeArgs a, float* sums_out, const float* sums_in,
                                     int32_t sums_len, int32_t num_new, cudaStream_t stream) {
  if (a.num_seqs == 0) return PA_OK;
  if (a.num_kv_heads > 65535 || a.num_seqs > 65535) return PA_ERR_UNSUPPORTED;
  uint8_t* at = static_cast<uint8_t*>(a.workspace) +
                decode_part_bytes(a.num_seqs, a.num_q_heads, a.num_kv_heads, a.head_size, a.plan);
  a.final_lse = reinterpret_cast<float*>(at);
  a.scores = reinterpret_cast<float*>(
      at + align256(static_cast<size_t>(a.num_seqs) * a.num_q_heads * sizeof(float)));
  const pa_status st = a.cache_dtype == PA_Q4 ? launch_paged_decode_q4(a, stream)
                                              : launch_paged_decode(a, stream);
  if (st != PA_OK) return st;
  const DecodeParams p = make_decode_params(a);
  const bool wide = sums_len % 4 == 0 && ((reinterpret_cast<uintptr_t>(sums_out) |
                                           reinterpret_cast<uintptr_t>(sums_in)) & 15u) == 0u;
  const SumsParams w{sums_out, sums_in, sums_len, num_new, wide};
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
