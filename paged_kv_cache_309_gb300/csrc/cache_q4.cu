// cache_q4.cu -- the 4-bit paged cache: rows quantised and scattered through
// slot_mapping, and gathered back.
//
// A kv head's row is cut into groups of 32 elements; with m = fp16(min x) and
// s = fp16(clamp((max x - m) / 15, 0, 1023)) an element's code is
// clamp(rne((x - m) / s), 0, 15) and stands for m + s * code.  The row is
// head_size / 2 code bytes followed by one (s, m) pair of fp16 per group.
//
// One lane holds a chunk of 8 consecutive elements (one 16-byte load of a
// 16-bit source, one 32-bit word of codes), four neighbouring lanes a group:
// its minimum and maximum are two shuffle steps.  A warp covers 128 chunks
// of a token's row (heads side by side, as they lie in source and cache).
#include "pa_internal.cuh"

namespace pa_detail {
namespace {

using namespace pa;

constexpr int kWarps = 8;
constexpr int kChunksPerLane = 4;
constexpr int kChunksPerWarp = 32 * kChunksPerLane;

// Byte offsets of chunk c of a row (head c / cph): its codes and its group's
// (s, m) pair.
struct RowPlace {
  int64_t code, meta;
};
__device__ __forceinline__ RowPlace row_place(int c, int cph) {
  const int head = c / cph, cc = c - head * cph;  // cph = head_size / 8 chunks per head
  const int64_t base = static_cast<int64_t>(head) * 5 * cph;
  return {base + 4 * cc, base + 4 * cph + 4 * (cc >> 2)};
}

// Quantises the lane's chunk together with the other three lanes of its
// group (all four lanes call with chunks of one group): returns the code word
// and the group's (s, m) as fp16 bits, s in the low half.
__device__ __forceinline__ uint32_t quantise(const float (&f)[8], uint32_t& meta) {
  float mn = f[0], mx = f[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    mn = min_nan(mn, f[e]);
    mx = max_nan(mx, f[e]);
  }
#pragma unroll
  for (int off = 1; off <= 2; off <<= 1) {
    mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, off));
    mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  }
  if (!(mn >= -3.4028235e38f && mx <= 3.4028235e38f)) {  // a NaN or an infinity
    meta = 0x7FFF7FFFu;
    return 0u;
  }
  const __half mh = __float2half_rn(fminf(fmaxf(mn, -65504.f), 65504.f));
  const float m = __half2float(mh);
  const __half sh = __float2half_rn(fminf(fmaxf(__fdiv_rn(mx - m, 15.f), 0.f), 1023.f));
  const float s = __half2float(sh);
  meta = static_cast<uint32_t>(__half_as_ushort(sh)) |
         (static_cast<uint32_t>(__half_as_ushort(mh)) << 16);
  uint32_t word = 0u;
  if (s > 0.f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = fminf(fmaxf(rintf(__fdiv_rn(f[e] - m, s)), 0.f), 15.f);
      word |= static_cast<uint32_t>(y) << (4 * e);
    }
  }
  return word;
}

template <typename S>
__global__ void __launch_bounds__(kWarps * 32) reshape_and_cache_q4_kernel(Q4CacheArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t t = wid / a.groups;
  const int grp = static_cast<int>(wid - t * a.groups);
  if (t >= a.num_tokens) return;
  int64_t s = __ldg(a.slot_mapping + t);  // the same slot in every lane
  if (s < 0) return;
  if (a.swa != nullptr) {
    if (s >= a.swa_len) return;
    s = __ldg(a.swa + s);
    if (s < 0) return;
  }
  if (s >= a.num_slots) return;
  const int64_t blk = s / a.block_size;
  const int64_t dst0 = blk * a.block_stride + (s - blk * a.block_size) * a.row_chunks * 5;
#pragma unroll
  for (int tensor = 0; tensor < 2; ++tensor) {
    const S* src = static_cast<const S*>(tensor ? a.value : a.key) +
                   t * (tensor ? a.value_stride : a.key_stride);
    uint8_t* dst = static_cast<uint8_t*>(tensor ? a.value_cache : a.key_cache) + dst0;
    if (tensor && a.value == nullptr) break;
#pragma unroll
    for (int i = 0; i < kChunksPerLane; ++i) {
      const int c = grp * kChunksPerWarp + 32 * i + lane;
      if (c - lane >= a.row_chunks) break;  // the whole warp
      float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (c < a.row_chunks) to_f32(load8(src + 8 * c), f);
      uint32_t meta;
      const uint32_t word = quantise(f, meta);
      if (c < a.row_chunks) {
        const RowPlace p = row_place(c, a.chunks_per_head);
        *reinterpret_cast<uint32_t*>(dst + p.code) = word;
        if ((c & 3) == 0) *reinterpret_cast<uint32_t*>(dst + p.meta) = meta;
      }
    }
  }
}

template <typename D>
__global__ void __launch_bounds__(kWarps * 32) gather_cache_q4_kernel(Q4CacheArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t t = wid / a.groups;
  const int grp = static_cast<int>(wid - t * a.groups);
  if (t >= a.num_tokens) return;
  const int64_t s = __ldg(a.slot_mapping + t);
  if (s < 0 || s >= a.num_slots) return;
  const int64_t blk = s / a.block_size;
  const int64_t src0 = blk * a.block_stride + (s - blk * a.block_size) * a.row_chunks * 5;
#pragma unroll
  for (int tensor = 0; tensor < 2; ++tensor) {
    if (tensor && a.value == nullptr) break;
    const uint8_t* src = static_cast<const uint8_t*>(tensor ? a.value_cache : a.key_cache) + src0;
    D* dst = static_cast<D*>(const_cast<void*>(tensor ? a.value : a.key)) +
             t * (tensor ? a.value_stride : a.key_stride);
#pragma unroll
    for (int i = 0; i < kChunksPerLane; ++i) {
      const int c = grp * kChunksPerWarp + 32 * i + lane;
      if (c >= a.row_chunks) break;
      const RowPlace p = row_place(c, a.chunks_per_head);
      const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(src + p.code));
      const uint32_t meta = __ldg(reinterpret_cast<const uint32_t*>(src + p.meta));
      const float sc = __half2float(__ushort_as_half(static_cast<uint16_t>(meta & 0xFFFFu)));
      const float m = __half2float(__ushort_as_half(static_cast<uint16_t>(meta >> 16)));
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f[e] = __fmaf_rn(static_cast<float>((word >> (4 * e)) & 15u), sc, m);
      store8(dst + 8 * c, from_f32<D>(f));
    }
  }
}

pa_status grid_of(Q4CacheArgs& a, unsigned* grid) {
  a.groups = (a.row_chunks + kChunksPerWarp - 1) / kChunksPerWarp;
  const int64_t blocks = (a.num_tokens * a.groups + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFFll) return PA_ERR_UNSUPPORTED;
  *grid = static_cast<unsigned>(blocks);
  return PA_OK;
}

}  // namespace

pa_status launch_reshape_and_cache_q4(Q4CacheArgs a, pa_dtype src, cudaStream_t stream) {
  unsigned grid = 0;
  const pa_status st = grid_of(a, &grid);
  if (st != PA_OK) return st;
  switch (src) {
    case PA_BF16: reshape_and_cache_q4_kernel<bf16><<<grid, kWarps * 32, 0, stream>>>(a); break;
    case PA_FP16: reshape_and_cache_q4_kernel<f16><<<grid, kWarps * 32, 0, stream>>>(a); break;
    case PA_FP32: reshape_and_cache_q4_kernel<float><<<grid, kWarps * 32, 0, stream>>>(a); break;
    default: return PA_ERR_UNSUPPORTED;
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status launch_gather_cache_q4(Q4CacheArgs a, pa_dtype dst, cudaStream_t stream) {
  unsigned grid = 0;
  const pa_status st = grid_of(a, &grid);
  if (st != PA_OK) return st;
  switch (dst) {
    case PA_BF16: gather_cache_q4_kernel<bf16><<<grid, kWarps * 32, 0, stream>>>(a); break;
    case PA_FP16: gather_cache_q4_kernel<f16><<<grid, kWarps * 32, 0, stream>>>(a); break;
    case PA_FP32: gather_cache_q4_kernel<float><<<grid, kWarps * 32, 0, stream>>>(a); break;
    default: return PA_ERR_UNSUPPORTED;
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa_detail
