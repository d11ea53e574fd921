// rope_cache.cu -- rotate queries and keys by position and append keys and
// values to the paged cache, in one pass over the projections' output.
//
// A rotated pair (x, x') of a head at position p becomes
//     y = x cos - x' sin,  y' = x' cos + x sin     (cos, sin: row p of a table)
// in fp32 with every product and sum rounded (no fused multiply-add), so the
// result does not depend on how a compiler contracts it; then one rounding to
// the output's type (keys: after the optional division by k_scale).
//
// One warp takes a part of a token's heads: q heads, then k heads, then v heads.  A
// lane holds an "item": two chunks of eight elements of a head, which for the
// rotated elements are the two members of eight pairs (halves rot / 2 apart, or
// two neighbouring chunks of four pairs each), so no value crosses lanes.  The
// lanes of a head are a power of two (head 128: 8 lanes, four heads side by side),
// so a lane keeps the same item for every head and its 16 cosines and
// sines are loaded once per warp.
#include <type_traits>

#include "pa_internal.cuh"
#include "rope_cache.cuh"

namespace pa_detail {
namespace {

using namespace pa;

constexpr int kWarps = 8;  // per CTA
constexpr int kSteps = 4;  // head groups per warp: 8 loads of 16 bytes in flight per lane (16-bit source)

// Plain loads: q may be rotated in place, so the rows are not read-only.
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}
template <typename T>
__device__ __forceinline__ Vec8<T> load_chunk(const T* p) {
  Vec8<T> v;
  if constexpr (sizeof(T) == 4) {
    v.u[0] = ld16(p);
    v.u[1] = ld16(p + 4);
  } else {
    v.u = ld16(p);
  }
  return v;
}

__device__ __forceinline__ void rotate(float& x, float& y, float c, float s) {
  const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = u;
}

// eight cached values of D from fp32, through the division by a scale
template <typename D>
__device__ __forceinline__ Vec8<D> to_cache(float (&f)[8], bool scaled, const Divisor& d) {
  if (scaled) {
    if constexpr (std::is_same<D, e4m3>::value) {
      Vec8<float> v = from_f32<float>(f);
      div8_for_e4m3(v, f, d, fminf(1.7e38f * d.s, 3.0e38f));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = div_rn(f[e], d);
    }
  }
  return from_f32<D>(f);
}

template <typename S, typename D, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32) rope_and_cache_kernel(const RopeArgs a) {
  const int lane = threadIdx.x & 31;
  const uint32_t wid = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const uint32_t t32 = wid / a.parts;
  const int64_t t = t32;
  if (t >= a.num_tokens) return;
  const int part = static_cast<int>(wid - t32 * a.parts);

  const int64_t pos = __ldg(a.positions + t);
  if (pos < 0 || pos >= a.max_positions) return;
  int64_t slot = __ldg(a.slot_mapping + t);
  if (a.swa != nullptr && slot >= 0) slot = slot < a.swa_len ? __ldg(a.swa + slot) : -1;
  if (slot >= a.num_slots) slot = -1;

  // this lane's item: its two chunks (element offsets inside a head) and pairs
  const int item = lane & ((1 << a.log2_lanes) - 1);
  const int rot_items = a.rot_dim >> 4;
  const bool turned = item < rot_items;
  int c0, c1;
  if (turned && !kInterleaved) {
    c0 = 8 * item;
    c1 = c0 + (a.rot_dim >> 1);
  } else {
    c0 = 16 * item;  // (the tail starts at rot_dim, a multiple of 16)
    c1 = c0 + 8;
  }
  const bool has0 = c0 < a.head_size, has1 = c1 < a.head_size;
  float cs[8], sn[8];
  if (turned) {
    const float4* row = reinterpret_cast<const float4*>(a.cos_sin + pos * a.rot_dim + 8 * item);
    const float4* sow = row + (a.rot_dim >> 3);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = __ldg(row + i), y = __ldg(sow + i);
      cs[4 * i] = x.x, cs[4 * i + 1] = x.y, cs[4 * i + 2] = x.z, cs[4 * i + 3] = x.w;
      sn[4 * i] = y.x, sn[4 * i + 1] = y.y, sn[4 * i + 2] = y.z, sn[4 * i + 3] = y.w;
    }
  }

  const int heads_per_step = 32 >> a.log2_lanes;
  const int head0 = part * kSteps * heads_per_step + (lane >> a.log2_lanes);
  const int hq = a.num_q_heads, hk = a.num_kv_heads;
  const int64_t blk = slot < 0 ? 0
                      : (a.block_size & (a.block_size - 1)) == 0
                          ? slot >> (__ffs(a.block_size) - 1)
                          : slot / a.block_size;
  const int64_t dst0 =
      blk * a.block_stride + (slot - blk * a.block_size) * hk * static_cast<int64_t>(a.head_size);
  auto source = [&](int h) -> const S* {
    if (h < hq) return static_cast<const S*>(a.q) + t * a.q_stride + h * a.head_size;
    if (h < hq + hk)
      return static_cast<const S*>(a.key) + t * a.key_stride + (h - hq) * a.head_size;
    return static_cast<const S*>(a.value) + t * a.value_stride + (h - hq - hk) * a.head_size;
  };

  Vec8<S> x[kSteps], y[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int h = head0 + i * heads_per_step;
    if (h < a.all_heads && (h < hq || slot >= 0)) {
      const S* src = source(h);
      if (has0) x[i] = load_chunk(src + c0);
      if (has1) y[i] = load_chunk(src + c1);
    }
  }
  const bool scaled = a.k_scale != nullptr;
  const Divisor ks = make_divisor(scaled ? __ldg(a.k_scale) : 1.f);
  const Divisor vs = make_divisor(scaled ? __ldg(a.v_scale) : 1.f);
  const bool raw = std::is_same<S, D>::value && !scaled;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int h = head0 + i * heads_per_step;
    if (h >= a.all_heads || (h >= hq && slot < 0)) continue;
    const bool is_q = h < hq, is_v = h >= hq + hk;
    const bool turn = turned && !is_v;
    float f[8], g[8];
    to_f32(x[i], f);
    to_f32(y[i], g);
    if (turn) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (kInterleaved) {
          if (e < 4) {
            rotate(f[2 * e], f[2 * e + 1], cs[e], sn[e]);
          } else {
            rotate(g[2 * e - 8], g[2 * e - 7], cs[e], sn[e]);
          }
        } else {
          rotate(f[e], g[e], cs[e], sn[e]);
        }
      }
    }
    if (is_q) {
      S* dst = static_cast<S*>(a.q_out) + t * a.q_out_stride + h * a.head_size;
      if (has0) store8(dst + c0, turn ? from_f32<S>(f) : x[i]);
      if (has1) store8(dst + c1, turn ? from_f32<S>(g) : y[i]);
    } else {
      const int hh = is_v ? h - hq - hk : h - hq;
      D* dst = static_cast<D*>(is_v ? a.value_cache : a.key_cache) + dst0 + hh * a.head_size;
      if (raw && !turn) {  // the bits as they are
        if constexpr (std::is_same<S, D>::value) {
          if (has0) store8(dst + c0, x[i]);
          if (has1) store8(dst + c1, y[i]);
        }
      } else {
        const Divisor& d = is_v ? vs : ks;
        if (has0) store8(dst + c0, to_cache<D>(f, scaled, d));
        if (has1) store8(dst + c1, to_cache<D>(g, scaled, d));
      }
    }
  }
}

template <typename S, typename D>
pa_status launch_typed(const RopeArgs& a, bool interleaved, unsigned grid, cudaStream_t stream) {
  if (interleaved) {
    rope_and_cache_kernel<S, D, true><<<grid, kWarps * 32, 0, stream>>>(a);
  } else {
    rope_and_cache_kernel<S, D, false><<<grid, kWarps * 32, 0, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <typename S>
pa_status launch_src(const RopeArgs& a, pa_dtype dst, bool interleaved, unsigned grid,
                     cudaStream_t stream) {
  switch (dst) {
    case PA_BF16: return launch_typed<S, bf16>(a, interleaved, grid, stream);
    case PA_FP16: return launch_typed<S, f16>(a, interleaved, grid, stream);
    case PA_FP32: return launch_typed<S, float>(a, interleaved, grid, stream);
    case PA_FP8_E4M3: return launch_typed<S, e4m3>(a, interleaved, grid, stream);
    default: return PA_ERR_UNSUPPORTED;
  }
}

}  // namespace

pa_status launch_rope_and_cache(RopeArgs a, pa_dtype src, pa_dtype dst, bool interleaved,
                                cudaStream_t stream) {
  const int items = (a.rot_dim >> 4) + (((a.head_size - a.rot_dim) / 8 + 1) >> 1);
  a.log2_lanes = 0;
  while ((1 << a.log2_lanes) < items) ++a.log2_lanes;
  a.all_heads = a.num_q_heads + 2 * a.num_kv_heads;
  const int per_warp = kSteps * (32 >> a.log2_lanes);
  a.parts = static_cast<uint32_t>((a.all_heads + per_warp - 1) / per_warp);
  const int64_t warps = a.num_tokens * a.parts;
  if (warps > 0x7FFFFFFFll) return PA_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>((warps + kWarps - 1) / kWarps);
  switch (src) {
    case PA_BF16: return launch_src<bf16>(a, dst, interleaved, grid, stream);
    case PA_FP16: return launch_src<f16>(a, dst, interleaved, grid, stream);
    case PA_FP32: return launch_src<float>(a, dst, interleaved, grid, stream);
    default: return PA_ERR_UNSUPPORTED;
  }
}

}  // namespace pa_detail
