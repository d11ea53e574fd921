// rope_cache.cu -- rotate queries and keys by position and append keys and
// values to the paged cache, in one pass over the projections' output.
//
// A rotated pair (x, x') of a head at position p becomes
//     y = x cos - x' sin,  y' = x' cos + x sin     (cos, sin: row p of a table)
// in fp32 with every product and sum rounded (no fused multiply-add), so the
// result does not depend on how a compiler contracts it; then one rounding to
// the output's type (keys: after the optional division by k_scale).
//
// One warp takes two steps of a token: a step is a group of heads side by side, all
// of q, of k or of v.  A lane holds an "item": two chunks of eight elements of a
// head, which for the rotated elements are the two members of eight pairs (halves
// rot / 2 apart, or two neighbouring chunks of four pairs each), so no value
// crosses lanes.  The lanes of a head are a power of two (head 128: 8 lanes, four
// heads), so a lane keeps the same item for every head and its 16 cosines and
// sines are loaded once per warp.
//
// Bounds and what was measured (GPU time, perf/gpu_times.py):
//  * a long batch moves bytes: 32768 tokens, 32 q and 8 kv heads of 128, bf16, take
//    130 us for 823 MB, 6.3 TB/s.  A warp that walked over all steps of its token
//    took 140 us, one that waited for position and slot before its rows' loads 185;
//  * a short one is a chain of two loads and a store (position, table row, row
//    out): 64 tokens, 1.9 us (3.5 us with a warp per token).  The rows
//    are therefore loaded before the position and slot are there;
//  * 5001 tokens of 10 / 5 heads of 96 divided into e4m3 take 12.9 us (20.2 before pairs of sums
//    and the steps of one kind): issue slots are 64 % used, by warps of which half the lanes' places
//    hold an item (6 items in 8 lanes, heads of a kind in groups of four: 120 items a token in
//    256 places).
#include <type_traits>

#include "pa_internal.cuh"
#include "rope_cache.cuh"

namespace pa_detail {
namespace {

using namespace pa;

constexpr int kWarps = 4;  // per CTA
constexpr int kCtasPerSm = 8;
constexpr int kSteps = 2;  // per warp: four loads of 16 bytes in flight per lane (16-bit source)

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

// Eight fp32 values as four pairs: a paired sum rounds each half as the scalar one
// does, in half the issued instructions.
struct F2x4 {
  float2 v[4];
};
__device__ __forceinline__ float2 add2_rn(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
template <typename T>
__device__ __forceinline__ F2x4 widen(const Vec8<T>& x) {
  F2x4 r;
  float f[8];
  to_f32(x, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = make_float2(f[2 * i], f[2 * i + 1]);
  return r;
}
template <typename T>
__device__ __forceinline__ Vec8<T> narrow(const F2x4& x) {
  if constexpr (std::is_same<T, bf16>::value) {
    return {make_uint4(pack_bf16x2(x.v[0].x, x.v[0].y), pack_bf16x2(x.v[1].x, x.v[1].y),
                       pack_bf16x2(x.v[2].x, x.v[2].y), pack_bf16x2(x.v[3].x, x.v[3].y))};
  } else if constexpr (std::is_same<T, f16>::value) {
    return {make_uint4(pack_f16x2(x.v[0].x, x.v[0].y), pack_f16x2(x.v[1].x, x.v[1].y),
                       pack_f16x2(x.v[2].x, x.v[2].y), pack_f16x2(x.v[3].x, x.v[3].y))};
  } else {
    const float f[8] = {x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y,
                        x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y};
    return from_f32<T>(f);
  }
}
// eight cached values of D, through the division by a scale
template <typename D>
__device__ __forceinline__ Vec8<D> divided(const F2x4& x, const Divisor& d) {
  float f[8] = {x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y, x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y};
  if constexpr (std::is_same<D, e4m3>::value) {
    const Vec8<float> v = from_f32<float>(f);
    div8_for_e4m3(v, f, d, fminf(1.7e38f * d.s, 3.0e38f));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = div_rn(f[e], d);
  }
  return from_f32<D>(f);
}

// Rounded products, one by one: a paired mul.rn was joined with the paired add.rn after it (one
// element in 30 thousand differed).  A paired instruction takes two issue cycles of the
// pipe, so nothing is lost in the pipe.
__device__ __forceinline__ float2 product(float2 a, float2 b) {
  return make_float2(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y));
}
// Pairs (x, y), the members in separate registers: x c + -(y s) is the rounded difference.
__device__ __forceinline__ void rotate_apart(float2& x, float2& y, float2 c, float2 s) {
  const float2 u = add2_rn(product(x, c), product(make_float2(-y.x, -y.y), s));
  y = add2_rn(product(y, c), product(x, s));
  x = u;
}
// One pair (p.x, p.y): (p.x c + -p.y s, p.y c + p.x s)
__device__ __forceinline__ float2 rotate_one(float2 p, float c, float s) {
  return add2_rn(product(p, make_float2(c, c)), product(make_float2(-p.y, p.x), make_float2(s, s)));
}

template <typename S, typename D, bool kInterleaved, bool kScaled>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) rope_and_cache_kernel(const RopeArgs a) {
  const int lane = threadIdx.x & 31;
  const uint32_t wid = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const uint32_t t32 = wid / a.parts;
  const int64_t t = t32;
  if (t >= a.num_tokens) return;
  const int step0 = static_cast<int>(wid - t32 * a.parts) * kSteps;

  // position and slot together; the rows' loads do not wait for them (a padded token's rows are
  // read in vain), but behind a second slot table, where most tokens may have no slot
  const int64_t pos = __ldg(a.positions + t);
  int64_t slot = __ldg(a.slot_mapping + t);
  if (a.swa != nullptr && slot >= 0) slot = slot < a.swa_len ? __ldg(a.swa + slot) : -1;

  // this lane's item: its two chunks (element offsets inside a head) and pairs
  const int item = lane & ((1 << a.log2_lanes) - 1);
  const bool turned = item < a.rot_dim >> 4;
  int c0, c1;
  if (turned && !kInterleaved) {
    c0 = 8 * item;
    c1 = c0 + (a.rot_dim >> 1);
  } else {
    c0 = 16 * item;  // (the tail starts at rot_dim, a multiple of 16)
    c1 = c0 + 8;
  }
  const bool has0 = c0 < a.head_size, has1 = c1 < a.head_size;
  const int log2_heads = 5 - a.log2_lanes;  // heads side by side
  // a step is such a group of heads of q (the first ones), of k or of v: kind 0, 1, 2
  auto kind_of = [&](int step) {
    return step < a.q_steps ? 0 : step < a.q_steps + a.kv_steps ? 1 : 2;
  };
  auto head_of = [&](int step, int kind) {
    const int first = kind == 0 ? 0 : kind == 1 ? a.q_steps : a.q_steps + a.kv_steps;
    return ((step - first) << log2_heads) + (lane >> a.log2_lanes);
  };

  Vec8<S> x[kSteps], y[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int kind = kind_of(step0 + i), h = head_of(step0 + i, kind);
    if (h < (kind == 0 ? a.num_q_heads : a.num_kv_heads) &&
        (kind == 0 || a.swa == nullptr || slot >= 0)) {
      const S* src = kind == 0   ? static_cast<const S*>(a.q) + t * a.q_stride
                     : kind == 1 ? static_cast<const S*>(a.key) + t * a.key_stride
                                 : static_cast<const S*>(a.value) + t * a.value_stride;
      src += h * a.head_size;
      if (has0) x[i] = load_chunk(src + c0);
      if (has1) y[i] = load_chunk(src + c1);
    }
  }
  if (pos < 0 || pos >= a.max_positions) return;
  if (slot >= a.num_slots) slot = -1;
  float2 cs[4], sn[4];
  if (turned && kind_of(step0) < 2) {
    const float4* row = reinterpret_cast<const float4*>(a.cos_sin + pos * a.rot_dim + 8 * item);
    const float4* sow = row + (a.rot_dim >> 3);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 c = __ldg(row + i), s = __ldg(sow + i);
      cs[2 * i] = make_float2(c.x, c.y), cs[2 * i + 1] = make_float2(c.z, c.w);
      sn[2 * i] = make_float2(s.x, s.y), sn[2 * i + 1] = make_float2(s.z, s.w);
    }
  }
  const int64_t blk = slot < 0 ? 0
                      : (a.block_size & (a.block_size - 1)) == 0
                          ? slot >> (__ffs(a.block_size) - 1)
                          : slot / a.block_size;
  const int64_t dst0 = blk * a.block_stride + (slot - blk * a.block_size) * a.num_kv_heads *
                                                  static_cast<int64_t>(a.head_size);
  constexpr bool kRaw = std::is_same<S, D>::value && !kScaled;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int kind = kind_of(step0 + i), h = head_of(step0 + i, kind);
    if (h >= (kind == 0 ? a.num_q_heads : a.num_kv_heads) || (kind != 0 && slot < 0)) continue;
    F2x4 f, g;
    const bool turn = turned && kind != 2;
    if (turn) {
      f = widen(x[i]);
      g = widen(y[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (kInterleaved) {
          f.v[e] = rotate_one(f.v[e], (e & 1) ? cs[e >> 1].y : cs[e >> 1].x,
                              (e & 1) ? sn[e >> 1].y : sn[e >> 1].x);
          g.v[e] = rotate_one(g.v[e], (e & 1) ? cs[2 + (e >> 1)].y : cs[2 + (e >> 1)].x,
                              (e & 1) ? sn[2 + (e >> 1)].y : sn[2 + (e >> 1)].x);
        } else {
          rotate_apart(f.v[e], g.v[e], cs[e], sn[e]);
        }
      }
    }
    // what is not turned keeps its bits where the type stays
    if (kind == 0 || kRaw) {
      if (turn) {
        x[i] = narrow<S>(f);
        y[i] = narrow<S>(g);
      }
      S* dst = kind == 0 ? static_cast<S*>(a.q_out) + t * a.q_out_stride
                         : static_cast<S*>(kind == 1 ? a.key_cache : a.value_cache) + dst0;
      dst += h * a.head_size;
      if (has0) store8(dst + c0, x[i]);
      if (has1) store8(dst + c1, y[i]);
    } else {
      if (!turn) {
        f = widen(x[i]);
        g = widen(y[i]);
      }
      D* dst = static_cast<D*>(kind == 1 ? a.key_cache : a.value_cache) + dst0 + h * a.head_size;
      if constexpr (kScaled) {
        const Divisor d = make_divisor(__ldg(kind == 1 ? a.k_scale : a.v_scale));
        if (has0) store8(dst + c0, divided<D>(f, d));
        if (has1) store8(dst + c1, divided<D>(g, d));
      } else {
        if (has0) store8(dst + c0, narrow<D>(f));
        if (has1) store8(dst + c1, narrow<D>(g));
      }
    }
  }
}

template <typename S, typename D>
pa_status launch_typed(const RopeArgs& a, bool interleaved, unsigned grid, cudaStream_t stream) {
  const bool scaled = a.k_scale != nullptr;
  const auto kernel = interleaved ? (scaled ? rope_and_cache_kernel<S, D, true, true>
                                            : rope_and_cache_kernel<S, D, true, false>)
                                  : (scaled ? rope_and_cache_kernel<S, D, false, true>
                                            : rope_and_cache_kernel<S, D, false, false>);
  kernel<<<grid, kWarps * 32, 0, stream>>>(a);
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
  const int heads = 32 >> a.log2_lanes;
  a.q_steps = (a.num_q_heads + heads - 1) / heads;
  a.kv_steps = (a.num_kv_heads + heads - 1) / heads;
  a.parts = static_cast<uint32_t>((a.q_steps + 2 * a.kv_steps + kSteps - 1) / kSteps);
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
