// cache_q4.cu -- the 4-bit paged cache: rows quantised and scattered through
// slot_mapping, and gathered back.
//
// A kv head's row is cut into groups of 32 elements; with m = fp16(min x) and
// s = fp16(clamp((max x - m) / 15, 0, 1023)) an element's code is
// clamp(rne((x - m) / s), 0, 15) and stands for m + s * code.  The row is
// head_size / 2 code bytes followed by one (s, m) pair of fp16 per group.
//
// One lane holds a unit of 16 consecutive elements, half a group (32 bytes of
// a 16-bit source, 8 bytes of codes): with 8 elements per lane the per-group
// arithmetic (minimum and maximum across lanes, scale, its reciprocal) ran in
// four lanes and cost more than the elements; with 16 one shuffle joins the
// halves and the kernel is bound by its issue slots beside HBM (32K tokens x 8
// heads of 128 from bf16: 31 us, 205 instructions for 512 elements, 0.77 of
// the cycles issuing; the gather back to bf16 30.5 us).  A warp takes 32 units of a token's K row and of its V row, all loads first.
//
// The quotient (x - m) / s must be the IEEE one, for the codes are defined by
// it.  With r within 2^-23 of 1 / s (relative), y0 = RN(t r) and one
// correction y = RN(y0 + (t - s y0) r), where the residual is exact (s has 11
// bits), y is RN of t / s (1 + d), |d| < 2^-45.  It rounds like t / s unless a
// midpoint between two floats lies between them, and such a midpoint times s is either
// t exactly (impossible: it has more than t's 24 bits) or at least 2^-36 s away from it.
#include "pa_internal.cuh"

namespace pa_detail {
namespace {

using namespace pa;

constexpr int kWarps = 8;        // per CTA of the write
constexpr int kGatherWarps = 4;  // of the gather

__device__ __forceinline__ float2 add2_rn(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// ------------------------------------------------- a unit of 16 elements --
template <typename S>
struct Unit {
  Vec8<S> v[2];
};
// 32 bytes in one access where the address allows it: two accesses of 16
// bytes each touch every 32-byte sector twice.
struct U8 {
  uint4 a, b;
};
__device__ __forceinline__ U8 ld32(const void* p, bool whole) {
  U8 v;
  if (whole) {
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v.a.x), "=r"(v.a.y), "=r"(v.a.z), "=r"(v.a.w), "=r"(v.b.x), "=r"(v.b.y),
                   "=r"(v.b.z), "=r"(v.b.w)
                 : "l"(p));
  } else {
    v.a = __ldg(static_cast<const uint4*>(p));
    v.b = __ldg(static_cast<const uint4*>(p) + 1);
  }
  return v;
}
__device__ __forceinline__ void st32(void* p, const U8& v, bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v.a.x),
                 "r"(v.a.y), "r"(v.a.z), "r"(v.a.w), "r"(v.b.x), "r"(v.b.y), "r"(v.b.z),
                 "r"(v.b.w)
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = v.a;
    static_cast<uint4*>(p)[1] = v.b;
  }
}
template <typename S>
__device__ __forceinline__ Unit<S> load_unit(const S* p, bool whole) {
  Unit<S> u;
  if constexpr (sizeof(S) == 2) {
    const U8 x = ld32(p, whole);
    u.v[0].u = x.a;
    u.v[1].u = x.b;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const U8 x = ld32(p + 8 * i, whole);
      u.v[i].u[0] = x.a;
      u.v[i].u[1] = x.b;
    }
  }
  return u;
}
template <typename S>
__device__ __forceinline__ void store_unit(S* p, const Unit<S>& u, bool whole) {
  if constexpr (sizeof(S) == 2) {
    st32(p, U8{u.v[0].u, u.v[1].u}, whole);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) st32(p + 8 * i, U8{u.v[i].u[0], u.v[i].u[1]}, whole);
  }
}

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, bf16) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, f16) {
  uint32_t d;
  asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, bf16) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, f16) {
  uint32_t d;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float2 widen(uint32_t w, bf16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 widen(uint32_t w, f16) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Minimum and maximum (NaN if any element is) of the group this lane and its
// neighbour (lane ^ 1) hold.
template <typename S>
__device__ __forceinline__ float2 group_min_max(const Unit<S>& u) {
  if constexpr (sizeof(S) == 2) {
    const uint32_t w[8] = {u.v[0].u.x, u.v[0].u.y, u.v[0].u.z, u.v[0].u.w,
                           u.v[1].u.x, u.v[1].u.y, u.v[1].u.z, u.v[1].u.w};
    uint32_t mn = w[0], mx = w[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      mn = min2(mn, w[i], S{});
      mx = max2(mx, w[i], S{});
    }
    // (minimum, -maximum) of the even and of the odd elements, joined as pairs
    const uint32_t even = __byte_perm(mn, mx, 0x5410u) ^ 0x80000000u;
    const uint32_t odd = __byte_perm(mn, mx, 0x7632u) ^ 0x80000000u;
    uint32_t p = min2(even, odd, S{});
    p = min2(p, __shfl_xor_sync(0xffffffffu, p, 1), S{});
    const float2 f = widen(p, S{});
    return make_float2(f.x, -f.y);
  } else {
    float f[8], mn, mx;
    to_f32(u.v[0], f);
    mn = mx = f[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      mn = min_nan(mn, f[e]);
      mx = max_nan(mx, f[e]);
    }
    to_f32(u.v[1], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mn = min_nan(mn, f[e]);
      mx = max_nan(mx, f[e]);
    }
    mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
    mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    return make_float2(mn, mx);
  }
}

// The codes of a unit.  kClamp: some lie outside [0, 15] before the clamp.
template <bool kClamp, typename S>
__device__ __forceinline__ uint2 codes_of(const Unit<S>& u, float m, float s, float r) {
  const float2 nm = make_float2(-m, -m), r2 = make_float2(r, r), ns = make_float2(-s, -s);
  // 1.5 * 2^23: the sum's last bit counts 1 (also just below 0), rounded to even
  const float2 magic = make_float2(12582912.f, 12582912.f);
  uint2 word;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float f[8];
    to_f32(u.v[half], f);
    uint32_t w = 0u;
#pragma unroll
    for (int e = 6; e >= 0; e -= 2) {
      const float2 t = add2_rn(make_float2(f[e], f[e + 1]), nm);
      float2 y = mul2_rn(t, r2);
      y = fma2_rn(fma2_rn(ns, y, t), r2, y);
      if (kClamp) {
        y.x = fminf(fmaxf(y.x, 0.f), 15.f);
        y.y = fminf(fmaxf(y.y, 0.f), 15.f);
      }
      const float2 c = add2_rn(y, magic);
      // c is 0x4B400000 + code; what those constants add up to goes below
      w = (w << 4) + __float_as_uint(c.y);
      w = (w << 4) + __float_as_uint(c.x);
    }
    // shifted by 0, 4 and 8; the rest fell out of the word
    (half ? word.y : word.x) = w - (0x4B400000u + 0xB4000000u + 0x40000000u);
  }
  return word;
}

// Quantises the lane's unit together with its neighbour's: two code words and
// the group's (s, m) as fp16 bits, s in the low half.
template <typename S>
__device__ __forceinline__ uint2 quantise(const Unit<S>& u, uint32_t& meta) {
  const float2 mm = group_min_max(u);
  const float mn = mm.x, mx = mm.y;
  const bool fine = mn >= -3.4028235e38f && mx <= 3.4028235e38f;  // no NaN, no infinity
  const __half mh = __float2half_rn(fminf(fmaxf(mn, -65504.f), 65504.f));
  const float m = __half2float(mh);
  // span / 15: RN(1 / 15) and one correction, as for the codes (15 has 4 bits)
  const float span = mx - m;
  float q = __fmul_rn(span, 0x1.111112p-4f);
  q = __fmaf_rn(__fmaf_rn(-15.f, q, span), 0x1.111112p-4f, q);
  const __half sh = __float2half_rn(fminf(fmaxf(q, 0.f), 1023.f));
  const float s = __half2float(sh);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  r = s > 0.f ? r : 0.f;  // s = 0: every code 0
  // codes outside [0, 15] before the clamp: the minimum's rounding, a
  // subnormal or saturated scale, values that are not finite
  const bool clamp = !(span * r <= 15.49f && (mn - m) * r >= -0.49f);
  uint2 word;
  if (__any_sync(0xffffffffu, clamp)) {
    word = codes_of<true>(u, m, s, r);
    meta = 0x7FFF7FFFu;
    if (!fine) return make_uint2(0u, 0u);
  } else {
    word = codes_of<false>(u, m, s, r);
  }
  meta = static_cast<uint32_t>(__half_as_ushort(sh)) |
         (static_cast<uint32_t>(__half_as_ushort(mh)) << 16);
  return word;
}

// Byte offsets of unit c of a row (head c / uph): its codes and its group's
// (s, m) pair.
struct RowPlace {
  int64_t code, meta;
};
__device__ __forceinline__ RowPlace row_place(int c, int uph) {
  // uph = head_size / 16 units per head, a power of two for most heads
  const int head = (uph & (uph - 1)) == 0 ? c >> (31 - __clz(uph)) : c / uph;
  const int cc = c - head * uph;
  const int64_t base = static_cast<int64_t>(head) * 10 * uph;
  return {base + 8 * cc, base + 8 * uph + 4 * (cc >> 1)};
}

// The slot of token t through the optional second-stage table, -1: skip.
__device__ __forceinline__ int64_t slot_of(const Q4CacheArgs& a, int64_t t) {
  int64_t s = __ldg(a.slot_mapping + t);
  if (s >= 0 && a.swa != nullptr) s = s < a.swa_len ? __ldg(a.swa + s) : -1;
  return s < a.num_slots ? s : -1;
}
// Byte offset of a slot's row in the cache.
__device__ __forceinline__ int64_t row_of(const Q4CacheArgs& a, int64_t s) {
  const int64_t blk = (a.block_size & (a.block_size - 1)) == 0
                          ? s >> (__ffs(a.block_size) - 1)
                          : s / a.block_size;
  return blk * a.block_stride + (s - blk * a.block_size) * a.row_units * 10;
}

template <typename S>
__global__ void __launch_bounds__(kWarps * 32, sizeof(S) == 2 ? 8 : 4) reshape_and_cache_q4_kernel(Q4CacheArgs a) {
  const int lane = threadIdx.x & 31;
  // a CTA takes 32 units of kWarps tokens; the row's groups of 32 are the grid's y axis
  // (a warp's number divided by the groups took a sixth of the instructions)
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= a.num_tokens) return;
  const int c = static_cast<int>(blockIdx.y) * 32 + lane;
  const int64_t s = slot_of(a, t);  // the same slot in every lane
  if (s < 0) return;
  const bool mine = c < a.row_units, has_v = a.value != nullptr;
  Unit<S> k{}, v{};
  if (mine) {
    k = load_unit(static_cast<const S*>(a.key) + t * a.key_stride + 16 * c, a.whole32);
    if (has_v) v = load_unit(static_cast<const S*>(a.value) + t * a.value_stride + 16 * c, a.whole32);
  }
  const RowPlace p = row_place(c, a.units_per_head);
  const int64_t dst = row_of(a, s);
#pragma unroll
  for (int tensor = 0; tensor < 2; ++tensor) {
    if (tensor && !has_v) break;
    uint32_t meta;
    const uint2 word = quantise(tensor ? v : k, meta);
    if (mine) {
      uint8_t* to = static_cast<uint8_t*>(tensor ? a.value_cache : a.key_cache) + dst;
      // (a row starts at a multiple of 4 bytes, for some head sizes not of 8)
      if (a.wide) {
        *reinterpret_cast<uint2*>(to + p.code) = word;
      } else {
        *reinterpret_cast<uint32_t*>(to + p.code) = word.x;
        *reinterpret_cast<uint32_t*>(to + p.code + 4) = word.y;
      }
      if ((c & 1) == 0) *reinterpret_cast<uint32_t*>(to + p.meta) = meta;
    }
  }
}

// The values of eight codes: code -> 2^23 + code by its bits, then exact
// arithmetic and one rounding.
template <typename D>
__device__ __forceinline__ Vec8<D> restore(uint32_t w, float2 s2, float2 m2) {
  float f[8];
  const float2 back = make_float2(-8388608.f, -8388608.f);
  uint32_t magic;  // 2^23, kept in a register: (x & 15) | magic is one instruction
  asm("mov.u32 %0, 0x4B000000;" : "=r"(magic));
  auto code = [&](uint32_t x) -> float {
    uint32_t d;
    asm("lop3.b32 %0, %1, 15, %2, 0xEA;" : "=r"(d) : "r"(x), "r"(magic));
    return __uint_as_float(d);
  };
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 c = make_float2(code(w >> (4 * e)), code(w >> (4 * e + 4)));
    const float2 y = fma2_rn(add2_rn(c, back), s2, m2);
    f[e] = y.x;
    f[e + 1] = y.y;
  }
  return from_f32<D>(f);
}

template <typename D>
__global__ void __launch_bounds__(kGatherWarps * 32) gather_cache_q4_kernel(Q4CacheArgs a) {
  const int lane = threadIdx.x & 31;
  // a CTA takes 32 units of kGatherWarps tokens, the next CTA the next 32 of the same
  // tokens (the groups on the grid's y axis, far apart in time: 63.5 us for 65K tokens, so 59.5)
  const uint32_t block = a.groups == 1 ? blockIdx.x : blockIdx.x / a.groups;
  const int64_t t = static_cast<int64_t>(block) * kGatherWarps + (threadIdx.x >> 5);
  if (t >= a.num_tokens) return;
  const int c = static_cast<int>(blockIdx.x - block * a.groups) * 32 + lane;
  const int64_t s = slot_of(a, t);
  if (s < 0 || c >= a.row_units) return;
  const RowPlace p = row_place(c, a.units_per_head);
  const int64_t src = row_of(a, s);
  const bool has_v = a.value != nullptr;
  uint2 word[2] = {};
  uint32_t meta[2] = {};
#pragma unroll
  for (int tensor = 0; tensor < 2; ++tensor) {
    if (tensor && !has_v) break;
    const uint8_t* from = static_cast<const uint8_t*>(tensor ? a.value_cache : a.key_cache) + src;
    if (a.wide) {
      word[tensor] = __ldg(reinterpret_cast<const uint2*>(from + p.code));
    } else {
      word[tensor].x = __ldg(reinterpret_cast<const uint32_t*>(from + p.code));
      word[tensor].y = __ldg(reinterpret_cast<const uint32_t*>(from + p.code + 4));
    }
    meta[tensor] = __ldg(reinterpret_cast<const uint32_t*>(from + p.meta));
  }
#pragma unroll
  for (int tensor = 0; tensor < 2; ++tensor) {
    if (tensor && !has_v) break;
    D* dst = static_cast<D*>(const_cast<void*>(tensor ? a.value : a.key)) +
             t * (tensor ? a.value_stride : a.key_stride) + 16 * c;
    const float2 sm = widen(meta[tensor], f16{});
    const float2 s2 = make_float2(sm.x, sm.x), m2 = make_float2(sm.y, sm.y);
    store_unit(dst, Unit<D>{{restore<D>(word[tensor].x, s2, m2), restore<D>(word[tensor].y, s2, m2)}},
               a.whole32);
  }
}

// What both launchers derive from the arguments.
void derive(Q4CacheArgs& a, int64_t elem_bytes) {
  a.groups = static_cast<uint32_t>((a.row_units + 31) / 32);
  // 8-byte accesses to the codes: head rows (10 * units bytes) and blocks on multiples of 8
  a.wide = a.units_per_head % 4 == 0 && a.block_stride % 8 == 0;
  // 32-byte accesses to the rows
  const int64_t key_step = a.key_stride * elem_bytes, value_step = a.value_stride * elem_bytes;
  a.whole32 = ((reinterpret_cast<uintptr_t>(a.key) | reinterpret_cast<uintptr_t>(a.value) |
                static_cast<uintptr_t>(key_step) | static_cast<uintptr_t>(value_step)) &
               31u) == 0u;
}

}  // namespace

pa_status launch_reshape_and_cache_q4(Q4CacheArgs a, pa_dtype src, cudaStream_t stream) {
  derive(a, src == PA_FP32 ? 4 : 2);
  const int64_t blocks = (a.num_tokens + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFFll || a.groups > 65535u) return PA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), a.groups);
  switch (src) {
    case PA_BF16: reshape_and_cache_q4_kernel<bf16><<<grid, kWarps * 32, 0, stream>>>(a); break;
    case PA_FP16: reshape_and_cache_q4_kernel<f16><<<grid, kWarps * 32, 0, stream>>>(a); break;
    case PA_FP32: reshape_and_cache_q4_kernel<float><<<grid, kWarps * 32, 0, stream>>>(a); break;
    default: return PA_ERR_UNSUPPORTED;
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status launch_gather_cache_q4(Q4CacheArgs a, pa_dtype dst, cudaStream_t stream) {
  derive(a, dst == PA_FP32 ? 4 : 2);
  const int64_t blocks = (a.num_tokens + kGatherWarps - 1) / kGatherWarps;
  if (blocks > 0x7FFFFFFFll / a.groups) return PA_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(blocks * a.groups);
  switch (dst) {
    case PA_BF16: gather_cache_q4_kernel<bf16><<<grid, kGatherWarps * 32, 0, stream>>>(a); break;
    case PA_FP16: gather_cache_q4_kernel<f16><<<grid, kGatherWarps * 32, 0, stream>>>(a); break;
    case PA_FP32: gather_cache_q4_kernel<float><<<grid, kGatherWarps * 32, 0, stream>>>(a); break;
    default: return PA_ERR_UNSUPPORTED;
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa_detail
