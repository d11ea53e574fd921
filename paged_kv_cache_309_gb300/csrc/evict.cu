// evict.cu -- eviction by accumulated attention weight: the choice of the
// tokens each (sequence, kv head) keeps, and the moving of their rows.
//
// Choice.  A sum becomes an unsigned key of the same order (NaN lowest,
// protected tokens highest); a radix search of four 8-bit digits finds the
// key of rank `budget`, and one ordered pass writes the indices of every key
// above it and of the first ties, ascending, with the sums beside them.
//
// Moving.  Row j of the kept list comes from token keep[j].  Into other
// blocks every row is independent.  In place (keep[j] >= j, ascending) one
// CTA walks a (sequence, kv head, column range) in chunks and stores a chunk
// only after every load of the chunks up to it: what a store overwrites,
// position j, can be the source of rows <= j only.
#include "pa_internal.cuh"

namespace pa_detail {
namespace {

using namespace pa;

constexpr int kSelThreads = 1024;

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sums over the CTA's threads of x (two 16-bit counts in one word);
// total: the sum over all.  warp_sums: 33 words of shared memory.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* warp_sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const uint32_t w = lane < kSelThreads / 32 ? warp_sums[lane] : 0u;
    uint32_t wi = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, wi, off);
      if (lane >= off) wi += y;
    }
    warp_sums[lane] = wi - w;
    if (lane == 31) warp_sums[32] = wi;
  }
  __syncthreads();
  const uint32_t before = warp_sums[warp] + incl - x;
  total = warp_sums[32];
  __syncthreads();
  return before;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_sums[33];
  __shared__ uint32_t found[2];  // digit, rank within it
  const int row = blockIdx.x;
  const int b = row / a.num_kv_heads;
  const int tid = threadIdx.x;
  const int L = min(max(__ldg(a.context_lens + b), 0), a.sums_len);
  const int n = min(L, a.budget);
  if (row == b * a.num_kv_heads && tid == 0) a.new_lens[b] = n;
  int32_t* keep = a.keep + static_cast<int64_t>(row) * a.budget;
  const float* in = a.sums_in + static_cast<int64_t>(row) * a.sums_len;
  float* out = a.sums_out == nullptr ? nullptr : a.sums_out + static_cast<int64_t>(row) * a.sums_len;
  for (int j = n + tid; j < a.budget; j += kSelThreads) keep[j] = -1;
  if (L <= a.budget) {
    for (int j = tid; j < n; j += kSelThreads) {
      keep[j] = j;
      if (out != nullptr && out != in) out[j] = in[j];
    }
    return;
  }
  auto key_of = [&](int t, float x) -> uint32_t {
    return t < a.num_sink || t >= L - a.num_recent ? 0xFFFFFFFFu : order_key(x);
  };
  uint32_t prefix = 0u;
  uint32_t rank = static_cast<uint32_t>(n);  // of the kept, the lowest key's rank from the top
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0u;
    __syncthreads();
    for (int t = tid; t < L; t += kSelThreads) {
      const uint32_t k = key_of(t, in[t]);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t left = rank;
      int d = 255;
      while (d > 0 && hist[d] < left) left -= hist[d--];
      found[0] = static_cast<uint32_t>(d);
      found[1] = left;
    }
    __syncthreads();
    prefix |= found[0] << shift;
    rank = found[1];
    __syncthreads();
  }
  // keys above `prefix` are kept, and the first `rank` equal to it
  uint32_t above = 0u, equal = 0u;
  for (int base = 0; base < L; base += kSelThreads) {
    const int t = base + tid;
    float x = 0.f;
    uint32_t is_above = 0u, is_equal = 0u;
    if (t < L) {
      x = in[t];
      const uint32_t k = key_of(t, x);
      is_above = k > prefix;
      is_equal = k == prefix;
    }
    uint32_t total;
    const uint32_t before = block_scan(is_above | (is_equal << 16), warp_sums, total);
    const uint32_t my_above = above + (before & 0xFFFFu), my_equal = equal + (before >> 16);
    if (is_above || (is_equal && my_equal < rank)) {
      const uint32_t j = my_above + min(my_equal, rank);
      keep[j] = t;
      if (out != nullptr) out[j] = x;  // j <= t: read above, by this chunk or an earlier one
    }
    above += total & 0xFFFFu;
    equal += total >> 16;
  }
}

// ----------------------------------------------------------------- moving --
constexpr int kMoveThreads = 256;
constexpr int kMoveUnits = 8;  // 16-byte units in flight per thread

// Units are 16 bytes; a CTA moves columns [u0, u0 + U) of rows [j0, j1) of one
// tensor, in chunks of kMoveThreads * kMoveUnits / U rows.
template <bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads) cache_compact_kernel(const CompactArgs a) {
  const int g = blockIdx.y, b = blockIdx.z;
  const int n = min(max(__ldg(a.keep_lens + b), 0), a.keep_len);
  const int row_units = a.row_units;
  int x = blockIdx.x;
  const int tensor = a.v_cache == nullptr ? 0 : x & 1;
  if (a.v_cache != nullptr) x >>= 1;
  uint4* cache = static_cast<uint4*>(tensor ? a.v_cache : a.k_cache);
  int u0 = 0, U = row_units, j0 = 0, j1 = n;
  if (kInPlace) {
    u0 = x * a.units_per_cta;
    U = min(a.units_per_cta, row_units - u0);
  } else {
    j0 = x * a.rows_per_cta;
    j1 = min(j0 + a.rows_per_cta, n);
  }
  if (j0 >= j1) return;
  const int32_t* keep = a.keep + (static_cast<int64_t>(b) * a.num_kv_heads + g) * a.keep_len;
  const int32_t* src_table = a.src_table + static_cast<int64_t>(b) * a.src_max_blocks;
  const int32_t* dst_table = a.dst_table + static_cast<int64_t>(b) * a.dst_max_blocks;
  // unit offset of logical row t of this head, or -1
  auto place = [&](const int32_t* table, int max_blocks, int t) -> int64_t {
    if (t < 0) return -1;
    const int blk = t / a.block_size;
    if (blk >= max_blocks) return -1;
    const int id = __ldg(table + blk);
    if (id < 0 || id >= a.num_blocks) return -1;
    return ((static_cast<int64_t>(id) * a.block_size + (t - blk * a.block_size)) * a.num_kv_heads +
            g) * row_units + u0;
  };
  const int chunk = max(1, kMoveThreads * kMoveUnits / U);  // rows
  for (int c0 = j0; c0 < j1; c0 += chunk) {
    uint4 v[kMoveUnits];
    int64_t to[kMoveUnits];
    const int units = min(chunk, j1 - c0) * U;
    for (int base = 0; base < units; base += kMoveThreads * kMoveUnits) {
#pragma unroll
      for (int i = 0; i < kMoveUnits; ++i) {
        const int at = base + threadIdx.x + kMoveThreads * i;
        to[i] = -1;
        if (at < units) {
          const int r = at / U, u = at - r * U;
          const int j = c0 + r, t = __ldg(keep + j);
          const int64_t from = place(src_table, a.src_max_blocks, t);
          const int64_t dst = place(dst_table, a.dst_max_blocks, j);
          if (from >= 0 && dst >= 0 && from != dst) {
            v[i] = cache[from + u];
            to[i] = dst + u;
          }
        }
      }
      if (kInPlace) __syncthreads();  // every load of the chunk, then its stores
#pragma unroll
      for (int i = 0; i < kMoveUnits; ++i)
        if (to[i] >= 0) cache[to[i]] = v[i];
      if (kInPlace) __syncthreads();
    }
  }
}

}  // namespace

pa_status launch_evict_select(const SelectArgs& a, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  evict_select_kernel<<<static_cast<unsigned>(rows), kSelThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status launch_cache_compact(CompactArgs a, bool in_place, cudaStream_t stream) {
  const unsigned tensors = a.v_cache == nullptr ? 1u : 2u;
  dim3 grid(1, static_cast<unsigned>(a.num_kv_heads), static_cast<unsigned>(a.num_seqs));
  if (in_place) {
    a.units_per_cta = a.row_units < 4 ? a.row_units : 4;
    grid.x = tensors * static_cast<unsigned>((a.row_units + a.units_per_cta - 1) / a.units_per_cta);
    cache_compact_kernel<true><<<grid, kMoveThreads, 0, stream>>>(a);
  } else {
    const int32_t rows = kMoveThreads * kMoveUnits / a.row_units;
    a.rows_per_cta = rows < 1 ? 1 : rows;
    const int64_t blocks =
        tensors * ((static_cast<int64_t>(a.keep_len) + a.rows_per_cta - 1) / a.rows_per_cta);
    if (blocks > 0x7FFFFFFFll) return PA_ERR_UNSUPPORTED;
    grid.x = static_cast<unsigned>(blocks);
    cache_compact_kernel<false><<<grid, kMoveThreads, 0, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa_detail
