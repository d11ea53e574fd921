// evict.cu -- eviction by accumulated attention weight: the choice of the
// tokens each (sequence, kv head) keeps, and the moving of their rows.
//
// Choice.  A sum becomes an unsigned key of the same order (NaN lowest,
// protected tokens highest); a radix search finds the key of rank `budget`,
// and one ordered pass writes the indices of every key above it and of the
// first ties, ascending, with the sums beside them.  A row is read once: the
// CTAs of a cluster hold a part of it each in shared memory, and join their
// digit counts through distributed shared memory.  Given the block tables (kPaged),
// tokens of dropped blocks get the lowest key of all and do not count as tokens: a
// kept one would have no row to move, and the row at its new place, whatever it
// holds, would be attended to (the look-ups: 59 us instead of 49 for 64 rows of 32K-128K).
// (One CTA re-reading its row for every digit: 222 us for 64 rows of 32K-128K, 27 us for 128
// rows of 2.3K; so: 49 and 7.3, bound by instruction issue, 0.68 of the cycles, not by the
// 21 MB read.)
//
// Moving.  Row j of the kept list comes from token keep[j].  The places of a
// chunk of rows are looked up once, a thread per row; then 16-byte units move,
// eight of K and eight of V in flight per thread (looked up per unit, the
// integer work alone took 136 us of a 284 us move of 1.07 GB; so: 161 us, HBM).
// Into other blocks every row is independent.  In place (keep[j] >= j,
// ascending) one CTA walks a column range of a (sequence, kv head) in chunks
// and stores a chunk only after every load of the chunks up to it: what a
// store overwrites, position j, can be the source of rows <= j only.
#include <atomic>

#include "pa_internal.cuh"

namespace pa_detail {
namespace {

using namespace pa;

constexpr int kSelThreads = 1024;
constexpr int kMaxSegment = 49152;  // and that shared memory holds at most (192 KB)
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;         // digits of 11, 11 and 10 bits
static_assert(kBins == 2 * kSelThreads, "a thread looks at two digits");
constexpr int kCandidates = 4096;   // keys of one first digit that every CTA of a cluster holds

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Whether token t of a sequence has a row (kPaged): its block is in the pool.
__device__ __forceinline__ bool has_row(const SelectArgs& a, const int32_t* table, int t) {
  const int blk = (a.block_size & (a.block_size - 1)) == 0 ? t >> (31 - __clz(a.block_size))
                                                           : t / a.block_size;
  if (blk >= a.max_blocks) return false;
  const int id = __ldg(table + blk);
  return id >= 0 && id < a.num_blocks;
}

// The order key with room below it for tokens without a row.
template <bool kPaged>
__device__ __forceinline__ uint32_t live_key(float x) {
  const uint32_t k = order_key(x);
  return kPaged && k == 0u ? 1u : k;  // (the lowest number's key is 0x007FFFFF)
}

// Tokens below L that have a row, counted by the whole CTA; shared: one word.
__device__ __forceinline__ int count_live(const SelectArgs& a, const int32_t* table, int L,
                                          int* shared) {
  if (threadIdx.x == 0) *shared = 0;
  __syncthreads();
  int live = 0;
  for (int64_t first = static_cast<int64_t>(threadIdx.x) * a.block_size; first < L;
       first += static_cast<int64_t>(blockDim.x) * a.block_size)
    if (has_row(a, table, static_cast<int>(first)))
      live += static_cast<int>(min(static_cast<int64_t>(a.block_size), L - first));
  live = __reduce_add_sync(0xffffffffu, live);
  if ((threadIdx.x & 31) == 0) atomicAdd(shared, live);
  __syncthreads();
  return *shared;
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

// Rows longer than a cluster holds: one CTA per row, re-read for every digit.
template <bool kPaged>
__global__ void __launch_bounds__(kSelThreads) evict_select_long_kernel(const SelectArgs a) {
  __shared__ int live_sum;
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_sums[33];
  __shared__ uint32_t found[2];  // digit, rank within it
  const int row = blockIdx.x;
  const int b = row / a.num_kv_heads;
  const int tid = threadIdx.x;
  const int L = min(max(__ldg(a.context_lens + b), 0), a.sums_len);
  const int32_t* table = kPaged ? a.block_tables + static_cast<int64_t>(b) * a.max_blocks : nullptr;
  const int live = kPaged ? count_live(a, table, L, &live_sum) : L;
  const int n = min(live, a.budget);
  if (row == b * a.num_kv_heads && tid == 0) a.new_lens[b] = n;
  int32_t* keep = a.keep + static_cast<int64_t>(row) * a.budget;
  const float* in = a.sums_in + static_cast<int64_t>(row) * a.sums_len;
  float* out = a.sums_out == nullptr ? nullptr : a.sums_out + static_cast<int64_t>(row) * a.sums_len;
  for (int j = n + tid; j < a.budget; j += kSelThreads) keep[j] = -1;
  if (kPaged && n == 0) return;
  if (n == L) {
    for (int j = tid; j < n; j += kSelThreads) {
      keep[j] = j;
      if (out != nullptr && out != in) out[j] = in[j];
    }
    return;
  }
  auto key_of = [&](int t, float x) -> uint32_t {
    if (kPaged && !has_row(a, table, t)) return 0u;
    return t < a.num_sink || t >= L - a.num_recent ? 0xFFFFFFFFu : live_key<kPaged>(x);
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

// ------------------------------------------------- a row held by a cluster --
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// two 32-bit words of another CTA of the cluster, at the address `local` has here
// (the barriers around the loads order them; no clobber, so that they overlap)
__device__ __forceinline__ uint2 cluster_load(const uint32_t* local, int rank) {
  uint32_t addr;
  uint2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ void cluster_store(const uint32_t* local, int rank, uint32_t x) {
  uint32_t addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}

template <bool kPaged>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectArgs a, int ranks) {
  constexpr uint32_t kNoRow = 0xFFFFFFFFu;  // a NaN's bits that stand for a token without a row
  __shared__ int live_sum;
  extern __shared__ float vals[];  // this CTA's part of the row
  __shared__ __align__(8) uint32_t hist[kBins];
  __shared__ uint32_t candidates[kCandidates];
  __shared__ uint32_t warp_sums[33];
  __shared__ uint32_t warp_above[kSelThreads / 32], warp_equal[kSelThreads / 32];
  __shared__ uint32_t found[4];  // digit, rank within it, its keys in the cluster, in lower CTAs
  __shared__ uint32_t appended;
  __shared__ __align__(8) uint32_t counts[2];  // of this CTA: above, equal
  const int row = blockIdx.x / ranks, rank_id = blockIdx.x - row * ranks;
  const int b = row / a.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = min(max(__ldg(a.context_lens + b), 0), a.sums_len);
  const int32_t* table = kPaged ? a.block_tables + static_cast<int64_t>(b) * a.max_blocks : nullptr;
  const int live = kPaged ? count_live(a, table, L, &live_sum) : L;
  const int n = min(live, a.budget);
  if (row == b * a.num_kv_heads && rank_id == 0 && tid == 0) a.new_lens[b] = n;
  int32_t* keep = a.keep + static_cast<int64_t>(row) * a.budget;
  const float* in = a.sums_in + static_cast<int64_t>(row) * a.sums_len;
  float* out = a.sums_out == nullptr ? nullptr : a.sums_out + static_cast<int64_t>(row) * a.sums_len;
  const int step = ranks * kSelThreads, me = rank_id * kSelThreads + tid;
  for (int64_t j = static_cast<int64_t>(n) + me; j < a.budget; j += step) keep[j] = -1;
  if (kPaged && n == 0) return;  // (here and below every CTA of the cluster: no barrier is missed)
  if (n == L) {
    for (int j = me; j < n; j += step) {
      keep[j] = j;
      if (out != nullptr && out != in) out[j] = in[j];
    }
    return;
  }
  const int seg = ((L + ranks - 1) / ranks + 31) & ~31;  // <= the shared memory's
  const int t0 = min(rank_id * seg, L), size = min(seg, L - t0);
  auto key = [&](int i, float x) -> uint32_t {
    const int t = t0 + i;
    if (kPaged && __float_as_uint(x) == kNoRow) return 0u;
    return t < a.num_sink || t >= L - a.num_recent ? 0xFFFFFFFFu : live_key<kPaged>(x);
  };
  auto clear_hist = [&]() { reinterpret_cast<uint2*>(hist)[tid] = make_uint2(0u, 0u); };
  // The digit that holds the key of rank `rank` (counted from the largest), from every
  // digit's count: this thread's are those of digits d + 1 (c.y) and d (c.x), lower.y
  // and lower.x of them in CTAs before this one.
  const int d = kBins - 2 - 2 * tid;
  auto find_digit = [&](uint2 c, uint2 lower, uint32_t rank) {
    uint32_t total;
    const uint32_t before = block_scan(c.x + c.y, warp_sums, total);
    if (before < rank && rank <= before + c.x + c.y) {
      const bool first = rank <= before + c.y;
      found[0] = static_cast<uint32_t>(first ? d + 1 : d);
      found[1] = rank - before - (first ? 0u : c.y);
      found[2] = first ? c.y : c.x;
      found[3] = first ? lower.y : lower.x;
    }
  };
  auto cluster_digits = [&](uint32_t rank) {
    uint2 c = make_uint2(0u, 0u), lower = c;
    if (ranks == 1) {
      c = *reinterpret_cast<const uint2*>(hist + d);
    } else {
      uint2 v[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        v[r] = r < ranks ? cluster_load(hist + d, r) : make_uint2(0u, 0u);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (r == rank_id) lower = c;
        c.x += v[r].x;
        c.y += v[r].y;
      }
    }
    find_digit(c, lower, rank);
  };
  auto all_sync = [&]() {
    if (ranks > 1) cluster_sync();
    else __syncthreads();
  };

  // ---- first digit (11 bits), counted as the row is read
  clear_hist();
  if (tid == 0) appended = 0u;
  __syncthreads();
  for (int i0 = tid; i0 < size; i0 += 8 * kSelThreads) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i0 + k * kSelThreads < size) x[k] = in[t0 + i0 + k * kSelThreads];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + k * kSelThreads;
      if (i < size) {
        if (kPaged) {  // (a NaN of the sums with those bits is another NaN)
          if (!has_row(a, table, t0 + i)) x[k] = __uint_as_float(kNoRow);
          else if (__float_as_uint(x[k]) == kNoRow) x[k] = __uint_as_float(kNoRow - 1u);
        }
        vals[i] = x[k];
        atomicAdd(&hist[key(i, x[k]) >> 21], 1u);
      }
    }
  }
  all_sync();
  cluster_digits(static_cast<uint32_t>(n));
  __syncthreads();
  uint32_t prefix = found[0] << 21, rank = found[1];
  const uint32_t num = found[2], lower = found[3];
  if (num <= kCandidates) {
    // the keys with that digit, given to every CTA, which find the rest of
    // the key by themselves
    for (int i = tid; i < size; i += kSelThreads) {
      const uint32_t k = key(i, vals[i]);
      if (k >> 21 == prefix >> 21) {
        const uint32_t at = lower + atomicAdd(&appended, 1u);
        if (ranks == 1) {
          candidates[at] = k;
        } else {
          for (int r = 0; r < ranks; ++r) cluster_store(candidates + at, r, k);
        }
      }
    }
    all_sync();
#pragma unroll
    for (int pass = 1; pass < 3; ++pass) {
      const int shift = pass == 1 ? 10 : 0, known = pass == 1 ? 21 : 10;
      clear_hist();
      __syncthreads();
      for (uint32_t i = tid; i < num; i += kSelThreads) {
        const uint32_t k = candidates[i];
        if (k >> known == prefix >> known)
          atomicAdd(&hist[(k >> shift) & (pass == 1 ? 2047u : 1023u)], 1u);
      }
      __syncthreads();
      find_digit(*reinterpret_cast<const uint2*>(hist + d), make_uint2(0u, 0u), rank);
      __syncthreads();
      prefix |= found[0] << shift;
      rank = found[1];
      __syncthreads();
    }
  } else {
    // many keys with that digit (ties): the other digits over the whole row too
#pragma unroll
    for (int pass = 1; pass < 3; ++pass) {
      const int shift = pass == 1 ? 10 : 0, known = pass == 1 ? 21 : 10;
      all_sync();  // every CTA has read the counts
      clear_hist();
      __syncthreads();
      for (int i = tid; i < size; i += kSelThreads) {
        const uint32_t k = key(i, vals[i]);
        if (k >> known == prefix >> known)
          atomicAdd(&hist[(k >> shift) & (pass == 1 ? 2047u : 1023u)], 1u);
      }
      all_sync();
      cluster_digits(rank);
      __syncthreads();
      prefix |= found[0] << shift;
      rank = found[1];
    }
  }
  // ---- keys above `prefix` are kept, and the first `rank` equal to it: each
  // warp counts its consecutive part, then writes at its place
  constexpr int kWarps = kSelThreads / 32;
  const int per = ((size + kWarps - 1) / kWarps + 31) & ~31;
  const int w0 = min(warp * per, size), w1 = min(w0 + per, size);
  uint32_t above = 0u, equal = 0u;
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = key(i, vals[i]);
    above += k > prefix;
    equal += k == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    warp_above[warp] = above;
    warp_equal[warp] = equal;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t x = warp_above[lane], y = warp_equal[lane];
    const uint32_t x0 = x, y0 = y;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t p = __shfl_up_sync(0xffffffffu, x, off), q = __shfl_up_sync(0xffffffffu, y, off);
      if (lane >= off) {
        x += p;
        y += q;
      }
    }
    warp_above[lane] = x - x0;
    warp_equal[lane] = y - y0;
    if (lane == 31) {
      counts[0] = x;
      counts[1] = y;
    }
  }
  all_sync();
  above = warp_above[warp];
  equal = warp_equal[warp];
  if (ranks > 1) {
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (r < rank_id) {
        const uint2 c = cluster_load(counts, r);
        above += c.x;
        equal += c.y;
      }
    }
    cluster_sync();  // no CTA leaves while its counts are read
  }
#pragma unroll 4
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const float x = i < w1 ? vals[i] : 0.f;
    const uint32_t k = i < w1 ? key(i, x) : 0u;
    const bool is_above = i < w1 && k > prefix, is_equal = i < w1 && k == prefix;
    const uint32_t ma = __ballot_sync(0xffffffffu, is_above);
    const uint32_t mq = __ballot_sync(0xffffffffu, is_equal);
    const uint32_t low = (1u << lane) - 1u;
    const uint32_t na = above + __popc(ma & low), ne = equal + __popc(mq & low);
    if (is_above || (is_equal && ne < rank)) {
      const uint32_t j = na + min(ne, rank);
      keep[j] = t0 + i;
      if (out != nullptr) out[j] = x;  // (in place: the whole row was read above)
    }
    above += __popc(ma);
    equal += __popc(mq);
  }
}

// ----------------------------------------------------------------- moving --
constexpr int kMoveThreads = 256;
constexpr int kMoveUnits = 4;         // 16-byte units of a tensor in flight per thread, of both
constexpr int kMoveUnitsInPlace = 8;  // of one tensor

// Units are 16 bytes; a CTA moves columns [u0, u0 + U) of rows [j0, j1) in chunks of
// kChunk / U rows.  kInPlace: of one tensor (K or V); else of both.
template <bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads, kInPlace ? 3 : 4)
    cache_compact_kernel(const CompactArgs a) {
  constexpr int kUnits = kInPlace ? kMoveUnitsInPlace : kMoveUnits;
  constexpr int kChunk = kMoveThreads * kUnits;
  // slots (block * block_size + offset) of a chunk's rows, -1: not moved
  __shared__ int2 places[kInPlace ? 2 : 1][kChunk];
  const int g = blockIdx.y, b = blockIdx.z;
  const int n = min(max(__ldg(a.keep_lens + b), 0), a.keep_len);
  const int tensors = kInPlace && a.v_cache != nullptr ? 2 : 1;
  const int tensor = kInPlace ? blockIdx.x % tensors : 0;
  const int x = kInPlace ? blockIdx.x / tensors : blockIdx.x;
  const int part = x % a.parts;
  const int u0 = part * a.units_per_cta;
  const int U = min(a.units_per_cta, a.row_units - u0);
  const int rows = kChunk / a.units_per_cta;  // of a chunk
  const int j0 = kInPlace ? 0 : x / a.parts * rows;
  const int j1 = kInPlace ? n : min(j0 + rows, n);
  if (j0 >= j1) return;
  const int32_t* keep = a.keep + (static_cast<int64_t>(b) * a.num_kv_heads + g) * a.keep_len;
  const int32_t* src_table = a.src_table + static_cast<int64_t>(b) * a.src_max_blocks;
  const int32_t* dst_table = a.dst_table + static_cast<int64_t>(b) * a.dst_max_blocks;
  uint4* k_cache = static_cast<uint4*>(kInPlace && tensor ? a.v_cache : a.k_cache);
  uint4* v_cache = kInPlace ? nullptr : static_cast<uint4*>(a.v_cache);
  // at / U for at < kChunk
  const uint32_t magic = U > 1 ? 0xFFFFFFFFu / static_cast<uint32_t>(U) + 1u : 0u;
  auto place = [&](const int32_t* table, int max_blocks, int t) -> int {
    if (t < 0) return -1;
    const int blk = (a.block_size & (a.block_size - 1)) == 0 ? t >> (31 - __clz(a.block_size))
                                                             : t / a.block_size;
    if (blk >= max_blocks) return -1;
    const int id = __ldg(table + blk);
    if (id < 0 || id >= a.num_blocks) return -1;
    return id * a.block_size + (t - blk * a.block_size);
  };
  auto look_up = [&](int c0, int2* to) {
    for (int r = threadIdx.x; r < rows && c0 + r < j1; r += kMoveThreads) {
      int2 p;
      p.x = place(src_table, a.src_max_blocks, __ldg(keep + c0 + r));
      p.y = place(dst_table, a.dst_max_blocks, c0 + r);
      if (p.x < 0 || p.y < 0 || p.x == p.y) p.y = -1;
      to[r] = p;
    }
  };
  auto unit = [&](int slot, int u) -> int64_t {
    return (static_cast<int64_t>(slot) * a.num_kv_heads + g) * a.row_units + u0 + u;
  };
  // Loads of the chunk at c0 (its places in `from`), and their stores
  auto load = [&](int c0, const int2* places_of, uint4 (&k)[kUnits], uint4* v,
                  int64_t (&to)[kUnits]) {
    const int units = min(rows, j1 - c0) * U;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int at = threadIdx.x + kMoveThreads * i;
      to[i] = -1;
      if (at < units) {
        const int r = U > 1 ? static_cast<int>(__umulhi(static_cast<uint32_t>(at), magic)) : at;
        const int u = at - r * U;
        const int2 p = places_of[r];
        if (p.y >= 0) {
          to[i] = unit(p.y, u);
          const int64_t from = unit(p.x, u);
          k[i] = k_cache[from];
          if (!kInPlace && v_cache != nullptr) v[i] = v_cache[from];
        }
      }
    }
  };
  auto store = [&](const uint4 (&k)[kUnits], const uint4* v, const int64_t (&to)[kUnits]) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if (to[i] >= 0) {
        k_cache[to[i]] = k[i];
        if (!kInPlace && v_cache != nullptr) v_cache[to[i]] = v[i];
      }
    }
  };
  look_up(j0, places[0]);
  __syncthreads();
  uint4 k0[kUnits];
  int64_t to0[kUnits];
  if constexpr (!kInPlace) {
    uint4 v0[kUnits];
    load(j0, places[0], k0, v0, to0);
    store(k0, v0, to0);
  } else {
    // (the next chunk's loads ahead of this one's stores, in a second set of
    // registers, made it slower: 223 -> 403 us for 1.07 GB)
    int buf = 0;
    for (int c0 = j0; c0 < j1; c0 += rows, buf ^= 1) {
      load(c0, places[buf], k0, nullptr, to0);
      if (c0 + rows < j1) look_up(c0 + rows, places[buf ^ 1]);
      __syncthreads();  // every load of the chunk, then its stores
      store(k0, nullptr, to0);
    }
  }
}

}  // namespace

namespace {

template <bool kPaged>
pa_status launch_select(const SelectArgs& a, cudaStream_t stream) {
  const unsigned rows = static_cast<unsigned>(a.num_seqs) * static_cast<unsigned>(a.num_kv_heads);
  // CTAs per row: parts of 16K sums are the fastest for a row (131072 sums: 25 us, parts of
  // 32K: 33), but only some 16 clusters of eight run at a time, so where the rows
  // fill the GPU parts of 32K give more (64 rows: 50 us instead of 75)
  int sms = num_sms_current_device();
  if (sms <= 0) sms = 148;
  auto ranks_for = [&](int64_t part) {
    int r = 1;
    while (r < kMaxCluster && r * part < a.sums_len) r *= 2;
    return r;
  };
  int ranks = ranks_for(16384);
  if (static_cast<int64_t>(rows) * ranks > sms) ranks = ranks_for(32768);
  if (static_cast<int64_t>(ranks) * kMaxSegment < a.sums_len) {
    evict_select_long_kernel<kPaged><<<rows, kSelThreads, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  }
  static std::atomic<uint64_t> smem_raised{0};
  if (!ensure_smem_limit(evict_select_kernel<kPaged>, kMaxSegment * 4, smem_raised)) return PA_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(rows * static_cast<unsigned>(ranks));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = (((a.sums_len + ranks - 1) / ranks + 31) & ~31) * sizeof(float);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, evict_select_kernel<kPaged>, a, ranks) != cudaSuccess) {
    cudaGetLastError();
    return PA_ERR_CUDA;
  }
  return PA_OK;
}

}  // namespace

pa_status launch_evict_select(const SelectArgs& a, cudaStream_t stream) {
  return a.block_tables != nullptr ? launch_select<true>(a, stream)
                                   : launch_select<false>(a, stream);
}

pa_status launch_cache_compact(CompactArgs a, bool in_place, cudaStream_t stream) {
  const int tensors = in_place && a.v_cache != nullptr ? 2 : 1;
  // columns per CTA: whole rows, as far as a chunk holds a row.  In place the columns
  // are the only parallelism beside sequences and kv heads: 128 bytes where those fill
  // the GPU (1.07 GB, 128 rows and tensors: 223 us, 64 bytes 273, whole rows 321), down to 32 where
  // they do not (16 of them: 97 us, 64 bytes 111, 128 bytes 156)
  const int chunk = kMoveThreads * (in_place ? kMoveUnitsInPlace : kMoveUnits);
  int sms = num_sms_current_device();
  if (sms <= 0) sms = 148;
  int most = in_place ? 8 : chunk;
  const int64_t lists = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads * tensors;
  while (in_place && most > 2 && lists * ((a.row_units + most - 1) / most) * 2 < 3 * sms) most /= 2;
  a.units_per_cta = a.row_units < most ? a.row_units : most;
  a.parts = (a.row_units + a.units_per_cta - 1) / a.units_per_cta;
  const int rows = chunk / a.units_per_cta;
  const int64_t blocks = in_place ? static_cast<int64_t>(tensors) * a.parts
                                  : (static_cast<int64_t>(a.keep_len) + rows - 1) / rows * a.parts;
  if (blocks > 0x7FFFFFFFll) return PA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(a.num_kv_heads),
                  static_cast<unsigned>(a.num_seqs));
  if (in_place)
    cache_compact_kernel<true><<<grid, kMoveThreads, 0, stream>>>(a);
  else
    cache_compact_kernel<false><<<grid, kMoveThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa_detail
