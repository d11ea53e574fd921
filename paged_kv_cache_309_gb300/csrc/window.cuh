// window.cuh -- what the sliding-window attention kernels share: the rows that a
// window leaves as one range of places, and their launches.
#pragma once

#include <cudaTypedefs.h>

#include "pa_internal.cuh"

namespace pa_detail {

// Pieces of 2^log2_rpb rows (part or all of a block) that hold a first token come first,
// then those from the one that the window starts in; the pieces between are left
// out, so places 0 .. len - 1 are rows 0 .. cut - 1, then rows cut + skip and on.
struct WindowRange {
  int low;   // first row of the window
  int cut;   // places below it are the rows of the same number
  int skip;  // rows left out there
  int len;   // places
  __device__ __forceinline__ int row(int place) const { return place < cut ? place : place + skip; }
  // which of the 64 rows from `first` on are visible
  __device__ __forceinline__ uint64_t visible(int first, int num_sink) const {
    return below(num_sink - first) | ~below(low - first);
  }
  static __device__ __forceinline__ uint64_t below(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
  }
};
// of a context of `len` rows whose window starts at row `low`
__device__ __forceinline__ WindowRange window_range(int len, int low, int num_sink, int log2_rpb) {
  WindowRange r;
  r.low = low;
  const int sinks = min(num_sink, len);
  const int first = (sinks + (1 << log2_rpb) - 1) >> log2_rpb;  // pieces with first tokens
  r.cut = first << log2_rpb;
  r.skip = max(0, (low >> log2_rpb) - first) << log2_rpb;
  r.len = len - r.skip;
  return r;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // decode.cu

size_t window_decode_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                     int32_t window, int32_t num_sink, int32_t max_context_len);
// (a.plan is not used)
pa_status launch_window_decode(const DecodeArgs& a, int32_t window, int32_t num_sink,
                               int32_t max_context_len, cudaStream_t stream);

struct WindowPrefillArgs {
  PrefillArgs p;
  int64_t total_tokens;  // rows of q and out
  int32_t window, num_sink;
};
pa_status launch_window_prefill(const WindowPrefillArgs& a, cudaStream_t stream);

}  // namespace pa_detail
