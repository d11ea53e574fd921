// window.cuh -- what the sliding-window attention kernels share: their launches, and
// the places that a window leaves (window_cut.h).
#pragma once

#include <cudaTypedefs.h>

#include "pa_internal.cuh"
#include "window_cut.h"

namespace pa_detail {

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
