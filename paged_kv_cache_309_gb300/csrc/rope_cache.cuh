// rope_cache.cuh -- arguments of the rotate-and-append launch (rope_cache.cu).
#pragma once

#include "pa_internal.cuh"

namespace pa_detail {

struct RopeArgs {
  void* q_out;
  const void* q;
  const void* key;
  const void* value;
  void* key_cache;
  void* value_cache;
  const float* cos_sin;  // [max_positions, rot_dim]: cosines, then sines
  const int64_t* positions;
  const int64_t* slot_mapping;
  const int64_t* swa;
  const float* k_scale;
  const float* v_scale;
  int64_t swa_len, num_tokens, max_positions, num_slots;
  int64_t q_out_stride, q_stride, key_stride, value_stride, block_stride;  // elements
  int32_t num_q_heads, num_kv_heads, head_size, rot_dim, block_size;
  // set by the launcher: lanes of a head (log2), steps of q's heads and of k's (and v's),
  // warps per token
  int32_t log2_lanes, q_steps, kv_steps;
  uint32_t parts;
};
pa_status launch_rope_and_cache(RopeArgs a, pa_dtype src, pa_dtype dst, bool interleaved,
                                cudaStream_t stream);

}  // namespace pa_detail
