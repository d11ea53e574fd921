// q4_cut.h -- the integer arithmetic of the 4-bit decode kernel's balanced cut
// and of the places its partials take in the workspace.  Plain C++: the kernel,
// its launch and a host test compile the same lines.
//
// Units of 64 tokens lie end to end in sequence order; unit t (counted over
// all sequences) of sequence b sits at cost t + kPieceCost (b + 1), the line is
// total = units + kPieceCost B long, and its chunk is floor(cost parts / total)
// with parts = min(C, total): a step of one unit moves at most one chunk on, so
// no chunk inside a sequence's span is empty.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PA_CUT_FN __host__ __device__ __forceinline__
#else
#define PA_CUT_FN inline
#endif

namespace pa_detail {
namespace q4cut {

constexpr int kUnit = 64;           // tokens per unit of the cut
constexpr int kPieceCost = 2;       // units charged for a sequence's start
constexpr int kMaxChunks = 32767;   // half of an `info` word each: first chunk, pieces
constexpr int kPartialFloats = 128; // of a partial row (the head size)

PA_CUT_FN int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }
PA_CUT_FN int64_t max64(int64_t a, int64_t b) { return a > b ? a : b; }

PA_CUT_FN int units_of_len(int len) { return (len + kUnit - 1) / kUnit; }
PA_CUT_FN int64_t total_cost(int64_t units, int num_seqs) {
  return units + static_cast<int64_t>(kPieceCost) * num_seqs;
}
PA_CUT_FN int64_t parts_of(int64_t total, int chunks) {
  return min64(total, static_cast<int64_t>(chunks));
}
// the chunk of unit t of sequence b
PA_CUT_FN int chunk_of(int64_t t, int b, int64_t total, int parts) {
  return static_cast<int>((t + static_cast<int64_t>(kPieceCost) * (b + 1)) * parts / total);
}
// chunk k begins at the first unit whose cost reaches ceil(k total / parts):
PA_CUT_FN int64_t chunk_begin_cost(int64_t k, int64_t total, int64_t parts) {
  return (k * total + parts - 1) / parts;
}
// whether that unit is one of sequence b's (n units, `pre` before it), given that no
// sequence before has it: decided by its last unit, or by its first where sequences stay whole
PA_CUT_FN bool begins_in(int64_t x, int64_t pre, int n, int b, bool whole) {
  return n > 0 && pre + (whole ? 0 : n - 1) + static_cast<int64_t>(kPieceCost) * (b + 1) >= x;
}
// and which it is
PA_CUT_FN int64_t begin_unit(int64_t x, int64_t pre, int b, bool whole) {
  return whole ? pre : max64(x - static_cast<int64_t>(kPieceCost) * (b + 1), pre);
}

// Partial slot of a piece of a split sequence in chunk c: c - 1 for one that goes on from
// chunk c - 1; for a sequence's first piece one of its own behind those.
PA_CUT_FN int start_slot_of(int chunks, int num_seqs, int b, int c_first) {
  return chunks - 1 + (num_seqs <= chunks - 1 ? b : c_first);
}
PA_CUT_FN int slot_of_piece(int chunks, int num_seqs, int b, int c_first, int c) {
  return c == c_first ? start_slot_of(chunks, num_seqs, b, c_first) : c - 1;
}
// `info` of a sequence: 0 where it is not split
PA_CUT_FN int32_t info_of(int c_first, int c_last) {
  return c_first == c_last ? 0 : c_first << 16 | (c_last - c_first + 1);
}

// The launch: one wave of CTAs (`resident` chunks per kv head or pair of them), as far as the
// workspace's partial rows (num_seqs * num_splits per query head, some of them for `info`)
// hold what the cut can leave: a piece behind every inner chunk boundary and a
// first piece for every sequence that crosses one.
struct Launch {
  int32_t chunks;
  int32_t slots;       // partial slots per kv head
  bool whole;          // no partials: chunks begin at sequence starts
  int64_t info_float;  // offset of `info` from the partial rows, in floats
};
PA_CUT_FN Launch launch_of(int64_t resident, int64_t num_seqs, int64_t num_splits, int64_t kv_heads,
                           int64_t group) {
  Launch l;
  int64_t chunks = resident;
  const int64_t rows =
      num_seqs * num_splits - (num_seqs + kPartialFloats - 1) / kPartialFloats;
  l.whole = num_splits == 1;
  if (l.whole) {
    chunks = min64(chunks, num_seqs);
  } else if (chunks - 1 + min64(num_seqs, chunks - 1) > rows) {
    chunks = num_seqs < rows - num_seqs ? rows - num_seqs + 1 : rows / 2 + 1;
  }
  chunks = max64(min64(chunks, kMaxChunks), 1);
  l.chunks = static_cast<int32_t>(chunks);
  l.slots = static_cast<int32_t>(chunks - 1 + min64(num_seqs, chunks - 1));
  l.info_float = kv_heads * l.slots * group * kPartialFloats;
  return l;
}

}  // namespace q4cut
}  // namespace pa_detail
