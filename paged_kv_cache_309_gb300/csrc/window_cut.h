// window_cut.h -- the integer arithmetic of the sliding-window attention calls: the rows that
// a window leaves as one range of places, and the cut of a decode batch with what it needs of
// the workspace.  Plain C++: the kernels, their launches and a host test compile the same lines.
#pragma once

#include <stddef.h>

#include "q4_cut.h"

namespace pa_detail {

// Pieces of 2^log2_rpb rows (part or all of a block) that hold a first token come first,
// then those from the one that the window starts in; the pieces between are left
// out, so places 0 .. len - 1 are rows 0 .. cut - 1, then rows cut + skip and on.
struct WindowRange {
  int low;   // first row of the window
  int cut;   // places below it are the rows of the same number
  int skip;  // rows left out there
  int len;   // places
  PA_CUT_FN int row(int place) const { return place < cut ? place : place + skip; }
  // which of the 64 rows from `first` on are visible
  PA_CUT_FN uint64_t visible(int first, int num_sink) const {
    return below(num_sink - first) | ~below(low - first);
  }
  static PA_CUT_FN uint64_t below(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
  }
};
// of a context of `len` rows whose window starts at row `low`
PA_CUT_FN WindowRange window_range(int len, int low, int num_sink, int log2_rpb) {
  WindowRange r;
  r.low = low;
  const int sinks = num_sink < len ? num_sink : len;
  const int first = (sinks + (1 << log2_rpb) - 1) >> log2_rpb;  // pieces with first tokens
  const int between = (low >> log2_rpb) - first;
  r.cut = first << log2_rpb;
  r.skip = (between > 0 ? between : 0) << log2_rpb;
  r.len = len - r.skip;
  return r;
}

namespace windowcut {

using namespace q4cut;

constexpr int kHeaderBytes = 256;  // of the workspace: the error word
constexpr int kCtasPerSm = 2;      // of the decode kernel

// The launch's cut and what it needs of the workspace: header, log-sum-exp partials, output
// partials, info words.
struct WindowPlan {
  int32_t chunks;
  int32_t slots;
  bool whole;
  size_t lse_offset, o_offset, info_offset, bytes;
};

// Cutting costs a second launch and a merge, about as much time as a CTA takes for so many
// units; a piece's own start and end about two.
constexpr int64_t kMergeUnits = 6;

PA_CUT_FN WindowPlan window_plan(int32_t sms, int32_t num_seqs, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t window, int32_t num_sink,
                                 int32_t max_context_len) {
  // a window of W rows and S first tokens touch at most W + S rows and what the pieces at
  // their ends hold besides
  const int64_t most = min64(static_cast<int64_t>(window) + num_sink + 2 * kUnit, max_context_len);
  const int64_t units = (most + kUnit - 1) / kUnit;
  WindowPlan w;
  int64_t chunks = static_cast<int64_t>(sms) * kCtasPerSm / num_kv_heads;
  chunks = max64(min64(chunks, kMaxChunks), 1);
  // Whole sequences where that takes no longer than an even cut with its merge, if the window
  // makes lengths alike (contexts of twice the window and more); else only short ones.
  // (64 sequences, window 2000, e4m3: 23 us whole, 31 cut; window 500: 9, 22)
  const int64_t rounds = (num_seqs + chunks - 1) / chunks;
  const int64_t piece = units + kPieceCost;
  const bool alike = max_context_len / 2 >= static_cast<int64_t>(window) + num_sink;
  w.whole = (alike && rounds * piece <= num_seqs * piece / chunks + kMergeUnits) ||
            units <= kMergeUnits;
  const int64_t cut = max64(min64(chunks, units * num_seqs), 1);
  if (cut == 1) w.whole = true;
  w.chunks = static_cast<int32_t>(w.whole ? max64(min64(chunks, num_seqs), 1) : cut);
  // The workspace is that of an even cut also where sequences stay whole: so it never shrinks as
  // num_seqs, window, num_sink or max_context_len grow, and one of the largest batch
  // serves all others.
  w.slots = static_cast<int32_t>(cut - 1 + min64(num_seqs, cut - 1));
  const size_t rows = static_cast<size_t>(num_q_heads) * w.slots;
  w.lse_offset = kHeaderBytes;
  w.o_offset = w.lse_offset + (rows * 4 + 255) / 256 * 256;
  w.info_offset = w.o_offset + rows * kPartialFloats * 4;
  w.bytes = w.info_offset + static_cast<size_t>(num_kv_heads) * num_seqs * 4;
  return w;
}

}  // namespace windowcut
}  // namespace pa_detail
