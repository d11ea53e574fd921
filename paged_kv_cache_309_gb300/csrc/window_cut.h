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

// Whether sequences stay whole, by the time of either way in ns.  A CTA takes kUnitTime for a
// unit, all of them together no less than kUnitMemory for each unit of each kv head; a cut adds a
// second launch and the merge of its partial rows.  Fitted to both ways of 4776 batches, timed in a
// copy of the launch that is told which (1 .. 256 sequences, 1 .. 16 kv heads, 1 .. 16 query heads
// each, windows 300 .. 16384, contexts of two to three windows or of any length up to three; rms
// 6 %): the choice costs 0.4 % over the better way in the mean, more than a tenth in 0.8 % of
// them.  Both sides, us whole / cut:
//  * bf16, 8 kv heads, window 1000: 8 sequences 20.1 / 13.4, 20 21.4 / 21.8, 36 27.0 / 31.6,
//    40 (a second round) 46.0 / 34.2;
//  * e4m3, 4 kv heads, window 2000: 16 sequences 20.6 / 16.1, 48 24.3 / 25.1, 63 25.9 / 30.9,
//    76 28.7 / 31.5, 80 49.4 / 35.2;
//  * e4m3, 1 kv head, window 300: 72 sequences 7.5 / 15.8; bf16, 8 kv heads, window 16384: 8
//    sequences 260 / 90.
struct Times {
  double unit, memory;
};
constexpr Times kBf16Times{1000.0, 5.0}, kE4m3Times{550.0, 2.6};
constexpr double kMergeTime = 4800.0, kPartialTime = 0.7;
constexpr int kShortUnits = 6;  // so few are never cut (one sequence of them: 6 us whole, 8 cut)

// chunks: of a whole wave; cut: of an even cut.  units: of the longest sequence, which the window
// makes the ordinary one.  Where some are shorter after all, whole sequences are uneven, a second
// round of them more so (window 16384, 64 of 21 .. 49152 tokens: 697 / 513): what that can
// cost, a sequence's time, is held against what a cut costs.
PA_CUT_FN bool stay_whole(int64_t chunks, int64_t cut, int64_t num_seqs, int64_t q_heads,
                          int64_t kv_heads, int64_t units, bool e4m3) {
  const Times t = e4m3 ? kE4m3Times : kBf16Times;
  const double one = units * t.unit, all = static_cast<double>(kv_heads) * units * t.memory;
  auto longer = [](double a, double b) { return a > b ? a : b; };
  const int64_t full = num_seqs / chunks, rest = num_seqs % chunks;
  const double whole =
      full * longer(one, chunks * all) + (rest > 0 ? longer(one, rest * all) : 0.0);
  const double merge =
      kMergeTime + kPartialTime * q_heads * static_cast<double>(cut + min64(num_seqs, cut));
  const double even = longer(num_seqs * one / cut, num_seqs * all) + merge;
  return whole <= even && one <= (num_seqs <= chunks ? 5.0 : 1.5) * merge;
}

PA_CUT_FN WindowPlan window_plan(int32_t sms, int32_t num_seqs, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t window, int32_t num_sink,
                                 int32_t max_context_len, bool e4m3) {
  // a window of W rows and S first tokens touch at most W + S rows and what the pieces at
  // their ends hold besides
  const int64_t most = min64(static_cast<int64_t>(window) + num_sink + 2 * kUnit, max_context_len);
  const int64_t units = (most + kUnit - 1) / kUnit;
  WindowPlan w;
  int64_t chunks = static_cast<int64_t>(sms) * kCtasPerSm / num_kv_heads;
  chunks = max64(min64(chunks, kMaxChunks), 1);
  const int64_t cut = max64(min64(chunks, units * num_seqs), 1);
  // (contexts of less than twice the window: lengths differ, and an even cut wins)
  const bool alike = max_context_len / 2 >= static_cast<int64_t>(window) + num_sink;
  w.whole = units <= kShortUnits ||
            (alike && stay_whole(chunks, cut, num_seqs, num_q_heads, num_kv_heads, units, e4m3));
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
