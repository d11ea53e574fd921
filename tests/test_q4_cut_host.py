"""The 4-bit decode kernel's cut, from the very lines the kernel and its launch
compile (csrc/q4_cut.h, built here with the host compiler): every unit lies in
one chunk, a split sequence has one piece in each chunk of its span, no two
pieces share a partial slot, and partials and piece counts end inside the
workspace the library asks for."""
import ctypes
import shutil
import subprocess

import numpy as np
import pytest

from paged_kv_cache_309_gb300 import build as pabuild
from paged_kv_cache_309_gb300 import pa

SRC = r"""
#include "q4_cut.h"
using namespace pa_detail::q4cut;
extern "C" void cut_launch(int64_t resident, int64_t seqs, int64_t splits, int64_t heads,
                           int64_t group, int64_t* out) {
  const Launch l = launch_of(resident, seqs, splits, heads, group);
  out[0] = l.chunks; out[1] = l.slots; out[2] = l.whole; out[3] = l.info_float;
}
extern "C" int cut_units(int len) { return units_of_len(len); }
// Rows (chunk, sequence, first unit, end, chunk of its first unit, of its last, slot, info) of
// all pieces; the search of a chunk's begin is the kernel's, sequence after sequence.
extern "C" int64_t cut_pieces(const int32_t* lens, int32_t B, int32_t chunks, int32_t whole,
                              int64_t* out, int64_t room) {
  int64_t units = 0, count = 0;
  for (int b = 0; b < B; ++b) units += units_of_len(lens[b]);
  const int64_t total = total_cost(units, B), parts = parts_of(total, chunks);
  auto begin = [&](int64_t k) -> int64_t {
    if (k >= parts) return units;
    const int64_t x = chunk_begin_cost(k, total, parts);
    int64_t pre = 0;
    for (int b = 0; b < B; ++b) {
      const int n = units_of_len(lens[b]);
      if (begins_in(x, pre, n, b, whole)) return begin_unit(x, pre, b, whole);
      pre += n;
    }
    return units;
  };
  for (int c = 0; c < chunks; ++c) {
    const int64_t lo = begin(c), hi = begin(c + 1);
    int64_t pre = 0;
    for (int b = 0; b < B; ++b) {
      const int n = units_of_len(lens[b]);
      const int64_t from = max64(lo, pre), to = min64(hi, pre + n);
      if (from < to) {
        if (count == room) return -1;
        const int c0 = whole ? c : chunk_of(pre, b, total, (int)parts);
        const int c1 = whole ? c : chunk_of(pre + n - 1, b, total, (int)parts);
        const int64_t row[8] = {c, b, from, to, c0, c1, slot_of_piece(chunks, B, b, c0, c),
                                info_of(c0, c1)};
        for (int i = 0; i < 8; ++i) out[8 * count + i] = row[i];
        ++count;
      }
      pre += n;
    }
  }
  return count;
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("cut")
    (d / "cut.cpp").write_text(SRC)
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I", pabuild.CSRC,
                    str(d / "cut.cpp"), "-o", str(d / "cut.so")], check=True)
    lib = ctypes.CDLL(str(d / "cut.so"))
    I64 = ctypes.c_int64
    lib.cut_launch.argtypes = [I64] * 5 + [ctypes.c_void_p]
    lib.cut_pieces.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                               ctypes.c_void_p, I64]
    lib.cut_pieces.restype = I64
    return lib


def check(cut, lens, resident, heads, group, splits):
    """heads: kv heads; their number of rows of `info` is at most that."""
    lens = np.ascontiguousarray(np.maximum(lens, 0), np.int32)
    B = len(lens)
    got = np.zeros(4, np.int64)
    cut.cut_launch(resident, B, splits, heads, group, got.ctypes.data)
    chunks, slots, whole, info_float = got.tolist()
    assert 1 <= chunks <= 32767 and (whole == 1) == (splits == 1)
    if not whole:
        # partial rows of the workspace: splits per (sequence, query head), 128 floats each
        floats = B * splits * heads * group * 128
        assert slots * heads * group * 128 <= info_float
        assert info_float + heads * B <= floats
        assert slots * heads * group <= B * splits * heads * group  # their log-sum-exps
    n = (lens.astype(np.int64) + 63) // 64
    room = chunks + int((n > 0).sum()) + 1
    rows = np.zeros((room, 8), np.int64)
    count = cut.cut_pieces(lens.ctypes.data, B, chunks, whole, rows.ctypes.data, room)
    assert count >= 0  # at most one piece per sequence and one more per inner boundary
    rows = rows[:count]
    seen = np.zeros(int(n.sum()) + 1, np.int64)
    np.add.at(seen, rows[:, 2], 1)
    np.add.at(seen, rows[:, 3], -1)
    assert (np.cumsum(seen)[:-1] == 1).all()  # every unit in one piece
    used = set()
    for b in range(B):
        mine = rows[rows[:, 1] == b]
        if n[b] == 0:
            assert len(mine) == 0
            continue
        c0, c1 = mine[0, 4], mine[0, 5]
        assert mine[:, 0].tolist() == list(range(c0, c1 + 1)), (b, mine)
        if c0 == c1:
            assert (mine[:, 7] == 0).all()
            continue
        assert not whole
        info = int(mine[0, 7])
        assert 0 < info < 2 ** 31 and info >> 16 == c0 and info & 0xFFFF == len(mine)
        for s in mine[:, 6].tolist():
            assert 0 <= s < slots and s not in used
            used.add(s)


@pytest.mark.parametrize("heads", [1, 3, 8, 40])
def test_invariants(cut, heads):
    rng = np.random.default_rng(heads)
    for case in range(150):
        B = int(rng.integers(1, 130))
        top = int(rng.choice([1, 64, 65, 300, 4096, 30000]))
        lens = rng.integers(0, top + 1, B)
        if case % 5 == 0:
            lens[int(rng.integers(B))] = 60000
        splits = int(rng.choice([1, 2, 3, 10, 76, 1000]))
        check(cut, lens, int(rng.choice([8, 304, 456])) // heads, heads, int(rng.choice([1, 4, 16])),
              splits)


def test_batches_of_one_and_of_many(cut):
    for L in (1, 64, 65, 128, 9001, 131072, 1 << 30):
        for splits in (1, 2, 141, 1216):
            for resident in (1, 114, 456, 40000):
                check(cut, [L], resident, 4, 8, splits)
                check(cut, [L, 0, 1], resident, 8, 1, splits)
    check(cut, [1 << 30], 40000, 1, 1, 100000)  # more chunks than an `info` word counts
    for splits in (1, 2, 3):
        check(cut, [1] * 2000, 57, 8, 4, splits)
        check(cut, [0] * 50, 57, 8, 4, splits)
        check(cut, [4096] * 700, 57, 8, 4, splits)


def test_units(cut):
    assert [cut.cut_units(x) for x in (0, 1, 64, 65, 1 << 30)] == [0, 1, 1, 2, 1 << 24]


def test_inside_the_workspace_of_the_library(cut):
    """With the library's own plans: the bytes it asks for hold what the launch lays out."""
    pabuild.build()
    lib = pa.library()
    sms = 148  # where there is no device
    rng = np.random.default_rng(0)
    for _ in range(400):
        B, HKV = int(rng.integers(1, 300)), int(rng.choice([1, 2, 3, 4, 8, 40]))
        G = int(rng.choice([1, 2, 4, 8, 16]))
        mcl = int(np.exp(rng.uniform(0, np.log(200000))))
        splits, tps = pa.pa_paged_decode_plan(B, HKV, mcl, sms)
        nbytes = lib.pa_paged_decode_workspace_size(B, HKV * G, HKV, 128, mcl)
        heads_per_cta = 2 if HKV % 2 == 0 else 1
        resident = sms * (3 if G <= 8 else 2) // (HKV // heads_per_cta)
        out = np.zeros(4, np.int64)
        cut.cut_launch(resident, B, splits, HKV, G, out.ctypes.data)
        if splits > 1:
            pad = lambda x: -(-x // 256) * 256
            first = 256 + pad(B * HKV * 4) + pad(B * HKV * G * splits * 4)
            end = first + (int(out[3]) + HKV // heads_per_cta * B) * 4
            assert end <= nbytes, (B, HKV, G, mcl, splits)
            assert int(out[1]) * HKV * G * 4 <= pad(B * HKV * G * splits * 4)
        lens = rng.integers(0, min(mcl, splits * tps) + 1, B)
        check(cut, lens, resident, HKV, G, splits)
