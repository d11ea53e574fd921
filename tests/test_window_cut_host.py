"""The integer arithmetic of the sliding-window calls, from the very lines the kernels and their
launches compile (csrc/window_cut.h, built here with the host compiler): every row that a query
sees has one place and its bit in the masks, and whatever a decode batch is cut into ends inside
the workspace that the library asks for."""
import ctypes
import shutil
import subprocess

import numpy as np
import pytest

from oracle import window as ow
from paged_kv_cache_309_gb300 import build as pabuild
from paged_kv_cache_309_gb300 import pa
from tests.test_q4_cut_host import SRC as PIECES

SMS = 148  # where there is no device

SRC = PIECES + r"""
#include "window_cut.h"
using namespace pa_detail;
// rows of places 0 .. len - 1 and whether each is visible to some query, by masks of 64 rows of
// one piece as the loads make them; gives the number of places
extern "C" int places(int len, int low, int sink, int log2_rpb, int32_t* row, uint8_t* seen, int room) {
  const WindowRange r = window_range(len, low, sink, log2_rpb);
  if (r.len > room) return -1;
  for (int at = 0; at < r.len; at += 1 << log2_rpb) {
    const uint64_t bits = r.visible(r.row(at), sink);
    for (int i = 0; i < 1 << log2_rpb && at + i < r.len; ++i) {
      row[at + i] = r.row(at) + i;
      seen[at + i] = bits >> i & 1;
    }
  }
  return r.len;
}
extern "C" void plan(int32_t sms, int32_t B, int32_t HQ, int32_t H, int32_t window, int32_t sink, int32_t most,
                     int32_t e4m3, int64_t* out) {
  const auto w = windowcut::window_plan(sms, B, HQ, H, window, sink, most, e4m3);
  const int64_t row[7] = {w.chunks, w.slots, w.whole, (int64_t)w.lse_offset, (int64_t)w.o_offset,
                          (int64_t)w.info_offset, (int64_t)w.bytes};
  for (int i = 0; i < 7; ++i) out[i] = row[i];
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("window_cut")
    (d / "cut.cpp").write_text(SRC)
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I", pabuild.CSRC,
                    str(d / "cut.cpp"), "-o", str(d / "cut.so")], check=True)
    lib = ctypes.CDLL(str(d / "cut.so"))
    P, I32 = ctypes.c_void_p, ctypes.c_int32
    lib.places.argtypes = [I32] * 4 + [P, P, I32]
    lib.plan.argtypes = [I32] * 8 + [P]
    lib.cut_pieces.argtypes = [P, I32, I32, I32, P, ctypes.c_int64]
    lib.cut_pieces.restype = ctypes.c_int64
    return lib


def places(cut, length, low, sink, log2_rpb):
    row, seen = np.zeros(length + 1, np.int32), np.zeros(length + 1, np.uint8)
    n = cut.places(length, low, sink, log2_rpb, row.ctypes.data, seen.ctypes.data, length + 1)
    assert 0 <= n <= length
    return row[:n], seen[:n].astype(bool)


def plan(cut, *args, e4m3=False, sms=SMS):
    out = np.zeros(7, np.int64)
    cut.plan(sms, *args, e4m3, out.ctypes.data)
    return out.tolist()


def test_places_of_a_decode_query(cut):
    rng = np.random.default_rng(0)
    for _ in range(3000):
        log2_rpb = int(rng.integers(3, 7))
        length, window, sink = (int(x) for x in np.exp(rng.uniform(0, 7.5, 3)))
        sink -= 1
        row, seen = places(cut, length, max(0, length - window), sink, log2_rpb)
        assert (np.diff(row) > 0).all() and row[-1] == length - 1
        assert row[seen].tolist() == ow.visible(length - 1, window, sink).tolist()
        assert len(row) <= window + sink + 2 * 64  # what the plan counts with


def test_places_of_a_prompt_item(cut):
    """An item's rows share the places that its first row's window and its last row leave; what no
    row sees is not among the seen."""
    rng = np.random.default_rng(1)
    for _ in range(3000):
        log2_rpb, ntok = int(rng.integers(3, 7)), int(rng.integers(1, 257))
        first, window, sink = (int(x) for x in np.exp(rng.uniform(0, 7, 3)))
        first, sink = first - 1, sink - 1
        row, seen = places(cut, first + ntok, max(0, first - window + 1), sink, log2_rpb)
        assert (np.diff(row) > 0).all() and row[-1] == first + ntok - 1
        union = set(ow.visible(first, window, sink).tolist()) | set(range(first, first + ntok)) | set(range(min(sink, first + ntok)))
        assert row[seen].tolist() == sorted(union)


def sizes(rng):
    H, G = int(rng.choice([1, 2, 3, 4, 8, 40, 500])), int(rng.choice([1, 2, 4, 8, 16]))
    B = int(rng.choice([rng.integers(1, 100), rng.integers(1, 400), rng.integers(1, 5000)]))
    window, sink = int(np.exp(rng.uniform(0, 9))), int(rng.choice([0, 4, 64, 300]))
    most = int(np.exp(rng.uniform(0, 11)))
    return B, H * G, H, window, sink, most


def test_pieces_end_inside_the_workspace(cut):
    """Every partial row and piece count of a batch lies in its own part of the workspace."""
    pabuild.build()
    lib = pa.library()
    rng = np.random.default_rng(2)
    split = 0
    for _ in range(1500):
        B, HQ, H, window, sink, most = sizes(rng)
        chunks, slots, whole, lse, o, info, size = plan(cut, B, HQ, H, window, sink, most,
                                                         e4m3=bool(rng.integers(2)))
        assert 1 <= chunks <= 32767 and lse >= 256 and o % 256 == 0 and info % 4 == 0
        assert lse + HQ * slots * 4 <= o and o + HQ * slots * 512 <= info
        nbytes = lib.pa_paged_window_decode_workspace_size(B, HQ, H, 128, window, sink, most)
        assert size <= nbytes
        if not whole:
            assert info + H * B * 4 <= size
        if B > 400:
            continue
        lens = [len(places(cut, n, max(0, n - window), sink, 4)[0]) if n else 0
                for n in rng.integers(0, most + 1, min(B, 60))]
        lens = np.resize(np.array(lens, np.int32), B)
        n = (lens.astype(np.int64) + 63) // 64
        room = chunks + B + 1
        rows = np.zeros((room, 8), np.int64)
        count = cut.cut_pieces(lens.ctypes.data, B, chunks, whole, rows.ctypes.data, room)
        assert count >= 0
        rows = rows[:count]
        assert (rows[:, 3] - rows[:, 2]).sum() == n.sum()
        cuts = rows[rows[:, 7] != 0]
        assert not (whole and len(cuts))
        assert len(set(cuts[:, 6].tolist())) == len(cuts) and ((cuts[:, 6] >= 0) & (cuts[:, 6] < slots)).all()
        split += len(cuts) > 0
    assert split > 100


def test_a_workspace_of_a_larger_batch_serves_a_smaller_one():
    """The size never falls as sequences, window, first tokens or contexts grow."""
    pabuild.build()
    size = pa.library().pa_paged_window_decode_workspace_size
    rng = np.random.default_rng(3)
    for H, HQ in ((8, 32), (4, 32), (1, 1), (2, 32), (40, 160)):
        for window, most in ((4096, 32768), (500, 1500), (2000, 8192), (100, 400), (5000, 5000)):
            row = [size(B, HQ, H, 128, window, 4, most) for B in range(0, 400)]
            assert row == sorted(row)
            row = [size(36, HQ, H, 128, window, 4, n) for n in range(0, 20000, 50)]
            assert row == sorted(row)
            row = [size(36, HQ, H, 128, n, 4, most) for n in range(1, 10000, 33)]
            assert row == sorted(row)
    for _ in range(2000):
        B, HQ, H, window, sink, most = sizes(rng)
        less = [int(rng.integers(1, x + 1)) for x in (B, window, sink + 1, most)]
        assert size(less[0], HQ, H, 128, less[1], less[2] - 1, less[3]) <= size(B, HQ, H, 128, window, sink, most)


@pytest.mark.parametrize("e4m3", [False, True])
def test_the_choice_does_not_flip_back(cut, e4m3):
    """Within one wave, a batch that is cut stays cut as sequences are removed, for every window."""
    both = 0
    for H, HQ in ((8, 32), (8, 16), (4, 32), (2, 16), (1, 8), (1, 16), (16, 16)):
        for window in (300, 500, 1000, 1024, 2000, 4096, 16384):
            whole = [plan(cut, B, HQ, H, window, 4, 4 * window, e4m3=e4m3, sms=152)[2]
                     for B in range(1, 304 // H + 1)]
            assert whole == sorted(whole), (H, window)
            both += 0 < sum(whole) < len(whole)
    assert both > 20


@pytest.mark.parametrize("e4m3,H,HQ,window,sequences", [
    # (us whole and cut of these batches stand at the choice; the times differ by a tenth and more)
    (False, 8, 16, 1000, {8: 0, 36: 1, 40: 0, 48: 0}),
    (True, 4, 32, 2000, {16: 0, 60: 1, 63: 1, 64: 1, 76: 1, 80: 0, 96: 0}),
    (True, 1, 16, 300, {56: 1, 72: 1, 128: 1}),
    (True, 8, 16, 1000, {4: 0, 28: 1, 36: 1, 40: 0}),
    (False, 8, 16, 16384, {1: 0, 8: 0, 24: 0, 48: 0, 80: 0}),
    (True, 4, 32, 16384, {56: 0, 60: 0}),  # (of uneven contexts)
])
def test_the_choice_is_the_faster_way(cut, e4m3, H, HQ, window, sequences):
    for B, want in sequences.items():
        assert plan(cut, B, HQ, H, window, 4, 3 * (window + 4), e4m3=e4m3, sms=152)[2] == want, B
