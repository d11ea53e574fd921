"""pa_evict_select_paged without a GPU: its refusals, and the oracle's rule."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import long_context as lc
from paged_kv_cache_309_gb300 import build as pabuild
from paged_kv_cache_309_gb300 import pa

P = ctypes.c_void_p
FAKE = P(0x100000)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.library()


def _select(lib, **kw):
    a = dict(keep=FAKE, new=FAKE, so=P(0x900000), si=P(0x300000), cl=P(0x200000), bt=FAKE, B=4, H=8,
             T=128, budget=64, sink=4, recent=16, bs=16, mb=8, nb=64)
    a.update(kw)
    return lib.pa_evict_select_paged(a["keep"], a["new"], a["so"], a["si"], a["cl"], a["bt"], a["B"],
                                     a["H"], a["T"], a["budget"], a["sink"], a["recent"], a["bs"],
                                     a["mb"], a["nb"], None)


def test_rejects(lib):
    assert _select(lib, B=0) == pa.PA_OK and _select(lib, B=0, bt=None) == pa.PA_OK
    for bad in (dict(keep=None), dict(new=None), dict(si=None), dict(cl=None), dict(cl=FAKE),
                dict(bt=None), dict(B=-1), dict(H=0), dict(T=0), dict(budget=0), dict(sink=-1),
                dict(recent=-1), dict(sink=60), dict(so=P(0x300000 + 4)), dict(bs=0), dict(bs=-16),
                dict(mb=0), dict(nb=-1)):
        assert _select(lib, **bad) == pa.PA_ERR_INVALID, bad
    for bad in (dict(B=1 << 24), dict(T=(1 << 30) + 1), dict(budget=(1 << 30) + 1)):
        assert _select(lib, **bad) == pa.PA_ERR_UNSUPPORTED, bad
    for n in ("keep", "new", "so", "si", "cl", "bt"):
        assert _select(lib, **{n: P(0x100002)}) == pa.PA_ERR_ALIGN, n


def test_binding_refusals(monkeypatch):
    sums = torch.zeros(2, 4, 30)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    good = dict(keep=i32(2, 4, 10), new_lens=i32(2), sums_out=sums.clone(), sums=sums,
                context_lens=i32(2), block_tables=i32(2, 3), budget=10, num_sink=1, num_recent=2,
                block_size=16, num_blocks=6)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_evict_select_paged(**good)
    monkeypatch.setattr(pa, "_on_device", lambda **kw: None)
    monkeypatch.setattr(pa, "_load", lambda: pytest.fail("reached the library"))
    for bad in (dict(budget=11), dict(keep=i32(2, 10)), dict(sums=sums.half()), dict(sums=sums[:1]),
                dict(new_lens=i32(3)), dict(context_lens=i32(4)[::2]), dict(block_tables=i32(3, 3)),
                dict(block_tables=i32(6)), dict(block_tables=i32(2, 3).long()),
                dict(block_tables=i32(3, 2).T), dict(num_sink=2 ** 31), dict(num_recent=2 ** 32),
                dict(block_size=2 ** 32 + 16), dict(num_blocks=2 ** 63), dict(num_blocks=-1)):
        with pytest.raises(ValueError):
            pa.pa_evict_select_paged(**{**good, **bad})


def test_oracle_by_hand():
    sums = np.array([[[5., 1., 3., 3., 9., 9., 0., 2.]]], np.float32)
    table = np.array([[2, 0, -1, 1]], np.int32)  # blocks of two: tokens 4 and 5 have no row
    keep, new = lc.evict_select(sums, [8], 4, 0, 0, table, 2, 3)
    assert keep.tolist() == [[[0, 2, 3, 7]]] and new.tolist() == [4]
    keep, new = lc.evict_select(sums, [8], 7, 0, 4, table, 2, 3)
    assert keep.tolist() == [[[0, 1, 2, 3, 6, 7, -1]]] and new.tolist() == [6]
    keep, new = lc.evict_select(sums, [8], 2, 0, 0, table, 2, 2)  # block 2 is not in the pool
    assert keep.tolist() == [[[2, 3]]] and new.tolist() == [2]
    keep, new = lc.evict_select(sums, [8], 3, 1, 1, table[:, :1], 2, 3)
    assert keep.tolist() == [[[0, 1, -1]]] and new.tolist() == [2]
