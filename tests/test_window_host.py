"""Refusals of the sliding-window calls on a host without a GPU: every call below returns or
raises during the argument checks; none reaches a kernel launch."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import window as ow
from paged_kv_cache_309_gb300 import build as pabuild
from paged_kv_cache_309_gb300 import pa

P = ctypes.c_void_p
FAKE, FAKE_MIS = P(0x100000), P(0x100008)
INVALID, UNSUPPORTED, ALIGN = pa.PA_ERR_INVALID, pa.PA_ERR_UNSUPPORTED, pa.PA_ERR_ALIGN


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.library()


def _rope(lib, **kw):
    a = dict(qo=P(0x200000), q=FAKE, k=FAKE, v=FAKE, src=pa.PA_BF16, n=4, hq=16, h=8, d=128, qos=2048, qs=4096,
             ks=4096, vs=4096, cs=FAKE, pos=FAKE, most=100, rot=128, inter=0, kc=FAKE, vc=FAKE, cd=pa.PA_BF16, nb=4,
             bs=16, bst=16 * 1024, slot=FAKE, swa=None, swal=0, ksc=None, vsc=None)
    assert set(kw) <= set(a)
    return lib.pa_rope_and_cache(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(qo=None)), (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(v=None)),
    (INVALID, dict(cs=None)), (INVALID, dict(pos=None)), (INVALID, dict(kc=None)), (INVALID, dict(vc=None)),
    (INVALID, dict(slot=None)), (INVALID, dict(n=-1)), (INVALID, dict(hq=0)), (INVALID, dict(h=0)),
    (INVALID, dict(d=0)), (INVALID, dict(rot=0)), (INVALID, dict(rot=144)), (INVALID, dict(most=-1)),
    (INVALID, dict(inter=2)), (INVALID, dict(bs=0)), (INVALID, dict(nb=-1)), (INVALID, dict(ksc=FAKE)),
    (INVALID, dict(vsc=FAKE)), (INVALID, dict(swa=FAKE, swal=-1)), (INVALID, dict(qs=1024)),
    (INVALID, dict(qos=1024)), (INVALID, dict(ks=512)), (INVALID, dict(vs=512)), (INVALID, dict(bst=1024)),
    (INVALID, dict(qo=FAKE)),  # in place with another stride
    (UNSUPPORTED, dict(src=pa.PA_FP8_E4M3)), (UNSUPPORTED, dict(cd=pa.PA_Q4)), (UNSUPPORTED, dict(cd=9)),
    (UNSUPPORTED, dict(d=132)), (UNSUPPORTED, dict(d=520, rot=16)), (UNSUPPORTED, dict(rot=24)),
    (UNSUPPORTED, dict(rot=8)), (UNSUPPORTED, dict(n=2 ** 40)), (UNSUPPORTED, dict(hq=2 ** 30)),
    (UNSUPPORTED, dict(nb=2 ** 62)),
    (ALIGN, dict(qo=FAKE_MIS)), (ALIGN, dict(q=FAKE_MIS)), (ALIGN, dict(k=FAKE_MIS)), (ALIGN, dict(v=FAKE_MIS)),
    (ALIGN, dict(cs=FAKE_MIS)), (ALIGN, dict(kc=FAKE_MIS)), (ALIGN, dict(vc=FAKE_MIS)),
    (ALIGN, dict(pos=P(0x100004))), (ALIGN, dict(slot=P(0x100004))), (ALIGN, dict(swa=P(0x100004), swal=4)),
    (ALIGN, dict(qs=4100)), (ALIGN, dict(qos=4100)), (ALIGN, dict(ks=4100)), (ALIGN, dict(vs=4100)),
    (ALIGN, dict(bst=16 * 1024 + 4)), (ALIGN, dict(ksc=P(0x100002), vsc=FAKE)),
    (pa.PA_OK, dict(n=0, q=None, cs=None)),
])
def test_rope_and_cache_rejects(lib, want, kw):
    assert _rope(lib, **kw) == want


def _decode(lib, **kw):
    a = dict(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, cd=pa.PA_BF16, ksc=None, vsc=None, bt=FAKE, cl=FAKE, B=4, HQ=32,
             HKV=8, d=128, bs=16, mbps=8, nb=64, window=64, sink=4, scale=0.088, maxctx=128, ws=FAKE, wsb=1 << 24)
    assert set(kw) <= set(a)
    return lib.pa_paged_window_decode_attention(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(window=0)), (INVALID, dict(window=-1)), (INVALID, dict(sink=-1)), (INVALID, dict(q=None)),
    (INVALID, dict(cl=None)), (INVALID, dict(HQ=12)), (INVALID, dict(maxctx=-1)), (INVALID, dict(ksc=FAKE, vsc=FAKE)),
    (INVALID, dict(cd=pa.PA_FP8_E4M3, ksc=FAKE)), (INVALID, dict(scale=float("inf"))), (INVALID, dict(B=-1)),
    (UNSUPPORTED, dict(cd=pa.PA_Q4)), (UNSUPPORTED, dict(cd=pa.PA_FP16)), (UNSUPPORTED, dict(d=64)),
    (UNSUPPORTED, dict(HQ=24)), (UNSUPPORTED, dict(bs=12)), (UNSUPPORTED, dict(nb=1 << 28)),
    (ALIGN, dict(out=FAKE_MIS)), (ALIGN, dict(ws=P(0x100010))), (ALIGN, dict(bt=P(0x100002))),
    (ALIGN, dict(cd=pa.PA_FP8_E4M3, ksc=P(0x100002), vsc=FAKE)),
    (pa.PA_ERR_WORKSPACE, dict(ws=None)), (pa.PA_ERR_WORKSPACE, dict(wsb=255)),
])
def test_window_decode_rejects(lib, want, kw):
    assert _decode(lib, **kw) == want


def test_window_workspace_size(lib):
    size = lib.pa_paged_window_decode_workspace_size
    assert size(8, 32, 8, 128, 0, 4, 1000) == 0 and size(8, 32, 8, 128, 64, -1, 1000) == 0
    assert size(8, 32, 8, 128, 64, 4, -1) == 0 and size(0, 32, 8, 128, 64, 4, 1000) >= 256
    # a window that reaches past the context adds nothing, and a context past the window neither
    assert size(8, 32, 8, 128, 2 ** 31 - 1, 2 ** 31 - 1, 5000) == size(8, 32, 8, 128, 5000, 0, 5000)
    assert size(8, 32, 8, 128, 500, 4, 10 ** 6) == size(8, 32, 8, 128, 500, 4, 10 ** 9)
    with pytest.raises(ValueError):
        pa.pa_paged_window_decode_workspace_size(8, 32, 8, 128, 2 ** 32 + 64, 4, 1000)


def _prefill(lib, **kw):
    a = dict(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, cd=pa.PA_BF16, bt=FAKE, cu=FAKE, cl=FAKE, B=4, HQ=32, HKV=8, d=128,
             bs=16, mbps=8, nb=64, window=64, sink=4, scale=0.088, mql=64, total=256, err=FAKE)
    assert set(kw) <= set(a)
    return lib.pa_paged_window_prefill_attention(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("want,kw", [
    (pa.PA_OK, dict(B=0)), (pa.PA_OK, dict(mql=0)), (INVALID, dict(window=0)), (INVALID, dict(sink=-1)),
    (INVALID, dict(B=0, window=0)), (INVALID, dict(err=None)), (INVALID, dict(cu=None)), (INVALID, dict(HQ=12)),
    (INVALID, dict(mql=-1)), (UNSUPPORTED, dict(cd=pa.PA_FP8_E4M3)), (UNSUPPORTED, dict(d=64)),
    (UNSUPPORTED, dict(HQ=24)), (UNSUPPORTED, dict(bs=4)), (UNSUPPORTED, dict(mbps=1 << 27)), (INVALID, dict(total=-1)), (UNSUPPORTED, dict(total=1 << 31)),
    (pa.PA_OK, dict(total=0)),
    (ALIGN, dict(out=FAKE_MIS)), (ALIGN, dict(err=P(0x100002))), (ALIGN, dict(cu=P(0x100002))),
])
def test_window_prefill_rejects(lib, want, kw):
    assert _prefill(lib, **kw) == want


def test_binding_refuses_host_tensors(monkeypatch):
    def fail():
        raise AssertionError("the binding reached the library with a host tensor")
    monkeypatch.setattr(pa, "_load", fail)
    q, c = torch.zeros((2, 8, 128), dtype=torch.bfloat16), torch.zeros((4, 16, 4, 128), dtype=torch.bfloat16)
    i32, i64 = torch.zeros((2, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    k = q[:, :4]
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_rope_and_cache(q, q, k, k, c, c, torch.zeros((8, 128)), i64, i64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_paged_window_decode_attention(q, q, c, c, i32, i32[:, 0], 4, 1, 0.1, 16, i64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_paged_window_prefill_attention(q, q, c, c, i32, i32[:, 0], i32[:1, 0], 4, 1, 0.1, 2, i32[0])
    with pytest.raises(ValueError):
        pa.pa_paged_window_prefill_attention(q, q, c, c, i32, i32[:, 0], i32[:1, 0], 4, 1, 0.1, 2, None)


def _range(length, low, sink, rpb):
    """The rows that a window leaves as one range, as the kernels cut it."""
    first = (min(sink, length) + rpb - 1) // rpb
    cut, skip = first * rpb, max(0, low // rpb - first) * rpb
    return cut, skip, length - skip


def test_places_cover_what_is_seen():
    """Every visible row has one place, in order; the places are within the plan's bound."""
    rng = np.random.default_rng(0)
    for _ in range(3000):
        rpb = int(2 ** rng.integers(3, 7))
        length, window, sink = (int(x) for x in np.exp(rng.uniform(0, 7, 3)))
        sink -= 1
        low = max(0, length - window)
        cut, skip, places = _range(length, low, sink, rpb)
        rows = [p if p < cut else p + skip for p in range(places)]
        assert rows == sorted(set(rows)) and (not rows or rows[-1] == length - 1)
        assert set(ow.visible(length - 1, window, sink).tolist()) <= set(rows)
        assert places <= window + sink + 2 * 64


def test_window_prefill_refuses_outputs_over_its_queries(lib):
    """Rows beside values that are not finite are made from their queries a second time, after others
    are written: in place they would come out wrong."""
    size = 256 * 32 * 128 * 2
    q = 1 << 28
    for out in (q, q + size - 256, q - size + 256, q + 256):
        assert _prefill(lib, q=P(q), out=P(out)) == INVALID


def test_empty_batches_are_nothing_to_do(lib):
    """Tensors without an element have no address: a batch of no sequence and a prompt batch of no row
    pass with null pointers; sizes are checked all the same."""
    none = dict(out=None, q=None, bt=None, cl=None, ws=None, wsb=0)
    assert _decode(lib, B=0, **none) == pa.PA_OK
    assert _decode(lib, B=0, **none, cd=pa.PA_FP8_E4M3) == pa.PA_OK
    for kw in (dict(HQ=0), dict(nb=0), dict(window=0), dict(sink=-1), dict(maxctx=-1), dict(ksc=FAKE)):
        assert _decode(lib, **{**dict(B=0), **none, **kw}) == INVALID
    assert _prefill(lib, total=0, out=None, q=None) == pa.PA_OK
    assert _prefill(lib, total=0, out=None, q=None, B=0, bt=None, cl=None) == pa.PA_OK
    for kw in (dict(HKV=0), dict(mql=-1), dict(window=0), dict(nb=0)):
        assert _prefill(lib, **{**dict(total=0, out=None, q=None), **kw}) == INVALID
