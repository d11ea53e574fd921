"""Host side of the long-context cache operators, without a GPU: the C ABI
refuses bad arguments before anything is launched, the binding refuses what
the kernels cannot address, and the oracle's forms hold on small cases."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import long_context as lc
from paged_kv_cache_309_gb300 import build as pabuild
from paged_kv_cache_309_gb300 import pa

P = ctypes.c_void_p
FAKE = P(0x100000)          # 16-byte aligned, never dereferenced
FAKE_MIS = P(0x100008)


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.library()


# ------------------------------------------------------------- the oracle --
def test_oracle_rows_hold_their_bounds():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 96)).astype(np.float32)
    back = lc.q4_restore(lc.q4_quantise(x))
    g, b = x.reshape(50, 3, 32), back.reshape(50, 3, 32)
    span = g.max(-1) - g.min(-1)
    # half a step, the scale's rounding (15 codes x 2^-11 of a step) and the minimum's
    bound = span / 30 * (1 + 2.0 ** -6) + np.abs(g).max(-1) * 2.0 ** -11
    assert (np.abs(g - b).max(-1) <= bound).all()


def test_oracle_row_layout_by_hand():
    x = np.zeros(32, np.float32)
    x[:4] = [0., 15., 30., 7.]  # m = 0, s = 2: codes 0, 7.5 -> 8 (even), 15, 3.5 -> 4 (even)
    row = lc.q4_quantise(x)
    assert row.shape == (20,)
    assert row[0] == 0x80 and row[1] == 0x4F and (row[2:16] == 0).all()
    assert row[16:].view(np.float16).tolist() == [2.0, 0.0]
    assert lc.q4_restore(row)[:4].tolist() == [0., 16., 30., 8.]


def test_oracle_nan_group():
    x = np.ones((2, 64), np.float32)
    x[0, 5] = np.nan
    x[1, 40] = -np.inf
    back = lc.q4_restore(lc.q4_quantise(x))
    assert np.isnan(back[0, :32]).all() and (back[0, 32:] == 1).all()
    assert (back[1, :32] == 1).all() and np.isnan(back[1, 32:]).all()


# ------------------------------------------------------ 4-bit cache, C ABI --
def _q4(lib, name="pa_reshape_and_cache_q4", **kw):
    a = dict(key=FAKE, value=FAKE, dt=pa.PA_BF16, n=4, h=8, d=128, ks=1024, vs=1024, kc=FAKE,
             vc=FAKE, nb=4, bs=16, bstride=16 * 640, slot=FAKE, swa=None, swa_len=0)
    a.update(kw)
    args = [a["key"], a["value"], a["dt"], a["n"], a["h"], a["d"], a["ks"], a["vs"], a["kc"],
            a["vc"], a["nb"], a["bs"], a["bstride"], a["slot"]]
    if name == "pa_reshape_and_cache_q4":
        args += [a["swa"], a["swa_len"]]
    return getattr(lib, name)(*args, None)


@pytest.mark.parametrize("name", ["pa_reshape_and_cache_q4", "pa_gather_cache_q4"])
def test_q4_cache_rejects(lib, name):
    rc = lambda **kw: _q4(lib, name, **kw)
    assert rc(n=0) == pa.PA_OK and rc(n=0, key=None) == pa.PA_OK
    for bad in (dict(key=None), dict(kc=None), dict(slot=None), dict(value=None), dict(vc=None),
                dict(n=-1), dict(h=0), dict(d=0), dict(bs=0), dict(nb=-1), dict(ks=512),
                dict(vs=512), dict(bstride=640)):
        assert rc(**bad) == pa.PA_ERR_INVALID, bad
    for bad in (dict(dt=pa.PA_FP8_E4M3), dict(dt=pa.PA_Q4), dict(dt=9), dict(d=120), dict(d=16)):
        assert rc(**bad) == pa.PA_ERR_UNSUPPORTED, bad
    for bad in (dict(ks=1028), dict(vs=1028), dict(bstride=16 * 640 + 2), dict(key=FAKE_MIS),
                dict(value=FAKE_MIS), dict(kc=FAKE_MIS), dict(vc=FAKE_MIS)):
        assert rc(**bad) == pa.PA_ERR_ALIGN, bad


def test_q4_write_rejects_window_length(lib):
    assert _q4(lib, swa=FAKE, swa_len=-1) == pa.PA_ERR_INVALID


def test_q4_dtype_is_refused_where_a_call_does_not_name_it(lib):
    assert lib.pa_reshape_and_cache(FAKE, FAKE, pa.PA_BF16, 4, 8, 128, 1024, 1024, FAKE, FAKE,
                                    pa.PA_Q4, 4, 16, 16 * 1024, FAKE, None, 0, None, None,
                                    None) == pa.PA_ERR_UNSUPPORTED
    assert lib.pa_paged_decode_attention(FAKE, FAKE, FAKE, FAKE, pa.PA_Q4, FAKE, FAKE, 4, 32, 8,
                                         128, 16, 8, 64, 0.1, 128, FAKE, 1 << 30,
                                         None) == pa.PA_ERR_UNSUPPORTED


# ----------------------------------------------------------- the binding --
def test_q4_row_bytes():
    assert pa.q4_row_bytes(128) == 80 and pa.q4_row_bytes(576) == 360
    for d in (0, -32, 100):
        with pytest.raises(ValueError):
            pa.q4_row_bytes(d)


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    c = torch.zeros(4, 16, 2, 80, dtype=torch.uint8)
    s = torch.zeros(4, dtype=torch.int64)
    for fn in (pa.pa_reshape_and_cache_q4, pa.pa_gather_cache_q4):
        with pytest.raises(ValueError, match="CUDA tensor"):
            fn(x, x, c, c, s)


def test_binding_refuses_wrong_shapes(monkeypatch):
    """The shape checks themselves, with the device check out of the way."""
    monkeypatch.setattr(pa, "_on_device", lambda **kw: None)
    monkeypatch.setattr(pa, "_load", lambda: pytest.fail("reached the library"))
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    c = torch.zeros(4, 16, 2, 80, dtype=torch.uint8)
    s = torch.zeros(4, dtype=torch.int64)
    for fn in (pa.pa_reshape_and_cache_q4, pa.pa_gather_cache_q4):
        for bad in ((x, x[:3], c, c, s), (x, x.half(), c, c, s), (x, None, c, c, s),
                    (x, x, c[..., :79], c, s), (x, x, c.char(), c.char(), s), (x, x, c, c[:3], s),
                    (x, x, c, c, s.int()), (x, x, c, c, s[:3]), (x.transpose(0, 1), x, c, c, s),
                    (x, x, c.transpose(1, 2), c, s), (x, x, c, c, torch.zeros(8, dtype=torch.int64)[::2])):
            with pytest.raises(ValueError):
                fn(*bad)


# ------------------------------------------------------- decode over 4 bits --
def _dec(lib, **kw):
    a = dict(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, cl=FAKE, B=4, HQ=32, HKV=8, d=128, bs=16,
             mbps=8, nb=64, scale=0.088, maxctx=128, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return lib.pa_paged_decode_attention_q4(
        a["out"], a["q"], a["kc"], a["vc"], a["bt"], a["cl"], a["B"], a["HQ"], a["HKV"], a["d"],
        a["bs"], a["mbps"], a["nb"], a["scale"], a["maxctx"], a["ws"], a["wsb"], None)


def test_decode_q4_rejects(lib):
    assert _dec(lib, B=0) == pa.PA_OK
    for bad in (dict(out=None), dict(q=None), dict(kc=None), dict(vc=None), dict(bt=None),
                dict(cl=None), dict(B=-1), dict(HQ=12), dict(HKV=0), dict(nb=0), dict(mbps=0),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(maxctx=-1)):
        assert _dec(lib, **bad) == pa.PA_ERR_INVALID, bad
    for bad in (dict(d=64), dict(HQ=24), dict(HQ=256), dict(bs=4), dict(bs=24), dict(bs=512),
                dict(nb=1 << 28), dict(B=65536)):
        assert _dec(lib, **bad) == pa.PA_ERR_UNSUPPORTED, bad
    for bad in (dict(out=FAKE_MIS), dict(q=FAKE_MIS), dict(kc=FAKE_MIS), dict(vc=FAKE_MIS),
                dict(ws=P(0x100010))):
        assert _dec(lib, **bad) == pa.PA_ERR_ALIGN, bad
    for bad in (dict(ws=None), dict(wsb=16)):
        assert _dec(lib, **bad) == pa.PA_ERR_WORKSPACE, bad


def _decode_tensors(row=80, dtype=torch.uint8):
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    c = torch.zeros(4, 16, 4, row, dtype=dtype)
    return dict(out=q.clone(), q=q, k_cache=c, v_cache=c.clone(),
                block_tables=torch.zeros(2, 3, dtype=torch.int32),
                context_lens=torch.zeros(2, dtype=torch.int32), scale=0.1, max_context_len=16,
                workspace=torch.zeros(256, dtype=torch.uint8))


def _bad_decode_tensors(good):
    q, c = good["q"], good["k_cache"]
    return [dict(q=q.float()), dict(out=q.half()), dict(out=q[:1]), dict(v_cache=c[:3]),
            dict(v_cache=c.to(torch.int16)), dict(k_cache=c[..., :79], v_cache=c[..., :79]),
            dict(block_tables=torch.zeros(2, 3, dtype=torch.int64)),
            dict(block_tables=torch.zeros(3, 3, dtype=torch.int32)),
            dict(context_lens=torch.zeros(3, dtype=torch.int32)),
            dict(context_lens=torch.zeros(2, dtype=torch.int64)),
            dict(k_cache=c.transpose(1, 2)), dict(q=q.transpose(0, 1))]


def test_decode_q4_binding_refusals(monkeypatch):
    good = _decode_tensors()
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_paged_decode_attention_q4(**good)
    monkeypatch.setattr(pa, "_on_device", lambda **kw: None)
    monkeypatch.setattr(pa, "_load", lambda: pytest.fail("reached the library"))
    bf16 = torch.zeros(4, 16, 4, 128, dtype=torch.bfloat16)
    for bad in _bad_decode_tensors(good) + [dict(k_cache=bf16, v_cache=bf16)]:
        with pytest.raises(ValueError):
            pa.pa_paged_decode_attention_q4(**{**good, **bad})


# ------------------------------------------------------- accumulated weights --
def _scored(lib, **kw):
    a = dict(out=FAKE, so=FAKE, si=FAKE, T=128, new=1, q=FAKE, kc=FAKE, vc=FAKE, cd=pa.PA_BF16,
             ks=None, vs=None, bt=FAKE, cl=FAKE, B=4, HQ=32, HKV=8, d=128, bs=16, mbps=8, nb=64,
             scale=0.088, maxctx=128, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return lib.pa_paged_decode_attention_scored(
        a["out"], a["so"], a["si"], a["T"], a["new"], a["q"], a["kc"], a["vc"], a["cd"], a["ks"],
        a["vs"], a["bt"], a["cl"], a["B"], a["HQ"], a["HKV"], a["d"], a["bs"], a["mbps"], a["nb"],
        a["scale"], a["maxctx"], a["ws"], a["wsb"], None)


def test_scored_rejects(lib):
    for cd in (pa.PA_BF16, pa.PA_FP8_E4M3, pa.PA_Q4):
        assert _scored(lib, B=0, cd=cd) == pa.PA_OK
    for bad in (dict(so=None), dict(si=None), dict(T=0), dict(T=-1), dict(new=-1), dict(ks=FAKE),
                dict(ks=FAKE, vs=FAKE), dict(ks=FAKE, vs=FAKE, cd=pa.PA_Q4), dict(q=None),
                dict(HQ=12), dict(so=P(0x100000 + 64)), dict(si=P(0x100000 + 4 * 8 * 128 * 4 - 4))):
        assert _scored(lib, **bad) == pa.PA_ERR_INVALID, bad
    for bad in (dict(cd=pa.PA_FP16), dict(cd=pa.PA_FP32), dict(cd=9), dict(d=64), dict(bs=12),
                dict(HQ=24), dict(B=65536, wsb=1 << 50), dict(T=(1 << 30) + 1)):
        assert _scored(lib, **bad) == pa.PA_ERR_UNSUPPORTED, bad
    for bad in (dict(so=P(0x100002), si=P(0x100002)), dict(out=FAKE_MIS), dict(ws=P(0x100010))):
        assert _scored(lib, **bad) == pa.PA_ERR_ALIGN, bad
    # the decode workspace alone is too small
    small = lib.pa_paged_decode_workspace_size(4, 32, 8, 128, 128)
    assert _scored(lib, wsb=small) == pa.PA_ERR_WORKSPACE
    need = lib.pa_paged_decode_scored_workspace_size(4, 32, 8, 128, 128)
    assert need >= small + 4 * 32 * 128 * 4
    assert _scored(lib, wsb=need - 1) == pa.PA_ERR_WORKSPACE
    assert lib.pa_paged_decode_scored_workspace_size(-1, 32, 8, 128, 128) == 0
    assert lib.pa_paged_decode_scored_workspace_size(4, 32, 0, 128, 128) == 0


def test_scored_binding_refusals(monkeypatch):
    sums = torch.zeros(2, 4, 30)
    good = dict(_decode_tensors(128, torch.bfloat16), sums_out=sums, sums=sums, num_new=1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_paged_decode_attention_scored(**good)
    monkeypatch.setattr(pa, "_on_device", lambda **kw: None)
    monkeypatch.setattr(pa, "_load", lambda: pytest.fail("reached the library"))
    one = torch.zeros(1)
    for bad in _bad_decode_tensors(good) + [
            dict(sums=sums.double(), sums_out=sums.double()), dict(sums=sums[:, :2]),
            dict(sums_out=sums[:, :, :20].contiguous()), dict(sums=sums.transpose(1, 2)),
            dict(num_new=-1), dict(k_scale=one), dict(k_scale=one, v_scale=one)]:
        with pytest.raises(ValueError):
            pa.pa_paged_decode_attention_scored(**{**good, **bad})


# ------------------------------------------------------------------ eviction --
def test_oracle_selection_by_hand():
    nan = np.nan
    sums = np.array([[[5., 1., 3., 3., nan, 3., 0., 9.]]], np.float32)
    keep, new = lc.evict_select(sums, [8], 4, 0, 0)
    assert keep.tolist() == [[[0, 2, 3, 7]]] and new.tolist() == [4]
    keep, _ = lc.evict_select(sums, [8], 4, 2, 1)
    assert keep.tolist() == [[[0, 1, 2, 7]]]
    keep, new = lc.evict_select(sums, [3], 4, 1, 1)
    assert keep.tolist() == [[[0, 1, 2, -1]]] and new.tolist() == [3]


def _select(lib, **kw):
    a = dict(keep=FAKE, new=FAKE, so=P(0x900000), si=P(0x300000), cl=P(0x200000), B=4, H=8, T=128,
             budget=64, sink=4, recent=16)
    a.update(kw)
    return lib.pa_evict_select(a["keep"], a["new"], a["so"], a["si"], a["cl"], a["B"], a["H"],
                               a["T"], a["budget"], a["sink"], a["recent"], None)


def test_select_rejects(lib):
    assert _select(lib, B=0) == pa.PA_OK
    for bad in (dict(keep=None), dict(new=None), dict(si=None), dict(cl=None), dict(cl=FAKE),
                dict(B=-1), dict(H=0), dict(T=0), dict(budget=0), dict(sink=-1), dict(recent=-1),
                dict(sink=60), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1),
                dict(so=P(0x300000 + 4)), dict(so=P(0x300000 - 4))):
        assert _select(lib, **bad) == pa.PA_ERR_INVALID, bad
    for bad in (dict(B=1 << 24), dict(T=(1 << 30) + 1), dict(budget=(1 << 30) + 1)):
        assert _select(lib, **bad) == pa.PA_ERR_UNSUPPORTED, bad
    for n in ("keep", "new", "so", "si", "cl"):
        assert _select(lib, **{n: P(0x100002)}) == pa.PA_ERR_ALIGN, n


def _compact(lib, **kw):
    a = dict(k=FAKE, v=FAKE, row=256, keep=FAKE, lens=FAKE, n=64, src=P(0x200000), sm=8,
             dst=P(0x300000), dm=4, B=4, H=8, bs=16, nb=64)
    a.update(kw)
    return lib.pa_cache_compact(a["k"], a["v"], a["row"], a["keep"], a["lens"], a["n"], a["src"],
                                a["sm"], a["dst"], a["dm"], a["B"], a["H"], a["bs"], a["nb"], None)


def test_compact_rejects(lib):
    for ok in (dict(B=0), dict(n=0), dict(nb=0), dict(B=0, k=None)):
        assert _compact(lib, **ok) == pa.PA_OK, ok
    for bad in (dict(k=None), dict(keep=None), dict(lens=None), dict(src=None), dict(dst=None),
                dict(row=0), dict(n=-1), dict(sm=0), dict(dm=0), dict(B=-1), dict(H=0), dict(bs=0),
                dict(nb=-1), dict(src=FAKE, dst=FAKE)):
        assert _compact(lib, **bad) == pa.PA_ERR_INVALID, bad
    for bad in (dict(B=65536), dict(H=65536), dict(nb=1 << 27), dict(n=(1 << 30) + 1)):
        assert _compact(lib, **bad) == pa.PA_ERR_UNSUPPORTED, bad
    for bad in (dict(row=72), dict(k=FAKE_MIS), dict(v=FAKE_MIS), dict(keep=P(0x100002)),
                dict(src=P(0x100002))):
        assert _compact(lib, **bad) == pa.PA_ERR_ALIGN, bad


def test_eviction_binding_refusals(monkeypatch):
    sums = torch.zeros(2, 4, 30)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    sel = dict(keep=i32(2, 4, 10), new_lens=i32(2), sums_out=sums.clone(), sums=sums,
               context_lens=i32(2), budget=10, num_sink=1, num_recent=2)
    c = torch.zeros(6, 16, 4, 80, dtype=torch.uint8)
    com = dict(k_cache=c, v_cache=c.clone(), keep=i32(2, 4, 10), keep_lens=i32(2),
               src_block_tables=i32(2, 3), dst_block_tables=i32(2, 2))
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_evict_select(**sel)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_cache_compact(**com)
    monkeypatch.setattr(pa, "_on_device", lambda **kw: None)
    monkeypatch.setattr(pa, "_load", lambda: pytest.fail("reached the library"))
    for bad in (dict(budget=11), dict(keep=i32(2, 4, 10).long()), dict(keep=i32(2, 10)),
                dict(keep=i32(2, 10, 4).transpose(1, 2)), dict(sums=sums.half()),
                dict(sums_out=sums[:, :, :20].contiguous()), dict(sums=sums[:1]), dict(new_lens=i32(3)),
                dict(context_lens=i32(2).long()), dict(context_lens=i32(4)[::2])):
        with pytest.raises(ValueError):
            pa.pa_evict_select(**{**sel, **bad})
    for bad in (dict(v_cache=c[:5]), dict(v_cache=c.char()), dict(k_cache=c.transpose(1, 2)),
                dict(keep=i32(2, 3, 10)), dict(keep=i32(2, 4, 10).long()), dict(keep_lens=i32(3)),
                dict(src_block_tables=i32(3, 3)), dict(dst_block_tables=i32(2, 2).long()),
                dict(src_block_tables=i32(3, 2).T), dict(keep_lens=i32(2).long())):
        with pytest.raises(ValueError):
            pa.pa_cache_compact(**{**com, **bad})


# ------------------------------------------- integers past 32 bits do not wrap --
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 64, -2 ** 31 - 1])
def test_binding_refuses_integers_past_32_bits(monkeypatch, value):
    monkeypatch.setattr(pa, "_on_device", lambda **kw: None)
    monkeypatch.setattr(pa, "_load", lambda: pytest.fail("reached the library"))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    sums = torch.zeros(2, 4, 30)
    sel = dict(keep=i32(2, 4, 10), new_lens=i32(2), sums_out=None, sums=sums,
               context_lens=i32(2), budget=10, num_sink=1, num_recent=2)
    for name in ("num_sink", "num_recent"):
        with pytest.raises(ValueError, match=name):
            pa.pa_evict_select(**{**sel, name: value})
    with pytest.raises(ValueError, match="max_context_len"):
        pa.pa_paged_decode_attention_q4(**{**_decode_tensors(), "max_context_len": value})
    with pytest.raises(ValueError, match="max_context_len"):
        pa.pa_paged_decode_attention_scored(
            **{**_decode_tensors(128, torch.bfloat16), "sums_out": sums, "sums": sums,
               "num_new": 1, "max_context_len": value})
    with pytest.raises(ValueError, match="max_context_len"):
        pa.pa_paged_decode_scored_workspace_size(2, 8, 4, 128, value)
