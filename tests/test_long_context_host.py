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
