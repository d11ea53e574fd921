"""GPU parity of decode attention over a 4-bit cache against the oracle.

The oracle attends in double over the values that the rows stand for.  Bounds,
with p the weights (they sum to 1), v the values, s c their code parts:
  output rounding to bf16                 2^-8 |out|
  weights rounded to fp16                 2^-11 sum p |v|
  s c rounded to fp16                     2^-11 sum p s c
  fp32 sums and scores                    2^-16 max |v| (scores below 2^6 off by 2^-18 at most)
so |got - ref| <= 2^-8 |ref| + 2^-11 (max |v| + max s c) + 2^-16 max |v|.
Those errors are independent from token to token, so for random data the
2-norm of the difference is below 2^-8 / sqrt(3) of the outputs' for the last
rounding plus 2^-11 / sqrt(3) (rms |v| + rms s c) / rms v for the others:
3.4e-3 of it for normal values (rms s c about 2.8 sigma); 4e-3 is asked.
"""
import numpy as np
import pytest
import torch

from oracle import long_context as lc
from paged_kv_cache_309_gb300 import pa
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

D = 128


def make(lens, H, G, bs, seed=0, extra_blocks=3, spread=1.0, offset=0.0, pad_cols=0):
    """A batch over a shuffled 4-bit pool; rows no sequence owns stand for NaN."""
    rng = np.random.default_rng(seed)
    need = [(n + bs - 1) // bs for n in lens]
    nb = sum(need) + extra_blocks
    perm = rng.permutation(nb).astype(np.int32)
    table = np.full((len(lens), max(1, max(need, default=1)) + pad_cols), nb - 1, np.int32)
    k = np.full((nb, bs, H, 80), 0xFF, np.uint8)  # fp16 0xFFFF: NaN
    v = np.full((nb, bs, H, 80), 0xFF, np.uint8)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        x = (rng.standard_normal((2, n, H, D)) * spread + offset).astype(np.float32)
        t = np.arange(n)
        k[table[b, t // bs], t % bs] = lc.q4_quantise(x[0])
        v[table[b, t // bs], t % bs] = lc.q4_quantise(x[1])
    q = torch.from_numpy(rng.standard_normal((len(lens), H * G, D)).astype(np.float32)).bfloat16()
    return dict(q=q, k=k, v=v, table=table, lens=np.array(lens, np.int32), bs=bs, H=H, G=G,
                scale=D ** -0.5)


def run(w, max_len=None, ws=None, stream=None):
    need_gpu()
    q = w["q"].cuda()
    out = torch.full_like(q, float("nan"))
    mcl = max(1, int(w["lens"].max())) if max_len is None else max_len
    if ws is None:
        ws = pa.decode_workspace(q.shape[0], q.shape[1], w["H"], D, mcl)
    k, v, table, lens = (torch.from_numpy(w[n]).cuda() for n in ("k", "v", "table", "lens"))
    pa.pa_paged_decode_attention_q4(out, q, k, v, table, lens, w["scale"], mcl, ws, stream=stream)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), pa.read_device_error(ws)


def reference(w, limit=None):
    return lc.decode(w["q"].float().numpy().astype(np.float64), lc.q4_restore(w["k"]),
                     lc.q4_restore(w["v"]), w["table"], w["lens"], w["bs"], w["scale"], limit)


def check(got, ref, vmax, span, norm=True):
    assert np.isfinite(got).all()
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * (vmax + span) + 2.0 ** -16 * vmax
    assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()
    if norm and np.linalg.norm(ref) > 0:
        assert np.linalg.norm(got - ref) <= 4e-3 * np.linalg.norm(ref)


def check_case(w, **kw):
    got, err = run(w, **kw)
    ref, _ = reference(w)
    assert err == 0
    vals = lc.q4_restore(w["v"])
    live = np.abs(vals[np.isfinite(vals)])
    pairs = np.ascontiguousarray(w["v"][..., 64:]).view(np.float16).astype(np.float64)
    span = 15 * np.nanmax(pairs[..., 0::2]) if np.isfinite(pairs).any() else 0.0
    check(got, ref, live.max() if live.size else 0.0, span)
    for b, n in enumerate(w["lens"]):
        if n == 0:
            assert (got[b] == 0).all()


@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
def test_ragged_batch(bs, G):
    check_case(make([0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000], 2, G, bs,
                    seed=bs + G, pad_cols=2))


@pytest.mark.parametrize("H", [1, 3, 5, 8])
def test_heads(H):
    check_case(make([37, 700, 5], H, 4, 16, seed=H))


@pytest.mark.parametrize("n", [1, 2, 7, 8, 31, 32, 33, 96, 2049, 9001])
def test_one_sequence(n):
    check_case(make([n], 1, 2, 16, seed=n))


def test_many_sequences():
    rng = np.random.default_rng(3)
    check_case(make(rng.integers(0, 600, 70).tolist(), 2, 2, 16, seed=3))


@pytest.mark.parametrize("bs", [16, 256])
def test_long_split_contexts(bs):
    """One sequence over many splits, beside a short one."""
    check_case(make([20000, 33], 1, 4, bs, seed=bs))


def test_context_hint_sets_the_splits_only():
    w = make([500, 900], 2, 4, 16, seed=11)
    a, _ = run(w)
    b, err = run(w, max_len=8192)
    assert err == 0
    assert np.linalg.norm(a - b) <= 2 * 2.3e-3 * np.linalg.norm(a)  # each rounded to bf16 once
    check_case(w, max_len=8192)


def test_lengths_beyond_the_plan_are_clipped_and_flagged():
    w = make([500, 20], 2, 4, 16, seed=12)
    got, err = run(w, max_len=128)
    assert err & pa.PA_DEVERR_CONTEXT_CLIPPED
    splits, per = pa.pa_paged_decode_plan(2, 2, 128)
    ref, _ = reference(w, limit=splits * per)
    check(got, ref, 8.0, 12.0)
    # and to the block table
    w2 = make([500, 20], 2, 4, 16, seed=12)
    w2["lens"] = np.array([512 + 40, 20], np.int32)
    w2["k"][w2["table"][0, 31], 4:] = lc.q4_quantise(np.zeros((12, 2, D), np.float32))
    w2["v"][w2["table"][0, 31], 4:] = lc.q4_quantise(np.zeros((12, 2, D), np.float32))
    got, err = run(w2, max_len=1024)
    assert err & pa.PA_DEVERR_CONTEXT_CLIPPED
    check(got, reference(w2)[0], 8.0, 12.0)


@pytest.mark.parametrize("bs", [8, 16, 64, 256])
def test_dropped_blocks(bs):
    w = make([300, 700, 90, 40], 2, 4, bs, seed=bs + 1)
    rng = np.random.default_rng(bs)
    drop = rng.random(w["table"].shape) < 0.3
    bad = rng.choice(np.array([-1, -2 ** 31, len(w["k"]), 2 ** 31 - 1], np.int64), w["table"].shape)
    w["table"] = np.where(drop, bad, w["table"]).astype(np.int32)
    w["table"][3] = -1  # nothing left: a zero row
    got, err = run(w)
    ref, _ = reference(w)
    assert err == 0 and (got[3] == 0).all()
    check(got, ref, 8.0, 12.0)


def test_physical_order_does_not_matter():
    w = make([400, 77], 2, 4, 16, seed=21)
    a, _ = run(w)
    perm = np.random.default_rng(5).permutation(len(w["k"]))
    inv = np.argsort(perm).astype(np.int32)
    w2 = dict(w, k=w["k"][perm], v=w["v"][perm], table=inv[w["table"]])
    b, _ = run(w2)
    assert (a == b).all()


@pytest.mark.parametrize("factor", [2.0 ** -40, 2.0 ** -12, 1.0, 2.0 ** 12])
def test_query_magnitudes(factor):
    """q scaled by a power of two and the softmax scale by its inverse: the same outputs."""
    w = make([200, 33], 2, 4, 16, seed=31)
    w2 = dict(w, q=(w["q"].float() * factor).bfloat16(), scale=w["scale"] / factor)
    a, _ = run(w)
    b, _ = run(w2)
    assert (a == b).all()


def test_heads_of_very_different_magnitude():
    """Each head's q has its own power of two: a small head beside a large one."""
    w = make([300], 1, 4, 16, seed=32)
    f = torch.tensor([1.0, 2.0 ** 10, 2.0 ** -30, 3.0])[None, :, None]
    w["q"] = (w["q"].float() * f).bfloat16()
    check_case(w)


@pytest.mark.parametrize("spread,offset", [(1e-3, 0.0), (1e-5, 0.0), (100.0, 0.0), (1.0, 30.0)])
def test_value_magnitudes(spread, offset):
    w = make([260, 19], 2, 4, 16, seed=41, spread=spread, offset=offset)
    if spread > 1 or offset:
        w["scale"] /= spread * spread if spread > 1 else offset
    got, err = run(w)
    ref, _ = reference(w)
    vals = lc.q4_restore(w["v"])
    pairs = np.ascontiguousarray(w["v"][..., 64:]).view(np.float16).astype(np.float64)
    # scores off by 2^-22 of the largest |q||k| sums: part of the 2^-16 for |q.k scale| < 2^6
    check(got, ref, np.nanmax(np.abs(vals)), 15 * np.nanmax(pairs[..., 0::2]), norm=offset == 0)


def test_sharp_softmax():
    """Scores hundreds apart: one token takes all the weight, the running maximum moves often."""
    w = make([900], 2, 4, 16, seed=51)
    w["scale"] = 30.0
    got, err = run(w)
    ref, _ = reference(w)
    vals = lc.q4_restore(w["v"])
    # scores reach 2000: fp32 sums of that size are off by 2^-13 at most, and so are weights
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -11) * 16
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all()


def test_nan_row_poisons_its_heads_only():
    for n in (40, 5000):
        w = make([n, n], 2, 4, 16, seed=61)
        t = n // 2
        w["v"][w["table"][0, t // 16], t % 16, 1] = lc.q4_quantise(np.full((D,), np.nan, np.float32))
        w["k"][w["table"][1, t // 16], t % 16, 0] = lc.q4_quantise(np.full((D,), np.nan, np.float32))
        got, _ = run(w)
        assert np.isnan(got[0, 4:]).all() and np.isfinite(got[0, :4]).all()
        assert np.isnan(got[1, :4]).all() and np.isfinite(got[1, 4:]).all()


def test_calls_sharing_a_workspace_and_replays():
    need_gpu()
    w = make([3000, 100, 0], 2, 4, 16, seed=71)
    ws = pa.decode_workspace(3, 8, 2, D, 3000)
    a, _ = run(w, ws=ws)
    b, _ = run(w, ws=ws)
    assert (a == b).all()  # fixed summation order
    q, k, v, table, lens = (w["q"].cuda(), *(torch.from_numpy(w[n]).cuda()
                                             for n in ("k", "v", "table", "lens")))
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_paged_decode_attention_q4(out, q, k, v, table, lens, w["scale"], 3000, ws)
    lens.copy_(torch.tensor([2500, 7, 1], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    w2 = dict(w, lens=np.array([2500, 7, 1], np.int32))
    ref, _ = reference(w2)
    got = out.float().cpu().numpy()
    # sequence 2 had no block: its table names a block of NaN rows
    check(got[:2], ref[:2], 8.0, 12.0)
    side = torch.cuda.Stream()
    c, _ = run(w, ws=pa.decode_workspace(3, 8, 2, D, 3000), stream=side)
    assert (a == c).all()


def test_write_then_attend():
    """The decode step: the newest tokens written in 4 bits, then attended to."""
    need_gpu()
    w = make([200, 64, 1], 2, 4, 16, seed=81)
    new = torch.randn(2, 3, 2, D, device="cuda").bfloat16()
    k, v, table, lens = (torch.from_numpy(w[n]).cuda() for n in ("k", "v", "table", "lens"))
    pos = w["lens"] - 1
    slots = torch.from_numpy(w["table"][np.arange(3), pos // 16].astype(np.int64) * 16 + pos % 16).cuda()
    pa.pa_reshape_and_cache_q4(new[0], new[1], k, v, slots)
    w["k"], w["v"] = k.cpu().numpy(), v.cpu().numpy()
    flat = w["k"].reshape(-1, 2, 80)[slots.cpu().numpy()]
    assert (flat == lc.q4_quantise(new[0].float().cpu().numpy())).all()
    check_case(w)
