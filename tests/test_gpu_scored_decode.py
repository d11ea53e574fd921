"""GPU parity of the decode attention that adds up attention weights.

The outputs are those of the cache's own decode call (compared with it, bit
for bit over 4 bits; its own tests check it against the oracle).  Weights against the
oracle in double: a score (base 2) is an fp32 sum of 128 exact products (or 4
groups' sums) with at most 24 roundings in a chain, each 2^-23 of a partial sum
below 2^5.1 (normal data: sum |q k| scale log2 e, or its 4-bit form with codes
not centred), so it is off by 7e-5 / 2 at most, and so is the log-sum-exp:
a weight by 2 ln 2 of that, 2^-13.3, plus 2^-21 for exp2: 2^-13 of it is asked
(2^-12 for 4 bits: the minimum's part adds a sum of the same size).  The
errors are independent over tokens: 2e-5 of the 2-norm.  Adding to a sum
rounds once (2^-24 of the result).
"""
import numpy as np
import pytest
import torch

from oracle import long_context as lc
from paged_kv_cache_309_gb300 import pa
from tests.gpu_util import need_gpu
from tests.test_gpu_q4_decode import D, make

pytestmark = pytest.mark.gpu


def batch(cache, lens, H, G, bs, **kw):
    """make()'s batch with device caches of the given type and their float64 values."""
    need_gpu()
    w = make(lens, H, G, bs, **kw)
    w["ks"] = w["vs"] = None
    if cache == "q4":
        w["kd"], w["vd"] = torch.from_numpy(w["k"]).cuda(), torch.from_numpy(w["v"]).cuda()
        w["k64"], w["v64"] = lc.q4_restore(w["k"]), lc.q4_restore(w["v"])
        return w
    for n in ("k", "v"):
        x = torch.from_numpy(lc.q4_restore(w[n])).float()  # NaN where no sequence is
        if cache == "e4m3":
            w[n + "s"] = torch.tensor([0.05 if n == "k" else 0.07]).cuda()
            c = (x.cuda() / w[n + "s"]).to(torch.float8_e4m3fn)
            w[n + "64"] = c.cpu().float().numpy().astype(np.float64) * float(w[n + "s"])
        else:
            c = x.bfloat16().cuda()
            w[n + "64"] = c.cpu().float().numpy().astype(np.float64)
        w[n + "d"] = c
    return w


def run(w, num_new, T=None, sums=None, max_len=None, ws=None, in_place=False):
    q = w["q"].cuda()
    B, HQ, _ = q.shape
    T = max(1, int(w["lens"].max())) if T is None else T
    mcl = max(1, int(w["lens"].max())) if max_len is None else max_len
    out = torch.full_like(q, float("nan"))
    if sums is None:
        sums = torch.rand(B, w["H"], T, generator=torch.Generator().manual_seed(1)).cuda()
    before = sums.cpu().numpy().astype(np.float64)
    dst = sums if in_place else torch.full_like(sums, -5.0)
    if ws is None:
        ws = pa.decode_scored_workspace(B, HQ, w["H"], D, mcl)
    table, lens = torch.from_numpy(w["table"]).cuda(), torch.from_numpy(w["lens"]).cuda()
    pa.pa_paged_decode_attention_scored(out, dst, sums, num_new, q, w["kd"], w["vd"], table, lens,
                                        w["scale"], mcl, ws, k_scale=w["ks"], v_scale=w["vs"])
    plain = torch.full_like(q, float("nan"))
    dws = pa.decode_workspace(B, HQ, w["H"], D, mcl)
    if w["kd"].dtype == torch.uint8:
        pa.pa_paged_decode_attention_q4(plain, q, w["kd"], w["vd"], table, lens, w["scale"], mcl, dws)
    else:
        pa.pa_paged_decode_attention(plain, q, w["kd"], w["vd"], table, lens, w["scale"], mcl, dws,
                                     k_scale=w["ks"], v_scale=w["vs"])
    torch.cuda.synchronize()
    if w["kd"].dtype == torch.uint8:
        same = out.view(torch.int16) == plain.view(torch.int16)
        assert (same | (out.isnan() & plain.isnan())).all()
    elif not pa.read_device_error(dws):
        # other ranges, the same values: each rounded to bf16 once (2^-7 of the smaller apart
        # at most), fp32 sums in another order
        a, b = out.float(), plain.float()
        assert (a.isnan() == b.isnan()).all()
        a, b = a.nan_to_num(), b.nan_to_num()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2e-4 * b.abs().amax().clamp(min=1.0)).all()
    return dst.cpu().numpy().astype(np.float64), before, pa.read_device_error(ws), out


def check(w, got, before, num_new, cache, untouched=-5.0, limit=None):
    _, weights = lc.decode(w["q"].float().numpy().astype(np.float64), w["k64"], w["v64"],
                           w["table"], w["lens"], w["bs"], w["scale"], limit)
    T = got.shape[2]
    want = np.full(got.shape, untouched)
    if untouched is None:
        want = before.copy()
    for b, n in enumerate(w["lens"]):
        n = int(n) if limit is None else min(int(n), limit)
        m = min(n, T)
        old = before[b, :, :m] * (np.arange(m) < n - num_new)
        ref = weights[b, :, :m]
        want[b, :, :m] = old + ref
        rel = 2.0 ** -12 if cache == "q4" else 2.0 ** -13
        tol = rel * ref + 2.0 ** -24 * np.abs(want[b, :, :m]) + 2.0 ** -100
        assert (np.abs(got[b, :, :m] - want[b, :, :m]) <= tol).all()
        assert (got[b, :, m:] == want[b, :, m:]).all()  # behind the sequence: as it was
        if num_new >= n and m == n and n > 0:
            assert np.linalg.norm(got[b, :, :m] - ref) <= 2e-5 * np.linalg.norm(ref) + 1e-30
            total = got[b].clip(0)[:, :m].sum(-1)
            live = ref.sum(-1) > 0
            assert (np.abs(total - w["G"])[live] <= 1e-4 * w["G"]).all()


CACHES = ["bf16", "e4m3", "q4"]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("bs", [8, 64, 256])
def test_ragged_batch(cache, G, bs):
    w = batch(cache, [0, 1, 16, 17, 63, 64, 65, 127, 129, 300, 1000], 2, G, bs, seed=bs + G)
    for num_new in (0, 1, 17, 5000):
        got, before, err, _ = run(w, num_new)
        assert err == 0
        check(w, got, before, num_new, cache)


@pytest.mark.parametrize("cache", CACHES)
def test_long_splits_and_odd_heads(cache):
    w = batch(cache, [20000, 33, 9001], 3, 4, 16, seed=7)
    got, before, err, _ = run(w, 1 << 40)
    assert err == 0
    check(w, got, before, 1 << 40, cache)


@pytest.mark.parametrize("cache", CACHES)
def test_dropped_blocks_weigh_nothing(cache):
    w = batch(cache, [300, 700, 40, 1500], 2, 4, 16, seed=8)
    drop = np.random.default_rng(2).random(w["table"].shape) < 0.3
    w["table"] = np.where(drop, -1, w["table"]).astype(np.int32)
    w["table"][2] = len(w["k"])
    for num_new in (0, 5000):
        got, before, err, _ = run(w, num_new)
        assert err == 0
        check(w, got, before, num_new, cache)


@pytest.mark.parametrize("cache", CACHES)
def test_rows_of_sums_longer_and_shorter_than_the_context(cache):
    w = batch(cache, [300, 70], 2, 2, 16, seed=9)
    for T in (1000, 100, 1):
        got, before, err, _ = run(w, 1, T=T)
        assert err == 0
        check(w, got, before, 1, cache)


@pytest.mark.parametrize("cache", CACHES)
def test_in_place_over_steps(cache):
    """Three decode steps into one array: the new token starts at zero, the rest add up."""
    w = batch(cache, [200, 61], 2, 4, 16, seed=10)
    sums = torch.full((2, 2, 256), float("nan"), device="cuda")
    want = np.full((2, 2, 256), np.nan)
    ws = pa.decode_scored_workspace(2, 8, 2, D, 256)
    full = w["lens"].copy()
    for step in range(3):
        w["lens"] = (full - 2 + step).astype(np.int32)
        num_new = 1 << 30 if step == 0 else 1
        run(w, num_new, sums=sums, max_len=256, ws=ws, in_place=True)
        _, weights = lc.decode(w["q"].float().numpy().astype(np.float64), w["k64"], w["v64"],
                               w["table"], w["lens"], 16, w["scale"])
        for b, n in enumerate(w["lens"]):
            new = np.arange(n) >= n - num_new
            want[b, :, :n] = np.where(new, 0, np.nan_to_num(want[b, :, :n])) + weights[b, :, :n]
    got = sums.cpu().numpy()
    assert (np.isnan(got) == np.isnan(want)).all()
    ok = ~np.isnan(want)
    assert (np.abs(got - want)[ok] <= (2.0 ** -12 * want)[ok]).all()


def test_clipped_lengths():
    w = batch("bf16", [500, 20], 2, 4, 16, seed=12)
    got, before, err, _ = run(w, 1, max_len=128)
    assert err & pa.PA_DEVERR_CONTEXT_CLIPPED
    check(w, got, before, 1, "bf16", limit=128)  # ranges of whole 64s


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("n", [40, 3000])
def test_nan_key_makes_its_heads_sums_nan(cache, n):
    w = batch(cache, [n, n], 2, 4, 16, seed=13)
    t = n // 2
    at = (int(w["table"][0, t // 16]), t % 16, 1)
    if cache == "q4":
        w["kd"][at] = torch.from_numpy(lc.q4_quantise(np.full((D,), np.nan, np.float32))).cuda()
    else:
        w["kd"].view(torch.int8 if cache == "e4m3" else torch.int16)[at] = 127 if cache == "e4m3" else 0x7FC0
    got, _, _, out = run(w, n)
    assert np.isnan(got[0, 1]).all() and np.isfinite(got[0, 0]).all() and np.isfinite(got[1]).all()
    assert out[0, 4:].isnan().all() and not out[0, :4].isnan().any() and not out[1].isnan().any()


def test_replayed_graph_sees_new_lengths():
    w = batch("q4", [900, 31], 2, 4, 16, seed=14)
    ws = pa.decode_scored_workspace(2, 8, 2, D, 1024)
    q, table = w["q"].cuda(), torch.from_numpy(w["table"]).cuda()
    lens = torch.from_numpy(w["lens"]).cuda()
    out, sums = torch.zeros_like(q), torch.zeros(2, 2, 1024, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_paged_decode_attention_scored(out, sums, sums, 1 << 30, q, w["kd"], w["vd"], table,
                                            lens, w["scale"], 1024, ws)
    w["lens"] = np.array([555, 12], np.int32)
    lens.copy_(torch.from_numpy(w["lens"]))
    g.replay()
    torch.cuda.synchronize()
    got = sums.cpu().numpy().astype(np.float64)
    check(w, got, np.zeros_like(got), 1 << 30, "q4", untouched=0.0)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("G", [1, 16])
def test_no_context_at_all(cache, G):
    """max_context_len 0: the outputs are 0 and no sum is touched."""
    w = batch(cache, [0, 0, 0], 2, G, 16, seed=14)
    got, _, err, out = run(w, 1, T=5, max_len=0)
    assert err == 0
    assert (out == 0).all()
    assert (got == -5.0).all()
