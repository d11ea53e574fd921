"""Randomised GPU parity of the long-context operators, and the sizes their other
tests do not reach: batches beyond one schedule round, whole-sequence chunks,
pools past 32-bit byte offsets, blocks shared between sequences."""
import numpy as np
import pytest
import torch

from oracle import long_context as lc
from paged_kv_cache_309_gb300 import pa
from tests.gpu_util import need_gpu
from tests.test_gpu_evict import ascending, check_select, pools, random_sums
from tests.test_gpu_q4_decode import D, check, make, reference, run
from tests.test_gpu_scored_decode import batch
from tests.test_gpu_scored_decode import check as check_sums
from tests.test_gpu_scored_decode import run as run_scored

pytestmark = pytest.mark.gpu

VMAX, SPAN = 8.0, 12.0  # bounds of normal values and of their groups' spans (tests/test_gpu_q4_decode.py)


def shapes(seed, cap=60000):
    rng = np.random.default_rng(seed)
    G, H = int(rng.choice([1, 2, 4, 8, 16])), int(rng.choice([1, 2, 3, 4, 5, 8]))
    bs = int(rng.choice([8, 16, 32, 64, 128, 256]))
    B = int(rng.choice([1, 2, 3, 7, 20, 65]))
    top = int(min(cap // (B * H), rng.choice([1, 40, 200, 1000, 5000, 20000])))
    lens = rng.integers(0, max(1, top) + 1, B)
    lens[int(rng.integers(B))] = max(1, top)
    return rng, G, H, bs, lens.tolist()


@pytest.mark.parametrize("seed", range(24))
def test_decode(seed):
    rng, G, H, bs, lens = shapes(seed)
    w = make(lens, H, G, bs, seed=seed, pad_cols=int(rng.integers(0, 3)))
    if seed % 3 == 0:
        drop = rng.random(w["table"].shape) < 0.2
        w["table"] = np.where(drop, -1, w["table"]).astype(np.int32)
    hint = int(w["lens"].max()) + int(rng.choice([0, 1, 100, 5000]))
    got, err = run(w, max_len=hint)
    assert err == 0
    check(got, reference(w)[0], VMAX, SPAN)


@pytest.mark.parametrize("seed", range(18))
def test_scored(seed):
    rng, G, H, bs, lens = shapes(100 + seed, cap=40000)
    cache = ["q4", "bf16", "e4m3"][seed % 3]
    w = batch(cache, lens, H, G, bs, seed=seed)
    if seed % 4 == 0:
        drop = rng.random(w["table"].shape) < 0.2
        w["table"] = np.where(drop, -1, w["table"]).astype(np.int32)
    num_new = int(rng.choice([0, 1, 30, 10 ** 6]))
    T = max(1, int(w["lens"].max()) + int(rng.integers(-5, 9)))
    got, before, err, _ = run_scored(w, num_new, T=T)
    assert err == 0
    check_sums(w, got, before, num_new, cache)


@pytest.mark.parametrize("seed", range(20))
def test_select(seed):
    rng = np.random.default_rng(seed)
    B, H, T = int(rng.integers(1, 6)), int(rng.integers(1, 5)), int(rng.choice([1, 7, 100, 3000, 40000]))
    sums = random_sums((B, H, T), seed, ["weights", "ties", "special", "signed"][seed % 4])
    budget = int(rng.integers(1, T + 3))
    sink = int(rng.integers(0, budget + 1))
    recent = int(rng.integers(0, budget - sink + 1))
    check_select(sums, rng.integers(0, T + 1, B).tolist(), budget, sink, recent,
                 ["apart", "same", "none"][seed % 3])


@pytest.mark.parametrize("B,lo,hi,G,H", [(700, 0, 150, 2, 8), (3000, 0, 40, 1, 2), (300, 60, 70, 4, 4),
                                         (129, 1, 300, 2, 2)])
def test_many_sequences(B, lo, hi, G, H):
    """Schedules of more than 128 sequences, with sequences split and (700 x 8) whole."""
    rng = np.random.default_rng(B)
    w = make(rng.integers(lo, hi + 1, B).tolist(), H, G, 16, seed=B)
    got, err = run(w)
    assert err == 0
    rows = np.unique(np.concatenate([rng.integers(0, B, 40), [0, 1, B - 2, B - 1]]))
    some = dict(w, q=w["q"][torch.from_numpy(rows)], table=w["table"][rows], lens=w["lens"][rows])
    check(got[rows], reference(some)[0], VMAX, SPAN)
    assert np.isfinite(got).all()
    assert (got[w["lens"] == 0] == 0).all()


def test_one_long_among_many_short():
    w = make([5] * 100 + [30000] + [9] * 60, 2, 2, 16, seed=5)
    got, err = run(w)
    assert err == 0
    check(got, reference(w)[0], VMAX, SPAN)


def test_sequences_that_share_blocks():
    """A common prefix: several tables name the same blocks."""
    w = make([640, 100], 2, 4, 16, seed=6)
    table = np.concatenate([w["table"][:1], w["table"][:1], w["table"][:1]]).copy()
    table[1, 20:] = w["table"][0, 20:][::-1]
    w2 = dict(w, table=table, lens=np.array([640, 640, 333], np.int32), q=w["q"][[0, 1, 0]])
    got, err = run(w2)
    assert err == 0
    check(got, reference(w2)[0], VMAX, SPAN)


def test_offsets_past_32_bits():
    """A 4-bit pool of more than 4 GiB per tensor: rows at its far end are written, read,
    attended to and moved."""
    need_gpu()
    H, bs, n = 8, 256, 700
    nb = (2 ** 32 // (H * 80) + 3 * n) // bs + 8
    kc, vc = (torch.zeros(nb, bs, H, 80, dtype=torch.uint8, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 32
    far = np.arange(nb - 3, nb)[None].astype(np.int32)
    t = np.arange(n)
    slots = far[0, t // bs].astype(np.int64) * bs + t % bs
    x = torch.randn(2, n, H, D, device="cuda").bfloat16()
    s = torch.from_numpy(slots).cuda()
    pa.pa_reshape_and_cache_q4(x[0], x[1], kc, vc, s)
    rows = lc.q4_quantise(x.float().cpu().numpy())
    assert (kc.view(-1, H, 80)[s].cpu().numpy() == rows[0]).all()
    assert int((kc[:-3] != 0).any()) == 0
    back = torch.zeros(2, n, H, D, device="cuda")
    pa.pa_gather_cache_q4(back[0], back[1], kc, vc, s)
    values = lc.q4_restore(rows)
    assert (np.abs(back.cpu().numpy() - values) <= np.abs(values) * 2.0 ** -23).all()
    # attention over the far end, then the rows compacted into it from there
    k, v = np.zeros((3, bs, H, 80), np.uint8), np.zeros((3, bs, H, 80), np.uint8)
    k[t // bs, t % bs], v[t // bs, t % bs] = rows[0], rows[1]
    q = torch.randn(1, H * 2, D).bfloat16()
    w = dict(q=q, k=k, v=v, table=np.arange(3, dtype=np.int32)[None], lens=np.array([n], np.int32),
             bs=bs, H=H, G=2, scale=D ** -0.5)
    ws = pa.decode_workspace(1, H * 2, H, D, n)
    out = torch.empty_like(q.cuda())
    table, lens = torch.from_numpy(far).cuda(), torch.tensor([n], dtype=torch.int32).cuda()
    pa.pa_paged_decode_attention_q4(out, q.cuda(), kc, vc, table, lens, w["scale"], n, ws)
    check(out.float().cpu().numpy().astype(np.float64), reference(w)[0], VMAX, SPAN)
    keep = ascending(1, H, 300, [n], 1)
    pa.pa_cache_compact(kc, vc, torch.from_numpy(keep).cuda(),
                        torch.tensor([300], dtype=torch.int32).cuda(), table, table)
    lc.compact(k, keep, [300], w["table"], w["table"])
    assert (kc[-3:].cpu().numpy() == k).all()
    pa.pa_cache_compact(kc, vc, torch.from_numpy(np.arange(300, dtype=np.int32)[None, None].repeat(H, 1)).cuda(),
                        torch.tensor([300], dtype=torch.int32).cuda(), table,
                        torch.arange(2, dtype=torch.int32, device="cuda")[None])
    assert (kc.view(-1, H, 80)[:300].cpu().numpy() == k.reshape(-1, H, 80)[:300]).all()


def test_two_streams_at_once():
    """Two calls at a time, each with its own workspace, many times over."""
    ws = [make([900, 100, 0, 2000], 2, 4, 16, seed=s) for s in (1, 2)]
    refs = [reference(w)[0] for w in ws]
    need_gpu()
    streams = [torch.cuda.Stream() for _ in ws]
    state = []
    for w in ws:
        q = w["q"].cuda()
        state.append((q, *(torch.from_numpy(w[n]).cuda() for n in ("k", "v", "table", "lens")),
                      pa.decode_workspace(4, 8, 2, D, 2000), [torch.empty_like(q) for _ in range(20)]))
    torch.cuda.synchronize()
    for i in range(20):
        for w, st, (q, k, v, table, lens, space, outs) in zip(ws, streams, state):
            pa.pa_paged_decode_attention_q4(outs[i], q, k, v, table, lens, w["scale"], 2000, space,
                                            stream=st)
    torch.cuda.synchronize()
    for ref, (*_, outs) in zip(refs, state):
        for o in outs:
            assert (o == outs[0]).all()
        check(outs[0].float().cpu().numpy().astype(np.float64), ref, VMAX, SPAN)


def test_one_workspace_for_every_decode_call():
    """The 4-bit and the bf16 calls in turn on one workspace leave each other right."""
    w = batch("bf16", [3000, 77], 2, 4, 16, seed=9)
    v = batch("q4", [2500, 900], 2, 4, 16, seed=10)
    ws = pa.decode_scored_workspace(2, 8, 2, D, 3000)
    first = {}
    for i in range(3):
        for name, x, fn in (("bf16", w, "plain"), ("q4", v, "plain"), ("bf16", w, "scored"),
                            ("q4", v, "scored")):
            q = x["q"].cuda()
            out, sums = torch.empty_like(q), torch.zeros(2, 2, 3000, device="cuda")
            table, lens = torch.from_numpy(x["table"]).cuda(), torch.from_numpy(x["lens"]).cuda()
            if fn == "scored":
                pa.pa_paged_decode_attention_scored(out, sums, sums, 0, q, x["kd"], x["vd"], table,
                                                    lens, x["scale"], 3000, ws)
            elif name == "q4":
                pa.pa_paged_decode_attention_q4(out, q, x["kd"], x["vd"], table, lens, x["scale"],
                                                3000, ws)
            else:
                pa.pa_paged_decode_attention(out, q, x["kd"], x["vd"], table, lens, x["scale"],
                                             3000, ws)
            if i == 0:
                first[name, fn] = (out, sums)
                ref, _ = lc.decode(x["q"].float().numpy().astype(np.float64), x["k64"], x["v64"],
                                   x["table"], x["lens"], 16, x["scale"])
                check(out.float().cpu().numpy().astype(np.float64), ref, VMAX, SPAN)
            assert (out == first[name, fn][0]).all() and (sums == first[name, fn][1]).all()
    assert pa.read_device_error(ws) == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "q4"])
def test_growing_context_hint_on_one_workspace(cache):
    """Short hints (one range) before long ones (several, counted): the counters stay zero."""
    w = batch(cache, [60, 33], 2, 4, 16, seed=11)
    full = batch(cache, [2000, 900], 2, 4, 16, seed=12)
    ws = pa.decode_scored_workspace(2, 8, 2, D, 2048)
    for x, hint in ((w, 64), (full, 2048), (w, 64), (full, 2000)):
        got, before, err, _ = run_scored(x, 10 ** 6, max_len=hint, ws=ws)
        assert err == 0
        check_sums(x, got, before, 10 ** 6, cache)


def test_scored_and_plain_plans_on_one_workspace():
    """1280 (sequence, kv head) pairs: one range in the scored call, several in the decode call."""
    rng = np.random.default_rng(3)
    w = batch("bf16", rng.integers(1, 200, 320).tolist(), 4, 1, 16, seed=13)
    ws = pa.decode_scored_workspace(320, 4, 4, D, 256)
    q = w["q"].cuda()
    table, lens = torch.from_numpy(w["table"]).cuda(), torch.from_numpy(w["lens"]).cuda()
    for _ in range(2):
        got, before, err, _ = run_scored(w, 0, max_len=256, ws=ws)
        assert err == 0
        check_sums(w, got, before, 0, "bf16")
        out = torch.empty_like(q)
        pa.pa_paged_decode_attention(out, q, w["kd"], w["vd"], table, lens, w["scale"], 256, ws)
        ref, _ = lc.decode(w["q"].float().numpy().astype(np.float64), w["k64"], w["v64"], w["table"],
                           w["lens"], 16, w["scale"])
        check(out.float().cpu().numpy().astype(np.float64), ref, VMAX, SPAN)
