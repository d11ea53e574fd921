"""GPU tests of the sliding-window calls where sizes and contents leave the ordinary: many
sequences, every way of cutting a batch, pools past 4 GiB, lengths and offsets that make
no sense, calls that share rows, and random batches.  Bounds as in test_gpu_window.py."""
import numpy as np
import pytest
import torch

from oracle import window as ow
from paged_kv_cache_309_gb300 import pa
from tests.gpu_util import need_gpu
from tests.test_gpu_window import BF16, E4M3, SCALE, Batch, compare, decode, prefill, queries

pytestmark = pytest.mark.gpu


def check_some(lens, hq, h, bs, window, sink, rows, seed, cache=BF16, most=None):
    batch = Batch(lens, h, bs, seed, cache=cache)
    q = queries(len(lens), hq, seed + 1)
    out, ws = decode(batch, q, window, sink, most=most)
    assert pa.read_device_error(ws) == 0
    rows = list(rows)
    ref = ow.decode(q[rows].double().numpy(), *batch.values(), batch.tables[rows], batch.lens[rows], window, sink, SCALE)
    compare(out[rows], ref, 2.0 ** -16 if cache == BF16 else 2.0 ** -11)


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("n,lo,hi,h,window", [
    (200, 300, 700, 2, 100),    # whole sequences, two and more to a CTA
    (300, 300, 700, 3, 130),    # more sequences than CTAs of a head
    (64, 0, 1500, 2, 1000),     # an even cut, few pieces a sequence
    (40, 2500, 2600, 8, 1024),  # the same with lengths alike
    (2, 3000, 3000, 1, 2900),   # many pieces a sequence
    (129, 1, 257, 1, 5000),     # a window that reaches past every context
])
def test_every_cut_of_a_batch(n, lo, hi, h, window, cache):
    lens = np.linspace(lo, hi, n).astype(int).tolist()
    check_some(lens, 2 * h, h, 16, window, 4, sorted({0, 1, n // 3, n // 2, n - 2, n - 1}), n + window, cache)


def test_thousands_of_sequences():
    lens = (np.arange(3000) % 41).tolist()
    check_some(lens, 2, 1, 8, 17, 3, range(0, 3000, 97), 1)


def test_lengths_that_make_no_sense():
    """Negative lengths are empty contexts, huge ones are clipped and flagged."""
    batch = Batch([64, 64, 64, 64], 2, 16, 2)
    q = queries(4, 4, 3)
    batch.lens = np.array([-5, 64, 2 ** 31 - 1, -2 ** 31], np.int32)
    out, ws = decode(batch, q, 20, 4, most=64)
    assert pa.read_device_error(ws) == pa.PA_DEVERR_CONTEXT_CLIPPED
    ref = ow.decode(q.double().numpy(), *batch.values(), batch.tables, [0, 64, 64, 0], 20, 4, SCALE)
    compare(out, ref, 2.0 ** -16)


def without_infinite_keys(batch, q, lens, starts, window, sink, infinite):
    """What ow.decode gives where the tokens infinite(t) have no weight (starts: rows of each sequence)."""
    hq, g = q.shape[1], q.shape[1] // batch.h
    refs = [np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape[:2])]
    kc, vc = batch.values()
    for b, n in enumerate(lens):
        new = starts[b + 1] - starts[b]
        for j in range(new):
            t = np.array([t for t in ow.visible(n - new + j, window, sink) if not infinite(b, t)], np.int64)
            for h in range(0, hq, g):
                x = ow.row(q[starts[b] + j, h:h + g].double().numpy(), kc[:, :, h // g], vc[:, :, h // g],
                           batch.tables[b], t, SCALE)
                for r, y in zip(refs, x):
                    r[starts[b] + j, h:h + g] = y
    return refs


def with_infinite_keys(lens, hq, new):
    """A batch whose queries are positive in element 0, and keys of -inf there: scores of -inf."""
    def infinite(b, t):
        return b == 2 or t < 40 or t % 7 == 3 or 150 <= t < 260
    batch = Batch(lens, 2, 16, 21)
    for b, n in enumerate(lens):
        for t in range(n):
            if infinite(b, t):
                batch.pools[0][batch.tables[b, t // 16], t % 16, :, 0] = -float("inf")
    q = queries(new, hq, 22)
    q[:, :, 0] = q[:, :, 0].abs() + 1
    return batch, q, infinite


@pytest.mark.parametrize("window", [90, 1000])
def test_decode_scores_of_minus_infinity(window):
    """They have no weight, first in a row or later; a row of them alone is zero."""
    lens = [700, 300, 100, 41]
    batch, q, infinite = with_infinite_keys(lens, 8, 4)
    out, _ = decode(batch, q, window, 4)
    compare(out, without_infinite_keys(batch, q, lens, range(5), window, 4, infinite), 2.0 ** -16)
    assert bool((out[2] == 0).all())


@pytest.mark.parametrize("window", [90, 1000])
def test_prefill_scores_of_minus_infinity(window):
    lens, new = [400, 300, 100, 41], [300, 300, 100, 1]
    batch, q, infinite = with_infinite_keys(lens, 4, sum(new))
    out, starts = prefill(batch, q, new, window, 4)
    compare(out, without_infinite_keys(batch, q, lens, starts.tolist(), window, 4, infinite), 2.0 ** -8)
    assert bool((out[600:700] == 0).all())


@pytest.mark.parametrize("scale", [-SCALE, 0.0, 3.0])
def test_any_scale(scale, monkeypatch):
    """Scores may be turned round or all be equal; a scale of 3 leaves few tokens with a weight."""
    monkeypatch.setattr("tests.test_gpu_window.SCALE", scale)
    lens, new = [400, 300, 33], [200, 300, 1]
    for cache, r in ((BF16, 2.0 ** -16), (E4M3, 2.0 ** -11)):
        batch, q = Batch(lens, 2, 16, 23, cache=cache), queries(3, 8, 24)
        out, _ = decode(batch, q, 130, 4)
        compare(out, ow.decode(q.double().numpy(), *batch.values(), batch.tables, lens, 130, 4, scale), r)
    batch, q = Batch(lens, 2, 16, 25), queries(sum(new), 8, 26)
    out, starts = prefill(batch, q, new, 130, 4)
    ref = ow.prefill(q.double().numpy(), *batch.values(), batch.tables, starts, lens, 130, 4, scale)
    compare(out, ref, 2.0 ** -8)


def test_one_block_for_all():
    """Sequences may share blocks."""
    batch = Batch([40, 40, 33], 2, 16, 4)
    batch.tables[:] = batch.tables[:1]
    q = queries(3, 8, 5)
    ref = ow.decode(q.double().numpy(), *batch.values(), batch.tables, batch.lens, 30, 2, SCALE)
    compare(decode(batch, q, 30, 2)[0], ref, 2.0 ** -16)


def test_prefill_many_short_sequences():
    """More sequences than a warp looks at at once, empty ones among them."""
    rng = np.random.default_rng(6)
    new = rng.integers(0, 90, 75).tolist()
    lens = [n + int(rng.integers(0, 200)) for n in new]
    batch = Batch(lens, 2, 16, 6)
    q = queries(sum(new), 8, 7)
    out, starts = prefill(batch, q, new, 60, 4)
    rows = set(rng.choice(sum(new), 120, replace=False).tolist())
    ref = ow.prefill(q.double().numpy(), *batch.values(), batch.tables, starts, lens, 60, 4, SCALE, rows)
    pick = sorted(rows)
    compare(out[pick], [x[pick] for x in ref], 2.0 ** -8)


@pytest.mark.parametrize("starts,lens", [
    ([0, 50, 20, 90], [50, 70, 70]),                  # a sequence that ends before it starts has no rows
    ([0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], [60, 5, 7]),  # far past the array
    ([-40, 30, 60, 90], [70, 30, 30]),                # rows before the array
    ([0, 0, 0, 0], [70, 30, 30]),
    ([0, 30, 60, 90], [-3, 2 ** 31 - 1, 0]),
])
def test_prefill_offsets_that_make_no_sense(starts, lens):
    """No row outside the array is touched and the call ends; rows of sound sequences are right."""
    need_gpu()
    batch = Batch([70, 70, 70], 2, 16, 8)
    q = queries(120, 4, 9)
    k, v, bt, _ = batch.device()
    guard = torch.full((360, 4, 128), 7.0, dtype=BF16, device="cuda")
    out, dq = guard[120:240], q.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_paged_window_prefill_attention(
        out, dq, k, v, bt, torch.tensor(starts, dtype=torch.int32, device="cuda"),
        torch.tensor(lens, dtype=torch.int32, device="cuda"), 25, 3, SCALE, 100, err)
    torch.cuda.synchronize()
    assert int(err) & ~pa.PA_DEVERR_CONTEXT_CLIPPED == 0
    assert bool((guard[:120] == 7).all()) and bool((guard[240:] == 7).all())
    got = out.double().cpu().numpy()
    cap = batch.tables.shape[1] * 16
    seen = np.zeros(120, int)
    for b in range(3):
        n = max(0, starts[b + 1] - starts[b])
        for j in range(min(n, 100)):
            if 0 <= starts[b] and starts[b] + j < 120:
                seen[starts[b] + j] += 1
    assert (got[seen == 0] == 7).all()
    for b in range(3):
        n, length = max(0, starts[b + 1] - starts[b]), min(max(lens[b], 0), cap)
        if starts[b] < 0 or lens[b] > cap:
            continue
        for j in range(0, min(n, 100, 120 - starts[b]), 7):
            i = starts[b] + j
            if seen[i] != 1:
                continue
            t = ow.visible(length - n + j, 25, 3)
            for g in range(2):
                ref = ow.row(q[i, 2 * g:2 * g + 2].double().numpy(), *(x[:, :, g] for x in batch.values()),
                             batch.tables[b], t[t < length], SCALE)
                compare(out[i, 2 * g:2 * g + 2], [ref[0], ref[1], np.full(2, ref[2]), np.full(2, ref[3])], 2.0 ** -8)


def test_tokens_past_max_q_len_are_left_out():
    batch = Batch([90, 40], 2, 16, 10)
    q = queries(130, 4, 11)
    k, v, bt, cl = batch.device()
    out = torch.full((130, 4, 128), 7.0, dtype=BF16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 90, 130], dtype=torch.int32, device="cuda")
    pa.pa_paged_window_prefill_attention(out, q.cuda(), k, v, bt, starts, cl, 25, 3, SCALE, 50, err)
    torch.cuda.synchronize()
    ref = ow.prefill(q.double().numpy(), *batch.values(), batch.tables, [0, 90, 130], batch.lens, 25, 3, SCALE)
    pick = list(range(50)) + list(range(90, 130))
    compare(out[pick], [x[pick] for x in ref], 2.0 ** -8)
    assert bool((out[50:90] == 7).all())


@pytest.mark.slow
def test_pools_past_4_gib():
    """Rows whose byte offset passes 2^32: written by the append, read by both attention calls."""
    need_gpu()
    bs, h, hq, n = 16, 8, 8, 70
    blocks = 2 ** 32 // (bs * h * 128 * 2) + 8
    kc, vc = (torch.zeros((blocks, bs, h, 128), dtype=BF16, device="cuda") for _ in range(2))
    table = torch.tensor([[blocks - 1, blocks - 3, 2, blocks - 7, blocks - 5]], dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(12)
    q, k, v = (torch.randn((n, x, 128), generator=gen).bfloat16().cuda() for x in (hq, h, h))
    pos = torch.arange(n, device="cuda")
    slot = table[0].long()[pos // bs] * bs + pos % bs
    cs = torch.cat([torch.ones(128, 64), torch.zeros(128, 64)], 1).cuda()  # no turn
    q_out = torch.empty_like(q)
    pa.pa_rope_and_cache(q_out, q, k, v, kc, vc, cs, pos, slot)
    assert torch.equal(q_out, q)
    assert torch.equal(kc.view(-1, h, 128)[slot], k) and torch.equal(vc.view(-1, h, 128)[slot], v)
    one = [x[None].double().cpu().numpy() for x in (k, v)]
    flat = [np.zeros((1, 80, h, 128)) for _ in range(2)]
    for f, x in zip(flat, one):
        f[:, :n] = x
    lens, starts = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, err = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_paged_window_prefill_attention(out, q, kc, vc, table, starts, lens, 30, 2, SCALE, n, err)
    qn = q.double().cpu().numpy()
    ref = ow.prefill(qn, *flat, np.zeros((1, 1), int), [0, n], [n], 30, 2, SCALE)
    compare(out, ref, 2.0 ** -8)
    ws = pa.window_decode_workspace(1, hq, h, 128, 30, 2, n)
    last = torch.empty_like(q[-1:])
    pa.pa_paged_window_decode_attention(last, q[-1:].contiguous(), kc, vc, table, lens, 30, 2, SCALE, n, ws)
    compare(last, [x[-1:] for x in ref], 2.0 ** -16)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = np.random.default_rng(100 + seed)
    h, g = int(rng.choice([1, 2, 3, 4])), int(rng.choice([1, 2, 4, 8, 16]))
    bs = int(rng.choice([8, 16, 32, 64, 128, 256]))
    window, sink = int(np.exp(rng.uniform(0, 7))), int(rng.choice([0, 1, 4, 30, 200]))
    drop = float(rng.choice([0, 0, 0.2]))
    lens = [int(np.exp(rng.uniform(0, 6.8))) for _ in range(int(rng.integers(1, 9)))]
    cache = BF16 if seed % 2 else E4M3
    batch = Batch(lens, h, bs, seed, cache=cache, drop=drop)
    q = queries(len(lens), h * g, seed + 1)
    out, ws = decode(batch, q, window, sink, most=max(lens) + int(rng.integers(0, 500)))
    ref = ow.decode(q.double().numpy(), *batch.values(), batch.tables, lens, window, sink, SCALE)
    compare(out, ref, 2.0 ** -16 if cache == BF16 else 2.0 ** -11)
    batch = Batch(lens, h, bs, seed, drop=drop)
    new = [int(rng.integers(1, n + 1)) for n in lens]
    q = queries(sum(new), h * g, seed + 2)
    out, starts = prefill(batch, q, new, window, sink)
    rows = set(rng.choice(sum(new), min(sum(new), 60), replace=False).tolist())
    ref = ow.prefill(q.double().numpy(), *batch.values(), batch.tables, starts, lens, window, sink, SCALE, rows)
    pick = sorted(rows)
    compare(out[pick], [x[pick] for x in ref], 2.0 ** -8)


@pytest.mark.parametrize("seed", range(8))
def test_prefill_short_items(seed):
    """Items of one step and few, of one and two query tiles in turn, empty sequences between them."""
    rng = np.random.default_rng(300 + seed)
    n, h, g = int(rng.integers(20, 50)), int(rng.integers(1, 4)), int(rng.choice([1, 2, 4, 8, 16]))
    new = [int(x) for x in rng.integers(0, int(rng.choice([3, 40, 130, 300])) + 1, n - 1)] + [5]
    lens = [a + int(x) for a, x in zip(new, rng.integers(0, int(rng.choice([1, 70, 500])), n))]
    window, sink = int(rng.choice([1, 2, 17, 64, 65, 130])), int(rng.choice([0, 1, 5, 64, 70]))
    batch = Batch(lens, h, int(rng.choice([8, 16, 64, 256])), seed, drop=0.1)
    q = queries(sum(new), h * g, seed + 1)
    out, starts = prefill(batch, q, new, window, sink)
    rows = sorted(rng.choice(sum(new), min(sum(new), 60), replace=False).tolist())
    ref = ow.prefill(q.double().numpy(), *batch.values(), batch.tables, starts, lens, window, sink, SCALE, set(rows))
    compare(out[rows], [x[rows] for x in ref], 2.0 ** -8)
    assert bool((prefill(batch, q, new, window, sink)[0] == out).all())


def test_calls_on_two_streams_at_once():
    """Two calls that share caches and lengths, each with its workspace, on two streams."""
    batch = Batch([900, 2000, 37], 2, 16, 13)
    q = queries(3, 8, 14)
    x, _ = decode(batch, q, 600, 4)
    k, v, bt, cl = batch.device()
    dq = q.cuda()
    outs = [torch.zeros_like(x) for _ in range(2)]
    ws = [pa.window_decode_workspace(3, 8, 2, 128, 600, 4, 2000) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(50):
        for i in range(2):
            pa.pa_paged_window_decode_attention(outs[i], dq, k, v, bt, cl, 600, 4, SCALE, 2000, ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert bool((outs[0] == x).all()) and bool((outs[1] == x).all())


@pytest.mark.parametrize("repeat", range(3))
def test_results_repeat(repeat):
    """The same call gives the same bits, whatever ran before it."""
    new = [300, 1, 220, 64]
    batch = Batch([700, 90, 220, 64], 2, 16, 15)
    q = queries(sum(new), 8, 16)
    first, _ = prefill(batch, q, new, 150, 4)
    for _ in range(20):
        assert torch.equal(prefill(batch, q, new, 150, 4)[0], first)


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_one_workspace_for_batches_of_every_size(cache):
    """A workspace of the largest batch, taken once, serves the smaller ones, cut or whole."""
    need_gpu()
    top, most, window, sink = 130, 900, 300, 4
    ws = pa.window_decode_workspace(top, 16, 4, 128, window, sink, most)
    ws.fill_(255)
    ws[:4] = 0
    r = 2.0 ** -16 if cache == BF16 else 2.0 ** -11
    for n in (130, 64, 33, 20, 7, 1):
        lens = np.linspace(min(n, 2) * 200, most, n).astype(int).tolist()
        batch = Batch(lens, 4, 16, n, cache=cache)
        q = queries(n, 16, n + 1)
        out, _ = decode(batch, q, window, sink, ws=ws)
        rows = sorted({0, n // 2, n - 1})
        ref = ow.decode(q[rows].double().numpy(), *batch.values(), batch.tables[rows], batch.lens[rows], window, sink, SCALE)
        compare(out[rows], ref, r)
    assert pa.read_device_error(ws) == 0


def with_bad_values(batch, rng, tokens):
    """Sets elements of the values of `tokens` tokens a sequence to infinities and NaN; gives the caches
    with these elements 0 and, of all elements, which are +inf or NaN and which -inf or NaN."""
    pool = batch.pools[1]
    for b, n in enumerate(batch.lens):
        for t in rng.choice(int(n), min(int(n), tokens), replace=False):
            blk = batch.tables[b, t // batch.bs]
            if not 0 <= blk < pool.shape[0]:
                continue
            for _ in range(int(rng.integers(1, 4))):
                what = float(rng.choice([np.inf, -np.inf, np.nan]))
                h, e = int(rng.integers(batch.h)), int(rng.integers(128))
                if rng.random() < 0.2:
                    pool[blk, t % batch.bs, h] = what
                else:
                    pool[blk, t % batch.bs, h, e] = what
    k, v = batch.values()
    nan = np.isnan(v)
    return [k, np.where(np.isfinite(v), v, 0.0)], (v == np.inf) | nan, (v == -np.inf) | nan


def check_bad_values(batch, q, new, window, sink, rng, tokens, rows=80):
    caches, up, down = with_bad_values(batch, rng, tokens)
    out, starts = prefill(batch, q, new, window, sink)
    pick = sorted(rng.choice(sum(new), min(sum(new), rows), replace=False).tolist())
    ref = ow.prefill(q.double().numpy(), *caches, batch.tables, starts, batch.lens, window, sink, SCALE, set(pick))
    g = q.shape[1] // batch.h
    sees = np.zeros((2,) + tuple(q.shape), bool)  # whether a row's element has seen +inf, -inf
    for b, n in enumerate(batch.lens):
        for j in range(new[b]):
            i = int(starts[b]) + j
            if i not in set(pick):
                continue
            t = ow.visible(int(n) - new[b] + j, window, sink)
            blk = batch.tables[b][t // batch.bs] if len(t) else np.zeros(0, int)
            there = (blk >= 0) & (blk < up.shape[0])
            for s, x in zip(sees, (up, down)):
                s[i] = x[blk[there], t[there] % batch.bs].any(0).repeat(g, 0)
    got = out[pick].double().cpu().numpy()
    up, down = sees[0][pick], sees[1][pick]
    assert np.isnan(got[up & down]).all()
    assert (got[up & ~down] == np.inf).all() and (got[down & ~up] == -np.inf).all()
    good = ~(up | down)
    out_, mag, size, total = (x[pick] for x in ref)
    bound = 2.0 ** -8 * np.abs(out_) + (2.0 ** -15 * size[..., None] + 2.0 ** -8 + 2.0 ** -14) * mag \
        + 2.0 ** -24 * total[..., None]
    err = np.abs(np.where(good, got, 0.0) - np.where(good, out_, 0.0))
    assert np.isfinite(got[good]).all() and (err[good] <= bound[good]).all()
    return int((~good).sum()), int(good.sum())


@pytest.mark.parametrize("seed", range(16))
def test_prefill_values_that_are_not_finite(seed):
    """Single elements and whole heads of tokens, infinities of both signs and NaN: the elements of the rows
    that see them take them on, all others are as if they were 0."""
    rng = np.random.default_rng(500 + seed)
    h, g = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 4, 8, 16]))
    bs = int(rng.choice([8, 16, 64, 256]))
    window, sink = int(rng.choice([1, 30, 64, 200, 1000])), int(rng.choice([0, 1, 5, 70]))
    new = [int(x) for x in rng.integers(1, 500, 3)]
    lens = [n + int(rng.choice([0, 7, 300])) for n in new]
    batch = Batch(lens, h, bs, seed, drop=float(rng.choice([0, 0.1])))
    q = queries(sum(new), h * g, seed + 1)
    bad, good = check_bad_values(batch, q, new, window, sink, rng, int(rng.choice([1, 3, 10, 1000])))
    assert bad + good > 0


def test_prefill_values_that_are_not_finite_over_many_items():
    """Several items to a CTA, some of them marked; a scale below zero; more tokens than n."""
    rng = np.random.default_rng(7)
    lens, new = [3000, 90, 2500], [3000, 100, 1200]
    batch = Batch(lens, 4, 16, 31)
    bad, good = check_bad_values(batch, queries(sum(new), 16, 32), new, 700, 4, rng, 4, rows=120)
    assert bad > 0 and good > 0
    batch = Batch(lens, 8, 32, 33)
    bad, good = check_bad_values(batch, queries(sum(new), 8, 34), new, 5000, 0, rng, 2, rows=60)
    assert bad > 0 and good > 0


def test_a_value_that_is_not_finite_does_not_make_the_call_slow():
    """One infinite element in two prompts costs a few passes over the items at the edges of its
    visibility; when every row that sees it was made again by itself the call took 160 times as long."""
    need_gpu()
    n, window, h, hq, bs = 4096, 2048, 8, 32, 16
    gen = torch.Generator(device="cuda").manual_seed(1)
    kc, vc = (torch.randn((2 * n // bs, bs, h, 128), generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((2 * n, hq, 128), generator=gen, device="cuda").bfloat16()
    bt = torch.arange(2 * n // bs, dtype=torch.int32, device="cuda").view(2, -1)
    starts = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    out, err = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")

    def took():
        best = 1e9
        for _ in range(3):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            pa.pa_paged_window_prefill_attention(out, q, kc, vc, bt, starts, lens, window, 4, SCALE, n, err)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    took()
    clean = took()
    vc[1500 // bs, 1500 % bs, :, 7] = float("inf")
    one = took()
    assert int(err) == 0 and one < 10 * clean + 1.0, (clean, one)


def test_empty_batches():
    """No sequence, no token: the calls return and write nothing (torch gives such tensors no address)."""
    need_gpu()
    kc, vc = (torch.zeros((4, 16, 2, 128), dtype=BF16, device="cuda") for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = pa.window_decode_workspace(0, 8, 2, 128, 30, 4, 64)
    none = torch.zeros((0, 8, 128), dtype=BF16, device="cuda")
    pa.pa_paged_window_decode_attention(none.clone(), none, kc, vc, torch.zeros((0, 4), **i32), torch.zeros(0, **i32),
                                        30, 4, SCALE, 64, ws)
    err = torch.zeros(1, **i32)
    pa.pa_paged_window_prefill_attention(none.clone(), none, kc, vc, torch.zeros((2, 4), **i32),
                                         torch.zeros(3, **i32), torch.full((2,), 5, **i32), 30, 4, SCALE, 64, err)
    pa.pa_paged_window_prefill_attention(none.clone(), none, kc, vc, torch.zeros((0, 4), **i32),
                                         torch.zeros(1, **i32), torch.zeros(0, **i32), 30, 4, SCALE, 0, err)
    pa.pa_rope_and_cache(none.clone(), none, none[:, :2], none[:, :2], kc, vc, torch.zeros((8, 64), device="cuda"),
                         torch.zeros(0, dtype=torch.int64, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    assert int(err) == 0 and pa.read_device_error(ws) == 0 and not bool(kc.any() or vc.any())


@pytest.mark.parametrize("window,sink", [(1, 0), (50, 4), (300, 70), (5000, 0)])
def test_prompt_rows_and_decode_see_the_same_tokens(window, sink):
    """A prompt's rows beside the decode call's at the same positions: within the sum of both bounds."""
    n, picks = 420, [0, 1, 49, 50, 51, 63, 64, 200, 299, 300, 419]
    batch = Batch([n], 2, 16, 40)
    q = queries(n, 8, 41)
    x, _ = prefill(batch, q, [n], window, sink)
    # the same tokens as a batch of contexts that end at these positions
    batch.tables = np.repeat(batch.tables, len(picks), 0)
    batch.lens = np.array([p + 1 for p in picks], np.int32)
    y, _ = decode(batch, q[picks], window, sink)
    out, mag, size, total = ow.decode(q[picks].double().numpy(), *batch.values(), batch.tables, batch.lens, window, sink,
                                      SCALE)
    bound = 2.0 ** -7 * np.abs(out) + (2.0 ** -14 * size[..., None] + 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -13) * mag \
        + 2.0 ** -23 * total[..., None]
    assert (np.abs((x[picks].double() - y.double()).cpu().numpy()) <= bound).all()
