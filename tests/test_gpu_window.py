"""GPU tests of the window attention calls against plain attention in 64 bits.

Bounds, from the arithmetic.  delta = 2^-16 size, with size the largest of scale * sum |q_i k_i|
over a row's tokens, bounds a score's error: 128 products summed in fp32 (128 * 2^-24 of the size),
the factor scale log2(e) and exp2's argument (a few 2^-24 more).  A weight is then off by at most
2 delta of itself (its own score and the sum's), to first order, and by its rounding r: bf16
caches in decode carry it as two bf16 terms (2^-16), e4m3 caches as fp16 (2^-11, or 2^-25 of the
largest where it is subnormal), prefill as one bf16 (2^-8).  With mag = sum p |v| and
total = sum |v| the output, rounded to bf16 once more, is within
    2^-8 |ref| + (2 delta + r + 2^-14) mag + 2^-24 total
(2^-14: fp32 sums and divisions, and the second order of the terms before).
"""
import numpy as np
import pytest
import torch

from oracle import window as ow
from paged_kv_cache_309_gb300 import pa
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
SCALE = 128 ** -0.5


class Batch:
    """Caches whose unused rows are NaN, with shuffled blocks."""

    def __init__(self, lens, h, bs, seed=0, cache=BF16, scales=None, drop=0.0, spread=1.0):
        gen = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        need = [(n + bs - 1) // bs for n in lens]
        nb = sum(need) + 2
        perm = rng.permutation(nb)
        self.tables = np.full((len(lens), max(1, max(need))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = perm[at:at + n]
            at += n
        self.tables[rng.random(self.tables.shape) < drop] = nb + 5  # outside the pool
        self.lens, self.bs, self.h, self.scales = np.array(lens, np.int32), bs, h, scales
        self.pools = []
        for i in range(2):
            x = torch.randn((nb, bs, h, 128), generator=gen) * (spread if i == 0 else 1.0)
            if scales is not None:
                x = x / scales[i]
            x = x.to(cache)
            for b, n in enumerate(lens):  # rows past a sequence's end
                if n % bs and 0 <= self.tables[b, n // bs] < nb:
                    x[self.tables[b, n // bs], n % bs:] = float("nan")
            self.pools.append(x)

    def spoil(self, keep, value):
        """Sets every row of a sequence that keep(b, t) denies to `value`."""
        for b, n in enumerate(self.lens):
            for t in range(int(n)):
                blk = self.tables[b, t // self.bs]
                if 0 <= blk < self.pools[0].shape[0] and not keep(b, t):
                    for p in self.pools:
                        p[blk, t % self.bs] = value

    def values(self):
        f = self.scales or (1.0, 1.0)
        return [p.double().numpy() * np.float64(np.float32(s)) for p, s in zip(self.pools, f)]

    def device(self):
        return [p.cuda() for p in self.pools] + [torch.from_numpy(self.tables).cuda(),
                                                 torch.from_numpy(self.lens).cuda()]

    def scale_args(self):
        if self.scales is None:
            return {}
        k, v = (torch.tensor([s], device="cuda") for s in self.scales)
        return dict(k_scale=k, v_scale=v)


def queries(n, hq, seed, spread=1.0):
    return (torch.randn((n, hq, 128), generator=torch.Generator().manual_seed(seed)) * spread).bfloat16()


def compare(got, ref, r):
    out, mag, size, total = ref
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    bound = 2.0 ** -8 * np.abs(out) + (2.0 ** -15 * size[..., None] + r + 2.0 ** -14) * mag \
        + 2.0 ** -24 * total[..., None]
    err = np.abs(got - out)
    assert (err <= bound).all(), (err.max(), np.argwhere(err > bound)[:4])


def decode(batch, q, window, sink, most=None, ws=None, stream=None):
    need_gpu()
    hq = q.shape[1]
    most = int(batch.lens.max()) if most is None else most
    if ws is None:
        ws = pa.window_decode_workspace(len(batch.lens), hq, batch.h, 128, window, sink, most)
    k, v, bt, cl = batch.device()
    dq = q.cuda()
    out = torch.full_like(dq, float("nan"))
    torch.cuda.synchronize()
    pa.pa_paged_window_decode_attention(out, dq, k, v, bt, cl, window, sink, SCALE, most, ws,
                                        stream=stream, **batch.scale_args())
    torch.cuda.synchronize()
    return out, ws


def check_decode(lens, hq, h, bs, window, sink, r=2.0 ** -16, seed=0, spread=1.0, **kw):
    batch = Batch(lens, h, bs, seed, spread=spread, **kw)
    q = queries(len(lens), hq, seed + 1, spread)
    out, ws = decode(batch, q, window, sink)
    assert pa.read_device_error(ws) == 0
    ref = ow.decode(q.double().numpy(), *batch.values(), batch.tables, lens, window, sink, SCALE)
    compare(out, ref, r)


WINDOWS = [(1, 0), (1, 1), (2, 3), (16, 4), (33, 0), (64, 64), (100, 5), (128, 130), (1000, 4), (5000, 2), (7, 5000)]


@pytest.mark.parametrize("window,sink", WINDOWS)
@pytest.mark.parametrize("bs", [8, 16, 64, 256])
def test_decode_windows(window, sink, bs):
    check_decode([0, 1, 2, 17, 63, 64, 65, 300, 1001], 8, 4, bs, window, sink, seed=window + bs)


@pytest.mark.parametrize("hq,h", [(1, 1), (8, 8), (8, 2), (16, 2), (16, 1), (48, 3)])
@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_decode_groups(hq, h, cache):
    check_decode([700, 33, 0, 128], hq, h, 16, 200, 4, seed=hq, cache=cache,
                 r=2.0 ** -16 if cache == BF16 else 2.0 ** -11)


@pytest.mark.parametrize("window,sink", WINDOWS)
def test_decode_e4m3_with_scales(window, sink):
    check_decode([1, 64, 500, 900], 16, 4, 32, window, sink, r=2.0 ** -11, seed=window, cache=E4M3,
                 scales=(0.05, 0.3))


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_decode_dropped_blocks(cache):
    check_decode([700, 900, 40, 3], 8, 2, 16, 300, 20, seed=5, cache=cache, drop=0.3,
                 r=2.0 ** -16 if cache == BF16 else 2.0 ** -11)
    check_decode([700, 900], 8, 2, 64, 300, 20, seed=6, cache=cache, drop=1.1,
                 r=2.0 ** -16 if cache == BF16 else 2.0 ** -11)  # nothing is there: zero rows


def test_decode_sharp_scores():
    check_decode([2000, 777], 8, 2, 16, 900, 4, seed=7, spread=3.0)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_decode_rows_outside_the_window_do_not_count(value, cache):
    lens, window, sink = [500, 129, 90], 70, 5
    a, b = Batch(lens, 2, 16, 8, cache=cache), Batch(lens, 2, 16, 8, cache=cache)
    b.spoil(lambda s, t: t >= lens[s] - window or t < sink, value if cache == BF16 else float("nan"))
    q = queries(3, 8, 9)
    x, y = decode(a, q, window, sink)[0], decode(b, q, window, sink)[0]
    assert bool((x == y).all())


def test_decode_blocks_behind_the_window_may_be_gone():
    lens, window, sink = [1000, 640], 200, 3
    a = Batch(lens, 2, 16, 10)
    q = queries(2, 8, 11)
    x = decode(a, q, window, sink)[0]
    for b, n in enumerate(lens):
        a.tables[b, 1:(n - window) // 16] = -1
    assert bool((x == decode(a, q, window, sink)[0]).all())


def test_decode_splits_of_a_wide_window():
    """One sequence whose window is split over many CTAs, with its lengths around the cuts."""
    for n in (8191, 8192, 8193, 9001):
        check_decode([n], 8, 1, 16, 8000, 64, seed=n)


def test_decode_clips_and_flags():
    batch = Batch([300, 100], 2, 16, 12)
    q = queries(2, 4, 13)
    out, ws = decode(batch, q, 50, 4, most=200)
    assert pa.read_device_error(ws) == pa.PA_DEVERR_CONTEXT_CLIPPED
    ref = ow.decode(q.double().numpy(), *batch.values(), batch.tables, [200, 100], 50, 4, SCALE)
    compare(out, ref, 2.0 ** -16)
    batch.tables = np.ascontiguousarray(batch.tables[:, :10])  # the table ends first
    batch.lens = np.array([300, 100], np.int32)
    out, ws = decode(batch, q, 50, 4, most=400)
    assert pa.read_device_error(ws) == pa.PA_DEVERR_CONTEXT_CLIPPED
    ref = ow.decode(q.double().numpy(), *batch.values(), batch.tables, [160, 100], 50, 4, SCALE)
    compare(out, ref, 2.0 ** -16)


def test_decode_widest_window_is_the_plain_call():
    batch = Batch([513, 64, 1, 0], 4, 16, 14)
    q = queries(4, 16, 15)
    x, _ = decode(batch, q, 2 ** 31 - 1, 2 ** 31 - 1)
    k, v, bt, cl = batch.device()
    out = torch.empty_like(x)
    pa.pa_paged_decode_attention(out, q.cuda(), k, v, bt, cl, SCALE, 513, pa.decode_workspace(4, 16, 4, 128, 513))
    ref = ow.decode(q.double().numpy(), *batch.values(), batch.tables, batch.lens, 1000, 0, SCALE)
    compare(x, ref, 2.0 ** -16)
    compare(out, ref, 2.0 ** -16)


def test_decode_stream_graph_and_shared_workspace():
    batch = Batch([900, 2000], 2, 16, 16)
    q = queries(2, 8, 17)
    x, ws = decode(batch, q, 600, 4)
    y, _ = decode(batch, q, 600, 4, ws=ws, stream=torch.cuda.Stream())
    assert bool((x == y).all())
    z = decode(batch, q, 37, 4, most=2000)[0]
    k, v, bt, cl = batch.device()
    outs, dq = [torch.zeros_like(x) for _ in range(2)], q.cuda()
    graphs = []
    for out, window in zip(outs, (600, 37)):  # two graphs that share the workspace, on one stream
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_paged_window_decode_attention(out, dq, k, v, bt, cl, window, 4, SCALE, 2000, ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert bool((outs[0] == x).all()) and bool((outs[1] == z).all())
    lens = [899, 1999]
    cl.copy_(torch.tensor(lens, dtype=torch.int32))  # a replay takes the lengths as they are then
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for out, window in zip(outs, (600, 37)):
        compare(out, ow.decode(q.double().numpy(), *batch.values(), batch.tables, lens, window, 4, SCALE), 2.0 ** -16)


# ---------------------------------------------------------------- prefill --
def prefill(batch, q, new, window, sink, rows=None, stream=None):
    need_gpu()
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k, v, bt, cl = batch.device()
    dq = q.cuda()
    out = torch.full_like(dq, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    pa.pa_paged_window_prefill_attention(out, dq, k, v, bt, torch.from_numpy(starts).cuda(), cl, window, sink,
                                         SCALE, max(new), err, stream=stream)
    torch.cuda.synchronize()
    assert int(err) == 0
    return out, starts


def check_prefill(lens, new, hq, h, bs, window, sink, seed=0, spread=1.0, sample=None, **kw):
    batch = Batch(lens, h, bs, seed, spread=spread, **kw)
    q = queries(sum(new), hq, seed + 1, spread)
    out, starts = prefill(batch, q, new, window, sink)
    rows = None
    if sample is not None:
        rows = set(np.random.default_rng(seed).choice(sum(new), sample, replace=False).tolist())
        rows |= {int(s) for s in starts[:-1]} | {int(s) - 1 for s in starts[1:]}
    ref = ow.prefill(q.double().numpy(), *batch.values(), batch.tables, starts, lens, window, sink, SCALE, rows)
    pick = slice(None) if rows is None else sorted(rows)
    compare(out[pick], [x[pick] for x in ref], 2.0 ** -8)


@pytest.mark.parametrize("window,sink", WINDOWS)
@pytest.mark.parametrize("bs", [16, 64])
def test_prefill_windows(window, sink, bs):
    check_prefill([1, 40, 300, 333], [1, 40, 300, 33], 8, 2, bs, window, sink, seed=window + bs)


@pytest.mark.parametrize("hq,h", [(1, 1), (4, 2), (8, 2), (16, 2), (16, 1)])
def test_prefill_groups(hq, h):
    check_prefill([500, 260], [200, 260], hq, h, 16, 130, 4, seed=hq)


@pytest.mark.parametrize("bs", [8, 32, 128, 256])
@pytest.mark.parametrize("window,sink", [(50, 0), (200, 30), (301, 140)])
def test_prefill_block_sizes(bs, window, sink):
    check_prefill([700, 129], [290, 129], 4, 2, bs, window, sink, seed=bs + window)


def test_prefill_long():
    check_prefill([4000, 2500], [4000, 700], 8, 2, 16, 1000, 4, seed=3, sample=60)
    check_prefill([6000], [600], 4, 1, 16, 77, 260, seed=4, sample=60)


def test_prefill_dropped_blocks_and_sharp_scores():
    check_prefill([300, 200], [150, 200], 4, 2, 16, 90, 20, seed=5, drop=0.3)
    check_prefill([300], [150], 4, 2, 64, 90, 20, seed=6, drop=1.1)
    check_prefill([600], [400], 4, 2, 16, 250, 4, seed=7, spread=3.0)


def test_prefill_rows_before_the_sequence_and_behind_the_last():
    """n > L: rows before position 0 are zero; rows of q behind the last sequence are left as they were."""
    lens, new = [5, 0, 40], [9, 3, 40]
    batch = Batch(lens, 2, 16, 8)
    q = queries(60, 4, 9)
    out, starts = prefill(batch, q, new, 8, 2)
    ref = ow.prefill(q.double().numpy(), *batch.values(), batch.tables, starts, lens, 8, 2, SCALE)
    compare(out[:52], [x[:52] for x in ref], 2.0 ** -8)
    assert bool((out[:4] == 0).all()) and bool((out[9:12] == 0).all()) and bool((out[52:] == 7).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["k", "v", "kv"])
def test_prefill_rows_that_are_not_seen_do_not_count(value, which):
    """Single tokens that are not finite, in the middle of tiles: rows that see one are not finite
    either, all others are what they are without them."""
    lens, new, window, sink = [500, 300], [400, 300], 90, 4
    bad = {0: (120, 250, 430), 1: (150, 2)}
    batch, clean = Batch(lens, 2, 16, 10), Batch(lens, 2, 16, 10)
    batch.spoil(lambda b, t: t not in bad[b], value)
    if which != "kv":
        batch.pools["vk".index(which)] = clean.pools["vk".index(which)]
    q = queries(sum(new), 8, 11)
    out, starts = prefill(batch, q, new, window, sink)
    ref = ow.prefill(q.double().numpy(), *clean.values(), clean.tables, starts, lens, window, sink, SCALE)
    unseen = [int(starts[b]) + j for b in range(2) for j in range(new[b])
              if not set(bad[b]) & set(ow.visible(lens[b] - new[b] + j, window, sink).tolist())]
    seen = [i for i in range(sum(new)) if i not in unseen]
    assert len(unseen) > 100 and len(seen) > 400
    compare(out[unseen], [x[unseen] for x in ref], 2.0 ** -8)
    assert not np.isfinite(out[seen].double().cpu().numpy()).any()


def test_prefill_widest_window_is_the_plain_call():
    batch = Batch([400, 64], 2, 16, 12)
    q = queries(364, 8, 13)
    x, starts = prefill(batch, q, [300, 64], 2 ** 31 - 1, 2 ** 31 - 1)
    k, v, bt, cl = batch.device()
    out, err = torch.empty_like(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_paged_prefill_attention(out, q.cuda(), k, v, bt, torch.from_numpy(starts).cuda(), cl, SCALE, 300, err)
    ref = ow.prefill(q.double().numpy(), *batch.values(), batch.tables, starts, batch.lens, 1000, 0, SCALE)
    compare(x, ref, 2.0 ** -8)
    compare(out, ref, 2.0 ** -8)


def test_prefill_stream_and_graph():
    batch = Batch([200, 150], 2, 16, 14)
    q = queries(250, 8, 15)
    x, starts = prefill(batch, q, [100, 150], 60, 4)
    y, _ = prefill(batch, q, [100, 150], 60, 4, stream=torch.cuda.Stream())
    assert bool((x == y).all())
    k, v, bt, cl = batch.device()
    dq, st = q.cuda(), torch.from_numpy(starts).cuda()
    out, err = torch.zeros_like(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_paged_window_prefill_attention(out, dq, k, v, bt, st, cl, 60, 4, SCALE, 150, err)
    g.replay()
    torch.cuda.synchronize()
    assert bool((x == out).all())


# ------------------------------------------------------------ used together --
def test_a_prompt_and_the_tokens_after_it():
    """A prompt rotated, appended and attended to in two chunks, then tokens one by one, on one cache:
    every output is that of plain attention over the rotated rows; the caches hold those rows."""
    need_gpu()
    H, HQ, bs, n, window, sink = 2, 8, 16, 150, 40, 3
    prompt, rot = 130, 64
    gen = torch.Generator().manual_seed(20)
    wide = torch.randn((n, (HQ + 2 * H) * 128), generator=gen).bfloat16()
    angle = np.arange(256)[:, None] * 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    table = np.random.default_rng(21).permutation(12).astype(np.int32)[None]
    dev, dcs = wide.cuda(), torch.from_numpy(cs).cuda()
    kc, vc = (torch.full((12, bs, H, 128), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    bt = torch.from_numpy(table).cuda()
    pos = torch.arange(n, device="cuda")
    slot = bt[0].long()[pos // bs] * bs + pos % bs
    q = torch.empty((n, HQ, 128), dtype=BF16, device="cuda")
    out = torch.empty_like(q)
    ws = pa.window_decode_workspace(1, HQ, H, 128, window, sink, n)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append(a, b):
        x = dev[a:b]
        parts = [x[:, i * 128:j * 128].unflatten(1, (j - i, 128)) for i, j in ((0, HQ), (HQ, HQ + H), (HQ + H, HQ + 2 * H))]
        pa.pa_rope_and_cache(q[a:b], *parts, kc, vc, dcs, pos[a:b], slot[a:b])

    for a, b in ((0, 70), (70, prompt)):
        append(a, b)
        pa.pa_paged_window_prefill_attention(
            out[a:b], q[a:b], kc, vc, bt, torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
            torch.tensor([b], dtype=torch.int32, device="cuda"), window, sink, SCALE, b - a, err)
    for t in range(prompt, n):
        append(t, t + 1)
        pa.pa_paged_window_decode_attention(out[t:t + 1], q[t:t + 1], kc, vc, bt,
                                            torch.tensor([t + 1], dtype=torch.int32, device="cuda"), window, sink,
                                            SCALE, n, ws)
    torch.cuda.synchronize()
    assert int(err) == 0 and pa.read_device_error(ws) == 0
    host = wide.float().numpy().reshape(n, HQ + 2 * H, 128)
    turned, size = ow.rotate(host[:, :HQ + H], cs, np.arange(n), False)
    at = slot.cpu().numpy()
    pools = [c.double().cpu().numpy() for c in (kc, vc)]
    rows = [p.reshape(-1, H, 128)[at] for p in pools]
    assert (np.abs(q.double().cpu().numpy() - turned[:, :HQ]) <= 2.0 ** -8 * np.abs(turned[:, :HQ])
            + 2.0 ** -22 * size[:, :HQ]).all()
    assert (np.abs(rows[0] - turned[:, HQ:]) <= 2.0 ** -8 * np.abs(turned[:, HQ:]) + 2.0 ** -22 * size[:, HQ:]).all()
    assert (rows[1] == host[:, HQ + H:]).all()
    ref = ow.prefill(q.double().cpu().numpy(), *pools, table, [0, n], [n], window, sink, SCALE)
    compare(out[:prompt], [x[:prompt] for x in ref], 2.0 ** -8)
    compare(out[prompt:], [x[prompt:] for x in ref], 2.0 ** -16)
