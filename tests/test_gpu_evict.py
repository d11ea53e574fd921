"""GPU parity of eviction: which tokens are kept and where their rows go.
Everything here is whole numbers and copies, so it is compared exactly."""
import numpy as np
import pytest
import torch

from oracle import long_context as lc
from paged_kv_cache_309_gb300 import pa
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def kept_sums(sums, keep, new):
    out = np.full(sums.shape, -7.0, np.float32)
    for b in range(sums.shape[0]):
        for g in range(sums.shape[1]):
            out[b, g, :new[b]] = sums[b, g, keep[b, g, :new[b]]]
    return out


def run_select(sums, lens, budget, sink, recent, out="apart"):
    need_gpu()
    B, H, T = sums.shape
    s = torch.from_numpy(sums).cuda()
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    keep = torch.full((B, H, budget), -99, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -99, dtype=torch.int32, device="cuda")
    dst = {"apart": torch.full_like(s, -7.0), "same": s, "none": None}[out]
    pa.pa_evict_select(keep, new, dst, s, cl, budget, sink, recent)
    torch.cuda.synchronize()
    if out != "same":
        assert (s.cpu().numpy().view(np.uint32) == sums.view(np.uint32)).all()
    return keep.cpu().numpy(), new.cpu().numpy(), None if dst is None else dst.cpu().numpy()


def check_select(sums, lens, budget, sink=0, recent=0, out="apart"):
    keep, new, got = run_select(sums, lens, budget, sink, recent, out)
    want, want_new = lc.evict_select(sums, lens, budget, sink, recent)
    assert (new == want_new).all()
    assert (keep == want).all()
    if got is not None:
        ref = kept_sums(sums, want, want_new)
        if out == "same":  # behind the kept the array is as it was
            for b in range(len(lens)):
                ref[b, :, want_new[b]:] = sums[b, :, want_new[b]:]
        assert ((got == ref) | (np.isnan(got) & np.isnan(ref))).all()


def random_sums(shape, seed, kind="weights"):
    rng = np.random.default_rng(seed)
    x = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        x = rng.integers(0, 4, shape).astype(np.float32)
    if kind == "special":
        pick = rng.integers(0, 9, shape)
        vals = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, -1.0, 1e-40, 3.4e38, -np.nan], np.float32)
        x = vals[pick]
    if kind == "signed":
        x = rng.standard_normal(shape).astype(np.float32)
    return x


@pytest.mark.parametrize("out", ["apart", "same", "none"])
@pytest.mark.parametrize("kind", ["weights", "ties", "special", "signed"])
def test_select_small(kind, out):
    sums = random_sums((9, 3, 90), 1, kind)
    lens = [0, 1, 31, 32, 33, 64, 89, 90, 77]
    for budget, sink, recent in ((32, 0, 0), (32, 4, 8), (1, 0, 0), (1, 1, 0), (1, 0, 1),
                                 (32, 16, 16), (90, 3, 3), (200, 0, 100)):
        check_select(sums, lens, budget, sink, recent, out)


@pytest.mark.parametrize("T", [1, 2, 1023, 1024, 1025, 5000, 20011])
@pytest.mark.parametrize("out", ["apart", "same"])
def test_select_lengths(T, out):
    for kind in ("weights", "ties"):
        sums = random_sums((2, 2, T), T, kind)
        check_select(sums, [T, max(0, T - 3)], max(1, T // 3), min(2, T // 6), T // 9, out)


@pytest.mark.parametrize("T", [70001, 131072, 300000])
def test_select_long(T):
    sums = random_sums((1, 1, T), T)
    sums[random_sums((1, 1, T), T + 1) < 0.5] = 0
    check_select(sums, [T], T // 4, 16, 1024, "same")
    check_select(np.zeros((1, 1, T), np.float32), [T], T // 2, 0, 64)
    check_select(random_sums((1, 1, T), 5, "signed"), [T - 77], T - 100, 0, 0)


def test_select_lengths_out_of_range():
    sums = random_sums((4, 2, 50), 3)
    check_select(sums, [-5, 51, 2 ** 31 - 1, -2 ** 31], 20, 2, 2)


def test_select_equal_high_digits():
    """Keys that differ in their last bits only."""
    base = np.float32(1.5).view(np.uint32) + np.random.default_rng(1).permutation(3000).astype(np.uint32)
    sums = base.view(np.float32).reshape(1, 1, 3000)
    check_select(sums, [3000], 1234)


def test_select_many_rows():
    sums = random_sums((70, 5, 300), 4)
    check_select(sums, np.random.default_rng(1).integers(0, 301, 70).tolist(), 100, 4, 20, "same")


# ----------------------------------------------------------------- compact --
TYPES = {"bf16": (torch.bfloat16, 128), "e4m3": (torch.float8_e4m3fn, 128), "q4": (torch.uint8, 80),
         "fp32": (torch.float32, 64), "latent": (torch.bfloat16, 576), "one": (torch.uint8, 16),
         "wide": (torch.uint8, 16 * 37)}


def pools(nb, bs, H, kind, seed):
    t, row = TYPES[kind]
    size = torch.empty(0, dtype=t).element_size()
    g = torch.Generator().manual_seed(seed)
    raw = [torch.randint(0, 256, (nb, bs, H, row * size), generator=g, dtype=torch.uint8)
           for _ in range(2)]
    return [r.cuda().view(t) for r in raw], [r.numpy().copy() for r in raw]


def ascending(B, H, n, L, seed):
    rng = np.random.default_rng(seed)
    keep = np.full((B, H, n), -1, np.int32)
    for b in range(B):
        for g in range(H):
            m = min(n, L[b])
            keep[b, g, :m] = np.sort(rng.permutation(L[b])[:m])
    return keep


def run_compact(kind, keep, keep_lens, src, dst, nb, bs, key_only=False, seed=0):
    need_gpu()
    H = keep.shape[1]
    (k, v), (kh, vh) = pools(nb, bs, H, kind, seed)
    st = torch.from_numpy(src).cuda()
    dt = st if dst is src else torch.from_numpy(dst).cuda()
    pa.pa_cache_compact(k, None if key_only else v, torch.from_numpy(keep).cuda(),
                        torch.tensor(keep_lens, dtype=torch.int32).cuda(), st, dt)
    torch.cuda.synchronize()
    lc.compact(kh, keep, keep_lens, src, dst)
    if not key_only:
        lc.compact(vh, keep, keep_lens, src, dst)
    assert (k.view(torch.uint8).cpu().numpy() == kh).all()
    assert (v.view(torch.uint8).cpu().numpy() == vh).all()


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("bs", [1, 8, 12, 16, 256])
def test_compact(kind, bs, in_place):
    L, n, H = [700, 513, 1, 0, 90], 512, 1 if kind == "latent" else 3
    rng = np.random.default_rng(bs)
    need = [(x + bs - 1) // bs for x in L]
    out = [(min(x, n) + bs - 1) // bs for x in L]
    nb = sum(need) + sum(out) + 2
    perm = rng.permutation(nb).astype(np.int32)
    src = np.full((5, max(need) + 1), -1, np.int32)
    dst = np.full((5, max(out)), -1, np.int32)
    at = 0
    for b in range(5):
        src[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        dst[b, :out[b]] = perm[at:at + out[b]]
        at += out[b]
    keep = ascending(5, H, n, L, bs)
    lens = [min(x, n) for x in L]
    run_compact(kind, keep, lens, src, src if in_place else dst, nb, bs,
                key_only=kind == "latent", seed=bs)


def test_compact_long_in_place():
    """Many chunks: rows move a little, a lot, and not at all."""
    for drop in (1, 50, 4000, 7000):
        L = 8192
        rng = np.random.default_rng(drop)
        keep = np.sort(rng.permutation(L)[:L - drop]).astype(np.int32)[None, None].repeat(2, 1)
        src = rng.permutation(L // 16).astype(np.int32)[None]
        run_compact("bf16", keep, [L - drop], src, src, L // 16, 16, seed=drop)


def test_compact_skips_what_is_out_of_range():
    rng = np.random.default_rng(0)
    src = rng.permutation(40).astype(np.int32)[:20].reshape(2, 10)
    dst = np.setdiff1d(np.arange(40), src).astype(np.int32)[:10].reshape(2, 5)
    src[0, 3], src[1, 2], dst[0, 1], dst[1, 4] = -1, 40, 2 ** 31 - 1, -2 ** 31
    keep = rng.integers(-5, 200, (2, 3, 100)).astype(np.int32)
    keep[0, 0, 5], keep[1, 1, 7] = 2 ** 31 - 1, -2 ** 31
    run_compact("q4", keep, [1000, -3], src, dst, 40, 16)
    run_compact("q4", keep, [77, 100], src, dst, 40, 16)


def test_compact_leaves_unowned_rows():
    """In place, rows behind the kept and other sequences' blocks are as they were."""
    src = np.array([[3, 1, 4], [5, 9, 2]], np.int32)
    keep = ascending(2, 2, 20, [40, 0], 1)
    run_compact("bf16", keep, [20, 0], src, src, 10, 16)
    run_compact("bf16", keep, [0, 0], src, src, 10, 16)


# ----------------------------------------------------- the set, as it is used --
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("cache", ["q4", "bf16"])
def test_write_attend_evict_attend(cache, in_place):
    """A prompt is written, three tokens are decoded with their weights added
    up, the light tokens are evicted, and decoding goes on over what is left:
    its outputs are the oracle's over the kept tokens."""
    need_gpu()
    B, H, G, D, bs, budget = 2, 2, 4, 128, 16, 96
    start, steps = [203, 130], 3
    gen = torch.Generator(device="cuda").manual_seed(3)
    nb = 64
    perm = torch.randperm(nb, generator=gen, device="cuda").int()
    table, new_table = perm[:32].view(B, 16).contiguous(), perm[32:44].view(B, 6).contiguous()
    if cache == "q4":
        kc, vc = (torch.zeros(nb, bs, H, 80, dtype=torch.uint8, device="cuda") for _ in range(2))
        write = pa.pa_reshape_and_cache_q4
    else:
        kc, vc = (torch.zeros(nb, bs, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        write = pa.pa_reshape_and_cache

    def values(c):
        return lc.q4_restore(c.cpu().numpy()) if cache == "q4" else c.cpu().double().numpy()

    def put(b, first, n, tab):
        x = torch.randn(2, n, H, D, generator=gen, device="cuda").bfloat16()
        t = torch.arange(first, first + n, device="cuda")
        write(x[0], x[1], kc, vc, tab[b, t // bs].long() * bs + t % bs)

    for b in range(B):
        put(b, 0, start[b], table)
    T = 256
    sums = torch.zeros(B, H, T, device="cuda")
    ws = pa.decode_scored_workspace(B, H * G, H, D, T)
    want = np.zeros((B, H, T))
    lens = np.array(start)
    for step in range(steps):
        lens = lens + 1
        for b in range(B):
            put(b, int(lens[b]) - 1, 1, table)
        cl = torch.from_numpy(lens.astype(np.int32)).cuda()
        q = torch.randn(B, H * G, D, generator=gen, device="cuda").bfloat16()
        out = torch.empty_like(q)
        pa.pa_paged_decode_attention_scored(out, sums, sums, 1 << 30 if step == 0 else 1, q, kc, vc,
                                            table, cl, D ** -0.5, T, ws)
        _, w = lc.decode(q.cpu().double().numpy(), values(kc), values(vc), table.cpu().numpy(), lens,
                         bs, D ** -0.5)
        for b in range(B):
            want[b, :, :lens[b]] += w[b, :, :lens[b]]
    got = sums.cpu().double().numpy()
    assert (np.abs(got - want) <= 2.0 ** -12 * want).all()

    old_k, old_v = values(kc), values(vc)
    old_table, old_sums = table.cpu().numpy(), sums.cpu().numpy()
    keep = torch.empty(B, H, budget, dtype=torch.int32, device="cuda")
    new_lens = torch.empty(B, dtype=torch.int32, device="cuda")
    pa.pa_evict_select(keep, new_lens, sums, sums, cl, budget, 4, 16)
    tab = table if in_place else new_table
    pa.pa_cache_compact(kc, vc, keep, new_lens, table, tab)
    ref_keep, _ = lc.evict_select(old_sums, lens, budget, 4, 16)
    assert (keep.cpu().numpy() == ref_keep).all() and (new_lens == budget).all()
    assert (sums[:, :, :budget].cpu().numpy() == np.take_along_axis(old_sums, ref_keep, 2)).all()

    q = torch.randn(B, H * G, D, generator=gen, device="cuda").bfloat16()
    out = torch.empty_like(q)
    pa.pa_paged_decode_attention_scored(out, sums, sums, 0, q, kc, vc, tab, new_lens, D ** -0.5, T, ws)
    assert pa.read_device_error(ws) == 0
    for b in range(B):
        for g in range(H):
            t = ref_keep[b, g]
            k = old_k[old_table[b, t // bs], t % bs, g]
            v = old_v[old_table[b, t // bs], t % bs, g]
            qs = q[b, g * G:(g + 1) * G].cpu().double().numpy()
            s = qs @ k.T * D ** -0.5
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            ref = p @ v
            err = out[b, g * G:(g + 1) * G].cpu().double().numpy() - ref
            # bf16 outputs of rounded weights and values: as for the decode call alone
            assert (np.abs(err) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * 20).all()
            add = old_sums[b, g, t] + p.sum(0)
            assert (np.abs(sums[b, g, :budget].cpu().numpy() - add) <= 2.0 ** -12 * add).all()


def test_captured_selection_and_move():
    need_gpu()
    B, H, T, budget, bs = 2, 2, 600, 200, 16
    sums = torch.from_numpy(random_sums((B, H, T), 8)).cuda()
    lens = torch.tensor([600, 100], dtype=torch.int32, device="cuda")
    keep = torch.empty(B, H, budget, dtype=torch.int32, device="cuda")
    new = torch.empty(B, dtype=torch.int32, device="cuda")
    (k, v), (kh, vh) = pools(100, bs, H, "bf16", 9)
    table = torch.randperm(100)[:76].view(2, 38).int().cuda()
    dst = torch.empty_like(sums)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_evict_select(keep, new, dst, sums, lens, budget, 4, 30)
        pa.pa_cache_compact(k, v, keep, new, table, table)
    lens.copy_(torch.tensor([401, 333], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    want, want_new = lc.evict_select(sums.cpu().numpy(), [401, 333], budget, 4, 30)
    assert (keep.cpu().numpy() == want).all() and (new.cpu().numpy() == want_new).all()
    lc.compact(kh, want, want_new, table.cpu().numpy(), table.cpu().numpy())
    assert (k.view(torch.uint8).cpu().numpy() == kh).all()


def test_sequential_prefix_feeds_prefill():
    """A cached 4-bit prefix read back to a bf16 cache gives the prefill attention its context."""
    need_gpu()
    H, G, D, bs, n, new = 2, 4, 128, 16, 150, 40
    x = torch.randn(2, n, H, D, device="cuda").bfloat16()
    kc, vc = (torch.zeros(20, bs, H, 80, dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.randperm(320, device="cuda")[:n]
    pa.pa_reshape_and_cache_q4(x[0], x[1], kc, vc, slots)
    stage = [torch.zeros(12, bs, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pa.pa_gather_cache_q4(stage[0].view(-1, H, D)[:n], stage[1].view(-1, H, D)[:n], kc, vc, slots)
    y = torch.randn(2, new, H, D, device="cuda").bfloat16()
    pa.pa_reshape_and_cache(y[0], y[1], *stage, torch.arange(n, n + new, device="cuda"))
    q = torch.randn(new, H * G, D, device="cuda").bfloat16()
    out, err = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_paged_prefill_attention(out, q, *stage, torch.arange(12, dtype=torch.int32, device="cuda")[None],
                                  torch.tensor([0, new], dtype=torch.int32, device="cuda"),
                                  torch.tensor([n + new], dtype=torch.int32, device="cuda"),
                                  D ** -0.5, new, err)
    assert int(err) == 0
    flat = slots.cpu().numpy()
    k = np.concatenate([lc.q4_restore(kc.cpu().numpy().reshape(-1, H, 80)[flat]), y[0].cpu().double().numpy()])
    v = np.concatenate([lc.q4_restore(vc.cpu().numpy().reshape(-1, H, 80)[flat]), y[1].cpu().double().numpy()])
    qs = q.cpu().double().numpy()
    for h in range(H * G):
        s = qs[:, h] @ k[:, h // G].T * D ** -0.5
        s[np.arange(n + new)[None] > n + np.arange(new)[:, None]] = -np.inf
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        ref = p @ v[:, h // G]
        got = out[:, h].cpu().double().numpy()
        # keys rounded to bf16 on the way (2^-8 of |k|): a score is off by its sum over 128
        # elements, |dk . q| scale < 2^-8 |k| |q| scale < 0.06 at most and far less on average;
        # the norm of the outputs is within a percent
        assert np.linalg.norm(got - ref) <= 1e-2 * np.linalg.norm(ref)


@pytest.mark.parametrize("T", [16384, 16385, 65537, 393216, 393217])
def test_select_at_the_cluster_sizes(T):
    """Row lengths where the number of CTAs per row changes, and beyond what a cluster holds."""
    sums = random_sums((2, 1, T), T, "weights")
    sums[:, :, ::3] = 0.5  # many ties
    check_select(sums, [T, T - 5000], T // 2 + 3, 7, 100, "same")
    check_select(sums, [T - 1, 40], 64, 4, 8)
