"""GPU parity of the choice over tables with dropped blocks, exact, and the set
as it is used with them: decode with weights, choose, move, decode on."""
import numpy as np
import pytest
import torch

from oracle import long_context as lc
from paged_kv_cache_309_gb300 import pa
from tests.gpu_util import need_gpu
from tests.test_gpu_evict import kept_sums, random_sums
from tests.test_gpu_q4_decode import D
from tests.test_gpu_scored_decode import batch

pytestmark = pytest.mark.gpu


def holed(lens, bs, share, seed, nb=1000, cols=None):
    """A table in which `share` of the blocks are dropped, in each way that can be."""
    rng = np.random.default_rng(seed)
    cols = max(1, max((max(0, min(n, 1 << 20)) + bs - 1) // bs for n in lens)) if cols is None else cols
    table = rng.integers(0, nb, (len(lens), cols)).astype(np.int32)
    bad = rng.choice(np.array([-1, nb, 2 ** 31 - 1, -2 ** 31], np.int32), table.shape)
    return np.where(rng.random(table.shape) < share, bad, table).astype(np.int32), nb


def check(sums, lens, budget, sink, recent, table, bs, nb, out="apart"):
    need_gpu()
    B, H, T = sums.shape
    s = torch.from_numpy(sums).cuda()
    keep = torch.full((B, H, budget), -99, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -99, dtype=torch.int32, device="cuda")
    dst = {"apart": torch.full_like(s, -7.0), "same": s, "none": None}[out]
    pa.pa_evict_select_paged(keep, new, dst, s, torch.tensor(lens, dtype=torch.int32).cuda(),
                             torch.from_numpy(table).cuda(), budget, sink, recent, bs, nb)
    torch.cuda.synchronize()
    want, want_new = lc.evict_select(sums, lens, budget, sink, recent, table, bs, nb)
    assert (new.cpu().numpy() == want_new).all()
    assert (keep.cpu().numpy() == want).all()
    if dst is None:
        return
    ref, got = kept_sums(sums, want, want_new), dst.cpu().numpy()
    if out == "same":
        for b in range(B):
            ref[b, :, want_new[b]:] = sums[b, :, want_new[b]:]
    assert ((got == ref) | (np.isnan(got) & np.isnan(ref))).all()


@pytest.mark.parametrize("out", ["apart", "same", "none"])
@pytest.mark.parametrize("kind", ["weights", "ties", "special", "signed"])
@pytest.mark.parametrize("bs", [1, 8, 12, 64])
@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_small(kind, out, bs, share):
    sums = random_sums((9, 3, 90), 1, kind)
    lens = [0, 1, 31, 32, 33, 64, 89, 90, 77]
    table, nb = holed(lens, bs, share, bs)
    for budget, sink, recent in ((32, 0, 0), (32, 4, 8), (1, 0, 0), (1, 1, 0), (1, 0, 1), (32, 16, 16),
                                 (90, 3, 3), (200, 0, 100)):
        check(sums, lens, budget, sink, recent, table, bs, nb, out)


def test_nan_sums_of_every_payload_are_tokens():
    sums = np.full((1, 2, 64), 0xFFFFFFFF, np.uint32).view(np.float32)
    sums[0, 0, 40:] = -np.inf
    table, nb = holed([64], 8, 0.4, 5)
    for budget in (5, 20, 64):
        check(sums, [64], budget, 1, 1, table, 8, nb)


@pytest.mark.parametrize("T", [16384, 16385, 65537, 393216, 393217])
def test_row_lengths(T):
    """Where the number of CTAs per row changes, and beyond what a cluster holds."""
    sums = random_sums((2, 1, T), T)
    sums[:, :, ::3] = 0.5
    lens = [T, T - 5000]
    table, nb = holed(lens, 16, 0.3, T)
    check(sums, lens, T // 2 + 3, 7, 100, table, 16, nb, "same")
    check(sums, lens, T, 7, 100, table, 16, nb)  # all that have a row
    check(sums, [T - 1, 40], 64, 4, 8, table, 16, nb)
    check(sums, lens, 64, 4, 8, np.full_like(table, -1), 16, nb)


def test_many_equal_first_digits():
    sums = np.full((1, 1, 20000), 1.5, np.float32)
    table, nb = holed([20000], 16, 0.3, 9)
    check(sums, [20000], 9000, 10, 10, table, 16, nb)


def test_lengths_and_tables_out_of_range():
    sums = random_sums((4, 2, 50), 3)
    lens = [-5, 51, 2 ** 31 - 1, -2 ** 31]
    table, nb = holed([50] * 4, 16, 0.2, 4, cols=2)  # 32 tokens of table for 50
    check(sums, lens, 40, 2, 2, table, 16, nb)
    check(sums, lens, 20, 2, 2, table, 2 ** 31 - 1, nb)
    check(sums, lens, 20, 2, 2, table, 16, 0)


@pytest.mark.parametrize("T", [300, 70000])
def test_without_holes_it_is_the_plain_choice(T):
    need_gpu()
    sums = torch.from_numpy(random_sums((3, 2, T), T)).cuda()
    lens = torch.tensor([T, 5, T // 2], dtype=torch.int32).cuda()
    table = torch.zeros(3, (T + 15) // 16, dtype=torch.int32, device="cuda")
    got = []
    for fn, extra in ((pa.pa_evict_select, ()), (pa.pa_evict_select_paged, (16, 1))):
        keep = torch.zeros(3, 2, T // 3, dtype=torch.int32, device="cuda")
        new, out = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros_like(sums)
        tab = (table,) if extra else ()
        fn(keep, new, out, sums, lens, *tab, T // 3, 4, 30, *extra)
        got.append((keep, new, out))
    for a, b in zip(*got):
        assert (a == b).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "q4"])
@pytest.mark.parametrize("budget", [96, 600])
def test_dropped_blocks_through_the_whole_set(cache, budget):
    """Sequences with dropped blocks, among them the first and the last: weights, choice, move
    to new blocks, decode.  The attention after it is the oracle's over the kept tokens."""
    G, H, bs = 4, 2, 16
    w = batch(cache, [200, 331, 40], H, G, bs, seed=6, extra_blocks=130)
    nb, need = len(w["k"]), [13, 21, 3]
    w["table"][0, [0, 5]] = -1
    w["table"][1, [2, 3, 20]] = nb
    w["table"][2, :3] = -1  # nothing left
    B, HQ = 3, H * G
    q = w["q"].cuda()
    table, cl = torch.from_numpy(w["table"]).cuda(), torch.from_numpy(w["lens"]).cuda()
    T = 352
    sums, out = torch.zeros(B, H, T, device="cuda"), torch.empty_like(q)
    ws = pa.decode_scored_workspace(B, HQ, H, D, T)
    kw = dict(k_scale=w["ks"], v_scale=w["vs"])
    pa.pa_paged_decode_attention_scored(out, sums, sums, T, q, w["kd"], w["vd"], table, cl, w["scale"],
                                        T, ws, **kw)
    old = sums.cpu().numpy()
    keep = torch.empty(B, H, budget, dtype=torch.int32, device="cuda")
    new = torch.empty(B, dtype=torch.int32, device="cuda")
    pa.pa_evict_select_paged(keep, new, sums, sums, cl, table, budget, 4, 32, bs, nb)
    owned = {int(x) for b in range(B) for x in w["table"][b, :need[b]] if 0 <= x < nb}
    free = [x for x in range(nb) if x not in owned]
    cols = (budget + bs - 1) // bs
    dst = torch.tensor(free[:B * cols], dtype=torch.int32).view(B, cols).cuda()
    pa.pa_cache_compact(w["kd"], w["vd"], keep, new, table, dst)
    pa.pa_paged_decode_attention_scored(out, sums, sums, 0, q, w["kd"], w["vd"], dst, new, w["scale"],
                                        T, ws, **kw)
    torch.cuda.synchronize()
    assert pa.read_device_error(ws) == 0
    ref_keep, ref_new = lc.evict_select(old, w["lens"], budget, 4, 32, w["table"], bs, nb)
    assert (keep.cpu().numpy() == ref_keep).all() and (new.cpu().numpy() == ref_new).all()
    assert ref_new.tolist() == [min(budget, 168), min(budget, 288), 0]  # 32 and 43 tokens have no row
    assert (out[2] == 0).all()
    qs, got = q.cpu().double().numpy(), out.cpu().double().numpy()
    for b in range(2):
        for g in range(H):
            t = ref_keep[b, g, :ref_new[b]]
            at = w["table"][b, t // bs], t % bs, g
            s = qs[b, g * G:(g + 1) * G] @ w["k64"][at].T * w["scale"]
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            ref = p @ w["v64"][at]
            # bf16 outputs of weights and values rounded as in the decode call alone
            assert (np.abs(got[b, g * G:(g + 1) * G] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * 20).all()
            add = old[b, g, t] + p.sum(0)
            assert (np.abs(sums[b, g, :ref_new[b]].cpu().numpy() - add) <= 2.0 ** -12 * add).all()


def test_captured():
    need_gpu()
    B, H, T, budget, bs = 2, 2, 600, 200, 16
    sums = torch.from_numpy(random_sums((B, H, T), 8)).cuda()
    lens = torch.tensor([600, 100], dtype=torch.int32, device="cuda")
    keep = torch.empty(B, H, budget, dtype=torch.int32, device="cuda")
    new = torch.empty(B, dtype=torch.int32, device="cuda")
    table, nb = holed([600, 600], bs, 0.3, 3)
    td = torch.zeros(B, table.shape[1], dtype=torch.int32, device="cuda")
    dst = torch.empty_like(sums)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_evict_select_paged(keep, new, dst, sums, lens, td, budget, 4, 30, bs, nb)
    lens.copy_(torch.tensor([401, 333], dtype=torch.int32))
    td.copy_(torch.from_numpy(table))
    graph.replay()
    torch.cuda.synchronize()
    want, want_new = lc.evict_select(sums.cpu().numpy(), [401, 333], budget, 4, 30, table, bs, nb)
    assert (keep.cpu().numpy() == want).all() and (new.cpu().numpy() == want_new).all()
