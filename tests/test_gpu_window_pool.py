"""The sliding-window calls as a layer with a window uses them: a pool that holds the window only, written
through the second slot table, read through a block table of its own; blocks behind the window are
given back, spoilt and taken by other tokens as sequences go on.  Bounds as in test_gpu_window.py."""
import numpy as np
import pytest
import torch

from oracle import window as ow
from paged_kv_cache_309_gb300 import pa
from tests.gpu_util import need_gpu
from tests.test_gpu_window import BF16, E4M3, SCALE, compare

pytestmark = pytest.mark.gpu

H, HQ, BS, FULL = 2, 8, 16, 512  # FULL: slots of a sequence in the cache of a layer without a window


class Pool:
    """Blocks of a window's layer for some sequences, and both slot tables."""

    def __init__(self, seqs, blocks, window, sink, cache):
        self.window, self.keep = window, (sink + BS - 1) // BS  # blocks with first tokens stay
        self.free = list(np.random.default_rng(1).permutation(blocks))
        self.table = np.full((seqs, FULL // BS), -1, np.int32)
        self.swa = torch.full((seqs * FULL,), -1, dtype=torch.int64, device="cuda")
        nan = torch.full((blocks, BS, H, 128), float("nan"), device="cuda").to(cache)
        self.k, self.v = nan, nan.clone()
        self.reused = 0

    def go_on(self, b, first, end):
        """Sequence b's tokens first .. end - 1 come: what lies behind their windows goes, they get slots."""
        for i in range(self.keep, max(0, first - self.window + 1) // BS):
            blk = int(self.table[b, i])
            if blk >= 0:
                self.k[blk] = self.v[blk] = float("nan")
                self.swa[b * FULL + i * BS:b * FULL + (i + 1) * BS] = -1
                self.table[b, i] = -1
                self.free.insert(0, blk)
                self.reused += 1
        for t in range(first, end):
            if self.table[b, t // BS] < 0:
                self.table[b, t // BS] = self.free.pop()
            self.swa[b * FULL + t] = int(self.table[b, t // BS]) * BS + t % BS


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("window,sink,chunk,blocks", [(40, 3, 50, 20), (64, 0, 33, 18), (17, 20, 16, 14), (1, 1, 24, 10)])
def test_a_pool_of_the_window_only(window, sink, chunk, blocks, cache):
    need_gpu()
    prompts, lens, rot = [150, 61], [230, 120], 64
    B = len(lens)
    scales = {} if cache == BF16 else dict(k_scale=torch.tensor([0.05], device="cuda"),
                                           v_scale=torch.tensor([0.03], device="cuda"))
    gen = torch.Generator().manual_seed(window)
    rows = torch.randn((B, max(lens), (HQ + 2 * H) * 128), generator=gen).bfloat16().cuda()
    angle = np.arange(256)[:, None] * 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    cs = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
    pool = Pool(B, blocks, window, sink, cache)
    # a layer without a window beside it keeps every token, for the plain form
    full = [torch.zeros((B * FULL // BS, BS, H, 128), device="cuda").to(cache) for _ in range(2)]
    q = torch.zeros((B, max(lens), HQ, 128), dtype=BF16, device="cuda")
    out = torch.zeros_like(q)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pa.window_decode_workspace(B, HQ, H, 128, window, sink, max(lens))

    def append(part):
        """Tokens (b, t) of a step, a padded one, and one whose slot in the window's pool is gone."""
        rowsets = torch.stack([rows[b, t] for b, t in part] + [rows[0, 0], rows[0, 1]])
        split = [rowsets[:, i * 128:j * 128].unflatten(1, (j - i, 128))
                 for i, j in ((0, HQ), (HQ, HQ + H), (HQ + H, HQ + 2 * H))]
        pos = torch.tensor([t for _, t in part] + [0, 1], device="cuda")
        slot = torch.tensor([b * FULL + t for b, t in part] + [-1, B * FULL - 1], device="cuda")
        turned, other = torch.empty_like(split[0]), torch.empty_like(split[0])
        pa.pa_rope_and_cache(turned, *split, pool.k, pool.v, cs, pos, slot, swa_slot_mapping=pool.swa, **scales)
        slot[-1] = -1
        pa.pa_rope_and_cache(other, *split, *full, cs, pos, slot, **scales)
        assert torch.equal(turned, other)
        for i, (b, t) in enumerate(part):
            q[b, t] = turned[i]
        return turned[:len(part)]

    done = [0] * B
    while any(d < p for d, p in zip(done, prompts)):  # prompts in chunks
        new = [min(chunk, p - d) for d, p in zip(done, prompts)]
        for b in range(B):
            pool.go_on(b, done[b], done[b] + new[b])
        part = [(b, done[b] + j) for b in range(B) for j in range(new[b])]
        turned = append(part).contiguous()
        done = [d + n for d, n in zip(done, new)]
        if cache == BF16:
            got = torch.empty_like(turned)
            pa.pa_paged_window_prefill_attention(
                got, turned, pool.k, pool.v, torch.from_numpy(pool.table).cuda(),
                torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda"),
                torch.tensor(done, dtype=torch.int32, device="cuda"), window, sink, SCALE, max(new), err)
            for i, (b, t) in enumerate(part):
                out[b, t] = got[i]
    while any(d < n for d, n in zip(done, lens)):  # then tokens, until each sequence ends
        live = [b for b in range(B) if done[b] < lens[b]]
        for b in live:
            pool.go_on(b, done[b], done[b] + 1)
        part = [(b, done[b]) for b in live]
        turned = append(part).contiguous()
        for b in live:
            done[b] += 1
        got = torch.empty_like(turned)
        pa.pa_paged_window_decode_attention(
            got, turned, pool.k, pool.v, torch.from_numpy(pool.table[live]).cuda(),
            torch.tensor([done[b] for b in live], dtype=torch.int32, device="cuda"), window, sink, SCALE,
            max(lens), ws, **scales)
        for i, (b, t) in enumerate(part):
            out[b, t] = got[i]
    torch.cuda.synchronize()
    assert int(err) == 0 and pa.read_device_error(ws) == 0 and pool.reused > 5
    factors = [1.0, 1.0] if cache == BF16 else [float(scales["k_scale"]), float(scales["v_scale"])]
    host = [c.double().cpu().numpy() * f for c, f in zip(full, factors)]
    for b in range(B):
        table = (b * FULL // BS + np.arange(FULL // BS))[None].astype(np.int32)
        ref = ow.prefill(q[b, :lens[b]].double().cpu().numpy(), *host, table, [0, lens[b]], [lens[b]], window, sink, SCALE)
        if cache == BF16:
            compare(out[b, :prompts[b]], [x[:prompts[b]] for x in ref], 2.0 ** -8)
        compare(out[b, prompts[b]:lens[b]], [x[prompts[b]:] for x in ref], 2.0 ** -16 if cache == BF16 else 2.0 ** -11)
