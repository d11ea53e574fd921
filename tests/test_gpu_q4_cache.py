"""GPU parity of the 4-bit cache's write and read-back against the oracle.

The format is defined by IEEE fp32 steps, so a cache's bytes are compared
bit for bit (any NaN pattern equal to any other in the (scale, minimum)
pairs).  The read-back is one fused multiply-add and one cast: compared with
the double value rounded once, at most one step of fp32 (2^-24 relative) plus
half a step of the output type away.
"""
import numpy as np
import pytest
import torch

from oracle import long_context as lc
from paged_kv_cache_309_gb300 import pa
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = {t: torch.finfo(TYPES[t]).eps for t in TYPES}


def same_rows(got, want):
    d = got.shape[-1] * 8 // 5
    assert (got[..., :d // 2] == want[..., :d // 2]).all()
    a = np.ascontiguousarray(got[..., d // 2:]).view(np.uint16)
    b = np.ascontiguousarray(want[..., d // 2:]).view(np.uint16)
    nan = ((a & 0x7FFF) > 0x7C00) & ((b & 0x7FFF) > 0x7C00)
    assert ((a == b) | nan).all()


def source(n, h, d, kind, rng, pad=0):
    x = torch.from_numpy(rng.standard_normal((n, h * d + pad)).astype(np.float32)).to(TYPES[kind])
    return x.cuda()[:, :h * d].unflatten(1, (h, d))


def write_case(n, h, d, bs, kind, seed=0, pad=0, swa_window=0, skip=0.1, block_pad=0, edit=None):
    need_gpu()
    rng = np.random.default_rng(seed)
    nb = (n + bs - 1) // bs + 1
    rb = pa.q4_row_bytes(d)
    pools = []
    for _ in range(2):
        whole = torch.full((nb, bs * h * rb + block_pad), 0xA5, dtype=torch.uint8, device="cuda")
        pools.append(whole)
    kc, vc = (p[:, :bs * h * rb].unflatten(1, (bs, h, rb)) for p in pools)
    key, value = source(n, h, d, kind, rng, pad), source(n, h, d, kind, rng, pad)
    if edit is not None:
        edit(key)
        edit(value)
    slots = rng.permutation(nb * bs)[:n].astype(np.int64)
    slots[rng.random(n) < skip] = -1
    if n > 2:
        slots[n // 2] = nb * bs + 5  # past the pool: skipped
    swa = None
    if swa_window:
        swa = np.full(nb * bs, -1, np.int64)
        live = slots[(slots >= 0) & (slots < nb * bs)][-swa_window:]
        swa[live] = rng.permutation(nb * bs)[:len(live)]
    pa.pa_reshape_and_cache_q4(key, value, kc, vc, torch.from_numpy(slots).cuda(),
                               None if swa is None else torch.from_numpy(swa).cuda())
    torch.cuda.synchronize()
    for x, c, p in ((key, kc, pools[0]), (value, vc, pools[1])):
        want = np.full((nb, bs, h, rb), 0xA5, np.uint8)
        lc.q4_write(x.float().cpu().numpy(), want, slots, swa)
        same_rows(c.cpu().numpy(), want)
        assert (p[:, bs * h * rb:] == 0xA5).all()
    return key, value, kc, vc, slots, swa


@pytest.mark.parametrize("n,h,d,bs,kind", [
    (1, 1, 32, 1, "bf16"), (1, 8, 128, 16, "bf16"), (7, 3, 96, 5, "fp16"), (65, 5, 128, 64, "fp32"),
    (300, 8, 128, 16, "bf16"), (300, 8, 128, 16, "fp16"), (33, 2, 576, 8, "bf16"),
    (19, 40, 64, 7, "fp32"), (5, 1, 1120, 16, "bf16"), (2, 17, 160, 16, "fp16")])
def test_write_bytes(n, h, d, bs, kind):
    write_case(n, h, d, bs, kind, seed=n + h + d)


def test_write_strided_rows_and_blocks():
    write_case(130, 5, 128, 16, "bf16", pad=72, block_pad=48)
    write_case(130, 3, 96, 16, "fp32", pad=8, block_pad=4)


@pytest.mark.parametrize("n", [1, 9, 700])
def test_write_through_sliding_window_table(n):
    write_case(n, 4, 128, 16, "bf16", seed=n, swa_window=max(1, n // 3))


def test_write_prompt_full_size():
    """32768 tokens of 8 heads, as the benchmark's prompt write."""
    write_case(32768, 8, 128, 16, "bf16", seed=5, skip=0.05)


def special(x):
    """Constant groups, huge and tiny spans, both signs of zero, minima that round up, ties."""
    f = x.reshape(x.shape[0], -1)
    big = torch.finfo(x.dtype).max
    rows = [lambda r: r.fill_(0.), lambda r: r.fill_(-0.), lambda r: r.fill_(3.1415),
            lambda r: r.mul_(1e-5), lambda r: r.mul_(1e-7), lambda r: r.mul_(3e4 if x.dtype == torch.float16 else 1e30).clamp_(-big, big),
            lambda r: r.mul_(1e-2).add_(1000.3), lambda r: r.mul_(400),
            lambda r: r.copy_((torch.arange(r.numel(), device=r.device) % 31).to(r.dtype) / 2),
            lambda r: r[::5].fill_(float("nan")), lambda r: r[3:4].fill_(float("inf")),
            lambda r: r[40:41].fill_(float("-inf")), lambda r: r[0:1].fill_(big),
            lambda r: r[31:32].fill_(-big)]
    for i, fn in enumerate(rows):
        row = f[i].clone()
        fn(row)
        x[i] = row.view(x.shape[1:])


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_write_special_values(kind):
    key, value, kc, vc, slots, _ = write_case(40, 2, 128, 16, kind, edit=special, skip=0.)
    # a group with a NaN or an infinity reads back as NaN, its neighbours do not
    k = torch.zeros_like(key, dtype=torch.float32)
    pa.pa_gather_cache_q4(k, torch.zeros_like(k), kc, vc, torch.from_numpy(slots).cuda())
    k = k.cpu().reshape(40, 8, 32)
    bad = ~torch.isfinite(key.cpu().float().reshape(40, 8, 32)).all(-1)
    bad[20] = False  # the skipped token's row stays zero
    assert (torch.isnan(k).all(-1) == bad).all() and (torch.isnan(k).any(-1) == bad).all()
    assert bad[9].all() and bad[10].sum() == 1 and bad[11].sum() == 1


def test_write_every_bf16_pattern():
    """All 65,536 bf16 codes as elements, next to ordinary values."""
    codes = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)

    def edit(x):
        flat = x.reshape(-1)
        flat[::8][:65536] = codes.cuda()
        x.copy_(flat.view(x.shape))
    write_case(512, 8, 128, 16, "bf16", edit=edit, skip=0.)


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,h,d,bs,pad", [(1, 1, 32, 1, 0), (200, 5, 128, 16, 24),
                                          (77, 3, 96, 5, 0), (9, 1, 1120, 4, 8)])
def test_gather(n, h, d, bs, pad, out):
    _, _, kc, vc, slots, _ = write_case(n, h, d, bs, "fp32", seed=n, block_pad=16)
    dst = [torch.full((n + 3, h * d + pad), 7.0, dtype=TYPES[out], device="cuda") for _ in range(2)]
    ko, vo = (t[:n, :h * d].unflatten(1, (h, d)) for t in dst)
    pa.pa_gather_cache_q4(ko, vo, kc, vc, torch.from_numpy(slots).cuda())
    for o, c, whole in ((ko, kc, dst[0]), (vo, vc, dst[1])):
        cache = c.cpu().numpy().reshape(-1, h, c.shape[-1])
        live = (slots >= 0) & (slots < len(cache))
        want = lc.q4_restore(cache[slots[live]])
        got = o.float().cpu().numpy().astype(np.float64)
        assert (got[~live] == 7.0).all()
        tiny = 2.0 ** -25 if out == "fp16" else 0.0  # half the last subnormal step
        tol = np.abs(want) * (2.0 ** -24 + EPS[out] / 2 * (1 + 2.0 ** -23)) + tiny
        assert (np.abs(got[live] - want) <= tol).all()
        assert (whole[n:] == 7.0).all() and (whole[:, h * d:] == 7.0).all()


def test_key_only():
    need_gpu()
    x = torch.randn(50, 1, 576, device="cuda", dtype=torch.bfloat16)
    cache = torch.zeros(4, 16, 1, pa.q4_row_bytes(576), dtype=torch.uint8, device="cuda")
    slots = torch.randperm(64, device="cuda")[:50]
    pa.pa_reshape_and_cache_q4(x, None, cache, None, slots)
    want = lc.q4_quantise(x.float().cpu().numpy())
    same_rows(cache.view(64, 1, -1)[slots].cpu().numpy(), want)
    back = torch.empty_like(x)
    pa.pa_gather_cache_q4(back, None, cache, None, slots)
    err = (back.float() - x.float()).abs().view(50, -1, 32)
    span = x.float().view(50, -1, 32).amax(-1) - x.float().view(50, -1, 32).amin(-1)
    # half a step of the 15 (1 + 2^-11: the scale's rounding), the minimum's fp16
    # rounding and the output's bf16 rounding
    mag = x.float().abs().view(50, -1, 32).amax(-1)
    assert (err.amax(-1) <= span / 30 * (1 + 2.0 ** -8) + mag * (2.0 ** -8 + 2.0 ** -10)).all()


def test_captured_and_replayed_on_another_stream():
    need_gpu()
    key, value = (torch.randn(40, 2, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kc, vc = (torch.zeros(3, 16, 2, 80, dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.arange(40, device="cuda")
    ko, vo = torch.zeros_like(key), torch.zeros_like(key)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_reshape_and_cache_q4(key, value, kc, vc, slots)
        pa.pa_gather_cache_q4(ko, vo, kc, vc, slots)
    key.copy_(torch.randn_like(key))
    g.replay()
    torch.cuda.synchronize()
    same_rows(kc.view(48, 2, 80)[:40].cpu().numpy(), lc.q4_quantise(key.float().cpu().numpy()))
    k2 = torch.zeros_like(kc)
    side = torch.cuda.Stream()
    pa.pa_reshape_and_cache_q4(key, value, k2, vc.clone(), slots, stream=side)
    side.synchronize()
    assert (k2 == kc).all()
