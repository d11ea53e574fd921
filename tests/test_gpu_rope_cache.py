"""GPU tests of pa_rope_and_cache against the definition.

Two checks on every element written.  Bits: the definition rounds each product
and sum to fp32, so the fp32 emulation (then the division, and torch's cast on the host)
gives the very codes.  Value: against the rotation in 64 bits,
    |y - ref| <= h(type) |ref| + 4 * 2^-24 size  (+ the smallest subnormal's half)
with h the half step of the output's type (bf16 2^-8, fp16 2^-11, fp32 2^-24,
e4m3 2^-4) and size the magnitudes of an element's two terms: two product roundings and a
sum's are each at most 2^-24 of the size, a division by the scale another.
"""
import numpy as np
import pytest
import torch

from oracle import window as ow
from paged_kv_cache_309_gb300 import pa
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
HALF_STEP = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -24, E4M3: 2.0 ** -4}
HALF_SMALLEST = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -150, E4M3: 2.0 ** -10}


def table(positions, rot, base=10000.0):
    angle = np.arange(positions)[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def cast(x, dtype):
    x = torch.from_numpy(np.ascontiguousarray(x))
    if dtype == E4M3:
        x = x.clamp(-448, 448)
    return x.to(dtype)


def case(n, hq, h, d, rot, src=BF16, seed=0, pad=0, most=4096):
    """Token rows that lie side by side in a wider row, as a fused projection leaves them."""
    gen = torch.Generator().manual_seed(seed)
    wide = torch.randn((n, (hq + 2 * h) * d + pad), generator=gen).to(src)
    pos = torch.randint(0, most, (n,), generator=gen)
    return wide, pos, table(most, rot)


def split(wide, hq, h, d):
    return (wide[:, :hq * d].unflatten(1, (hq, d)), wide[:, hq * d:(hq + h) * d].unflatten(1, (h, d)),
            wide[:, (hq + h) * d:(hq + 2 * h) * d].unflatten(1, (h, d)))


def same(got, want):
    """Equal bits, any NaN for any NaN."""
    got, want = got.cpu(), want.cpu()
    if got.dtype == E4M3:
        g, w = got.view(torch.uint8), want.view(torch.uint8)
        return bool(((g == w) | (((g & 127) == 127) & ((w & 127) == 127))).all())
    bits = torch.int32 if got.dtype == FP32 else torch.int16
    return bool(((got.view(bits) == want.view(bits)) | (got.isnan() & want.isnan())).all())


def check(n, hq, h, d, rot, interleaved=False, src=BF16, dst=BF16, bs=16, scales=None, swa=False, seed=0,
          pad=0, in_place=False, spoil=None, block_pad=0, stream=None):
    need_gpu()
    wide, pos, cs = case(n, hq, h, d, rot, src, seed, pad)
    if spoil is not None:
        spoil(wide, pos)
    rng = np.random.default_rng(seed + 1)
    nb = (n + bs - 1) // bs + 2
    slot = rng.permutation(nb * bs)[:n]
    if n > 3:
        slot[rng.random(n) < 0.1] = -1
        slot[1] = nb * bs + 3  # outside the pool
    remap = None
    if swa:
        remap = rng.permutation(nb * bs)
        remap[rng.random(nb * bs) < 0.4] = -1
        remap = remap[:nb * bs - bs]  # some slots lie past the table
    gen = torch.Generator().manual_seed(seed + 2)
    pool = [torch.randn((nb, bs * h * d + block_pad), generator=gen).to(dst) for _ in range(2)]
    dev = wide.cuda()
    q, k, v = split(dev, hq, h, d)
    out = q if in_place else torch.full((n, hq, d), 7.0, dtype=src, device="cuda")
    caches = [p.cuda() for p in pool]
    views = [c[:, :bs * h * d].unflatten(1, (bs, h, d)) for c in caches]
    sc = [None, None] if scales is None else [torch.tensor([s], device="cuda") for s in scales]
    pa.pa_rope_and_cache(out, q, k, v, *views, torch.from_numpy(cs).cuda(), pos.cuda(),
                         torch.from_numpy(slot).cuda(), interleaved=interleaved,
                         swa_slot_mapping=None if remap is None else torch.from_numpy(remap).cuda(),
                         k_scale=sc[0], v_scale=sc[1], stream=stream)
    torch.cuda.synchronize()
    hq_, hk_, hv_ = split(wide, hq, h, d)
    ok = (pos >= 0) & (pos < len(cs))
    at = pos.clamp(0, len(cs) - 1).numpy()
    # queries
    want = cast(ow.rotate_f32(hq_.float().numpy(), cs, at, interleaved), src)
    want[..., rot:] = hq_[..., rot:]
    left = hq_ if in_place else torch.full_like(want, 7.0)
    want[~ok] = left[~ok]
    assert same(out.contiguous(), want)
    if spoil is None:
        ref, size = ow.rotate(hq_.float().numpy(), cs, at, interleaved)
        err = np.abs(out.double().cpu().numpy() - ref)
        assert (err <= HALF_STEP[src] * np.abs(ref) + 2.0 ** -22 * size + HALF_SMALLEST[src]).all()
    # caches, whole
    where = ow.slots(slot, remap, nb * bs)
    for i, rows in enumerate((ow.rotate_f32(hk_.float().numpy(), cs, at, interleaved), hv_.float().numpy())):
        host = pool[i].clone()
        flat = host[:, :bs * h * d].unflatten(1, (bs, h, d))
        if scales is not None:
            rows = rows / np.float32(scales[i])
        stored = cast(rows, dst)
        if scales is None and src == dst:  # what is not turned keeps its bits
            turned = rot if i == 0 else 0
            stored[..., turned:] = (hk_, hv_)[i][..., turned:]
        for t, s in enumerate(where):
            if s >= 0 and ok[t]:
                flat[s // bs, s % bs] = stored[t]
        assert same(caches[i], host), "kv"[i]
        if spoil is None:
            full = ow.rotate(hk_.float().numpy(), cs, at, interleaved)[0] if i == 0 else hv_.double().numpy()
            mag = ow.rotate(hk_.float().numpy(), cs, at, interleaved)[1] if i == 0 else np.abs(full)
            if scales is not None:
                full, mag = full / scales[i], mag / np.float64(np.float32(scales[i]))
            if dst == E4M3:
                full = np.clip(full, -448, 448)
            got = views[i].double().cpu().numpy()
            for t, s in enumerate(where):
                if s >= 0:
                    e = np.abs(got[s // bs, s % bs] - full[t])
                    assert (e <= HALF_STEP[dst] * np.abs(full[t]) * 1.001 + 2.0 ** -22 * mag[t]
                            + HALF_SMALLEST[dst] * 1.001).all()
    # the projection's rows are not written (but queries rotated in place)
    if not in_place:
        assert same(dev, wide)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 32), (96, 96), (96, 32), (256, 256), (80, 16), (24, 16),
                                   (16, 16), (512, 512), (504, 16), (192, 176), (40, 32)])
def test_head_shapes(d, rot, interleaved):
    check(37, 6, 3, d, rot, interleaved, seed=d + rot)


@pytest.mark.parametrize("n", [1, 2, 8, 64, 511])
@pytest.mark.parametrize("hq,h", [(1, 1), (16, 8), (7, 1), (32, 4), (5, 5)])
def test_tokens_and_heads(n, hq, h):
    check(n, hq, h, 128, 128, seed=n + hq)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("src", [BF16, FP16, FP32])
@pytest.mark.parametrize("dst", [BF16, FP16, FP32, E4M3])
def test_types(src, dst, interleaved):
    check(50, 6, 2, 64, 64, interleaved, src, dst, seed=3)
    check(50, 6, 2, 64, 48, interleaved, src, dst, seed=4, scales=(0.05, 0.3))


@pytest.mark.parametrize("bs", [1, 7, 16, 24, 256])
def test_block_sizes_and_strides(bs):
    check(61, 4, 2, 128, 128, bs=bs, pad=24, block_pad=64, seed=bs)


def test_window_table():
    check(120, 4, 2, 128, 128, swa=True, seed=11)
    check(120, 4, 2, 128, 64, True, FP16, E4M3, swa=True, scales=(0.02, 0.04), seed=12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(interleaved):
    check(70, 8, 2, 128, 128, interleaved, in_place=True, pad=8, seed=13)


def test_positions_outside_the_table_leave_the_token_out():
    def spoil(wide, pos):
        pos[0], pos[5], pos[9] = -1, 4096, 2 ** 62
    check(20, 4, 2, 128, 128, spoil=spoil, seed=14)
    check(20, 4, 2, 128, 128, spoil=spoil, seed=14, in_place=True)


@pytest.mark.parametrize("dst,scales", [(BF16, None), (E4M3, None), (E4M3, (0.05, 1e-38)), (FP16, (1e-30, 0.0))])
def test_values_that_are_not_finite(dst, scales):
    def spoil(wide, pos):
        flat = wide.view(-1)
        flat[::97] = float("nan")
        flat[5::89] = float("inf")
        flat[7::83] = -float("inf")
        flat[11::79] = 3e38
        flat[13::73] = -0.0
        flat[17::71] = 1e-40
    check(40, 4, 2, 128, 64, dst=dst, scales=scales, spoil=spoil, seed=15)


def test_many_heads():
    check(3, 128, 64, 128, 128, seed=16)
    check(3, 130, 1, 16, 16, True, seed=17)


def test_no_tokens():
    need_gpu()
    e = torch.empty((0, 4, 64), dtype=BF16, device="cuda")
    k = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    c = torch.ones((2, 16, 2, 64), dtype=BF16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    pa.pa_rope_and_cache(e, e, k, k, c, c.clone(), torch.zeros((8, 64), device="cuda"), none, none)
    assert bool((c == 1).all())


def test_on_another_stream_and_in_a_graph():
    need_gpu()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    check(33, 4, 2, 128, 128, seed=18, stream=s)
    wide, pos, cs = case(33, 4, 2, 128, 128, seed=19)
    dev, cs = wide.cuda(), torch.from_numpy(cs).cuda()
    q, k, v = split(dev, 4, 2, 128)
    out = torch.zeros((33, 4, 128), dtype=BF16, device="cuda")
    kc, vc = (torch.zeros((4, 16, 2, 128), dtype=BF16, device="cuda") for _ in range(2))
    pos, slot = pos.cuda(), torch.randperm(64, device="cuda")[:33]
    args = (out, q, k, v, kc, vc, cs, pos, slot)
    pa.pa_rope_and_cache(*args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_rope_and_cache(*args)
    dev.copy_(torch.randn_like(dev))  # a replay takes the inputs as they are then
    pos.copy_(pos.flip(0))
    kc.zero_()
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (out, kc, vc)]
    kc.zero_()
    pa.pa_rope_and_cache(*args)
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got, (out, kc, vc)))
