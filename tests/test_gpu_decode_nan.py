"""NaN in decode attention: a head whose scores hold a NaN gives NaN, whatever
the split plan, in the plain, the fused and the scored call alike; the other
heads stay finite."""
import numpy as np
import pytest
import torch

from paged_kv_cache_309_gb300 import pa
from paged_kv_cache_309_gb300 import workloads as wl
from tests.gpu_util import need_gpu, to_dev
from tests.test_gpu_q4_decode import D
from tests.test_gpu_scored_decode import batch

pytestmark = pytest.mark.gpu

# lengths and whether their plan has several ranges
PLANS = [([40, 33], False), ([700, 130], True), ([9000, 64], True)]


def calls(w, lens):
    """Outputs of the plain, the scored and the fused call and the scored sums."""
    q = w["q"].cuda()
    B, HQ, _ = q.shape
    H, mcl = w["H"], max(lens)
    table, cl = torch.from_numpy(w["table"]).cuda(), torch.from_numpy(w["lens"]).cuda()
    kw = dict(k_scale=w["ks"], v_scale=w["vs"])
    plain, step, scored = (torch.zeros_like(q) for _ in range(3))
    ws = pa.decode_workspace(B, HQ, H, D, mcl)
    pa.pa_paged_decode_attention(plain, q, w["kd"], w["vd"], table, cl, w["scale"], mcl, ws, **kw)
    sums = torch.zeros(B, H, mcl, device="cuda")
    sws = pa.decode_scored_workspace(B, HQ, H, D, mcl)
    pa.pa_paged_decode_attention_scored(scored, sums, sums, mcl, q, w["kd"], w["vd"], table, cl,
                                        w["scale"], mcl, sws, **kw)
    # the fused step: a finite new token in place of each sequence's last one
    new = torch.randn(2, B, H, D, device="cuda").bfloat16()
    at = w["lens"].astype(np.int64) - 1
    slots = w["table"][np.arange(B), at // w["bs"]].astype(np.int64) * w["bs"] + at % w["bs"]
    pa.pa_paged_decode_step(step, q, new[0], new[1], torch.from_numpy(slots).cuda(), w["kd"], w["vd"],
                            table, cl, w["scale"], mcl, ws, **kw)
    torch.cuda.synchronize()
    assert pa.read_device_error(ws) == 0 and pa.read_device_error(sws) == 0
    return dict(plain=plain, scored=scored, step=step), sums


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("lens,several", PLANS)
def test_nan_query(cache, G, lens, several):
    need_gpu()
    assert (pa.pa_paged_decode_plan(2, 2, max(lens))[0] > 1) == several
    w = batch(cache, lens, 2, G, 16, seed=1)
    w["q"][0, 1] = float("nan")
    outs, sums = calls(w, lens)
    for name, out in outs.items():
        assert out[0, 1].isnan().all(), name
        out[0, 1] = 0
        assert not out.isnan().any(), name
    assert sums[0, 0, :lens[0]].isnan().all()  # the sum of its kv head's query heads
    assert not sums[0, 1].isnan().any() and not sums[1].isnan().any()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("lens,several", PLANS)
def test_nan_key_in_every_range(cache, G, lens, several):
    need_gpu()
    w = batch(cache, lens, 2, G, 16, seed=2)
    raw, code = (torch.int8, 127) if cache == "e4m3" else (torch.int16, 0x7FC0)
    for t in range(5, lens[0], 64):
        w["kd"].view(raw)[int(w["table"][0, t // 16]), t % 16, 1] = code
    outs, sums = calls(w, lens)
    for name, out in outs.items():
        assert out[0, G:].isnan().all(), name
        assert not out[0, :G].isnan().any() and not out[1].isnan().any(), name
    assert sums[0, 1, :lens[0]].isnan().all()
    assert not sums[0, 0].isnan().any() and not sums[1].isnan().any()


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("lens", [[40, 33], [9000, 64]])
def test_nan_query_of_the_latent_decode(heads, lens):
    need_gpu()
    w = wl.make_mla_decode("nan", 3, 2, 1, 1, heads, context_lens=lens)
    q = torch.randn(2, heads, 576, device="cuda").bfloat16()
    q[0, 1] = float("nan")
    out = torch.zeros(2, heads, 512, dtype=torch.bfloat16, device="cuda")
    ws = pa.mla_decode_workspace(2, heads, max(lens))
    pa.pa_mla_decode_attention(out, q, to_dev(w.latent_cache, "bf16"),
                               torch.from_numpy(w.block_tables).cuda(),
                               torch.from_numpy(w.context_lens).cuda(), w.scale, max(lens), ws)
    torch.cuda.synchronize()
    assert pa.read_device_error(ws) == 0
    assert out[0, 1].isnan().all()
    out[0, 1] = 0
    assert not out.isnan().any()
