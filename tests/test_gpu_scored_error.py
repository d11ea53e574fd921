"""The scored decode call on a workspace whose error word says that a wait ran
out: the sums stay as they were (an aborted launch leaves scores of earlier
calls behind), and follow again once the word is cleared."""
import pytest
import torch

from paged_kv_cache_309_gb300 import pa
from tests.test_gpu_q4_decode import D
from tests.test_gpu_scored_decode import batch, check

pytestmark = pytest.mark.gpu


def call(w, sums_out, sums, ws, mcl):
    q = w["q"].cuda()
    out = torch.full_like(q, float("nan"))
    pa.pa_paged_decode_attention_scored(
        out, sums_out, sums, 1, q, w["kd"], w["vd"], torch.from_numpy(w["table"]).cuda(),
        torch.from_numpy(w["lens"]).cuda(), w["scale"], mcl, ws, k_scale=w["ks"], v_scale=w["vs"])
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "q4"])
@pytest.mark.parametrize("lens,G", [([40, 33], 2), ([900, 0, 65], 4), ([5000], 16)])
@pytest.mark.parametrize("in_place", [True, False])
def test_sums_are_left_after_a_timeout(cache, lens, G, in_place):
    w = batch(cache, lens, 2, G, 16, seed=3)
    mcl, B = max(lens), len(lens)
    ws = pa.decode_scored_workspace(B, 2 * G, 2, D, mcl)
    word = ws[:4].view(torch.int32)
    sums = torch.rand(B, 2, mcl, device="cuda")
    before = sums.clone()
    dst = sums if in_place else torch.full_like(sums, -5.0)
    kept = dst.clone()
    want = call(w, torch.empty_like(sums), sums, ws, mcl)
    assert pa.read_device_error(ws) == 0
    for bits in (pa.PA_DEVERR_WAIT_TIMEOUT, pa.PA_DEVERR_WAIT_TIMEOUT | pa.PA_DEVERR_CONTEXT_CLIPPED):
        word.fill_(bits)
        out = call(w, dst, sums, ws, mcl)
        assert (dst == kept).all() and (sums == before).all()
        assert (out == want).all()
        assert int(word) == bits
    for bits in (pa.PA_DEVERR_CONTEXT_CLIPPED, 0):  # no other bit holds the sums
        sums.copy_(before)
        word.fill_(bits)
        call(w, dst, sums, ws, mcl)
        got = dst.cpu().numpy().astype("float64")
        check(w, got, before.cpu().numpy().astype("float64"), 1, cache,
              untouched=None if in_place else -5.0)
