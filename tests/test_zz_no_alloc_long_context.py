"""The promise of every call, for the long-context ones: they take no device
memory and do not wait for the GPU, on the current stream or a given one."""
import pytest
import torch

from paged_kv_cache_309_gb300 import pa
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

B, H, G, D, BS, T, BUDGET = 3, 2, 4, 128, 16, 1024, 256


def state():
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(4)
    nb = 3 * B * T // BS
    x = torch.randn(2, 2000, H, D, generator=g, device="cuda").bfloat16()
    s = dict(key=x[0], value=x[1], lens=torch.tensor([1000, 37, 640], dtype=torch.int32, device="cuda"))
    perm = torch.randperm(nb, generator=g, device="cuda").int()
    s["table"] = perm[:B * T // BS].view(B, -1).contiguous()
    s["dst"] = perm[B * T // BS:B * T // BS + B * BUDGET // BS].view(B, -1).contiguous()
    s["q"] = torch.randn(B, H * G, D, generator=g, device="cuda").bfloat16()
    s["slots"] = torch.randperm(nb * BS, generator=g, device="cuda")[:2000]
    s["q4"] = [torch.randint(0, 60, (nb, BS, H, 80), generator=g, device="cuda", dtype=torch.uint8)
               for _ in range(2)]
    s["bf16"] = [torch.randn(nb, BS, H, D, generator=g, device="cuda").bfloat16() for _ in range(2)]
    s["e4m3"] = [c.to(torch.float8_e4m3fn) for c in s["bf16"]]
    s["back"] = [torch.zeros(2000, H, D, device="cuda") for _ in range(2)]
    s["out"] = torch.zeros_like(s["q"])
    s["sums"] = torch.rand(B, H, T, generator=g, device="cuda")
    s["sums_out"] = torch.zeros_like(s["sums"])
    s["keep"] = torch.zeros(B, H, BUDGET, dtype=torch.int32, device="cuda")
    s["new"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["ws"] = pa.decode_scored_workspace(B, H * G, H, D, T)
    return s


def all_calls(s, stream=None):
    """Every long-context call once; what each leaves, in order."""
    kw = dict(stream=stream)
    yield "write", lambda: pa.pa_reshape_and_cache_q4(s["key"], s["value"], *s["q4"], s["slots"], **kw)
    yield "gather", lambda: pa.pa_gather_cache_q4(*s["back"], *s["q4"], s["slots"], **kw)
    yield "decode", lambda: pa.pa_paged_decode_attention_q4(
        s["out"], s["q"], *s["q4"], s["table"], s["lens"], D ** -0.5, T, s["ws"], **kw)
    for cache in ("q4", "bf16", "e4m3"):
        yield "scored " + cache, lambda: pa.pa_paged_decode_attention_scored(
            s["out"], s["sums_out"], s["sums"], 1, s["q"], *s[cache], s["table"], s["lens"], D ** -0.5,
            T, s["ws"], **kw)
    yield "select", lambda: pa.pa_evict_select(s["keep"], s["new"], s["sums_out"], s["sums"], s["lens"],
                                               BUDGET, 4, 16, **kw)
    yield "select paged", lambda: pa.pa_evict_select_paged(
        s["keep"], s["new"], s["sums_out"], s["sums"], s["lens"], s["table"], BUDGET, 4, 16, BS,
        s["q4"][0].shape[0], **kw)
    for cache in ("q4", "bf16"):
        yield "move " + cache, lambda: pa.pa_cache_compact(*s[cache], s["keep"], s["new"], s["table"],
                                                           s["dst"], **kw)
    yield "move in place", lambda: pa.pa_cache_compact(*s["e4m3"], s["keep"], s["new"], s["table"],
                                                       s["table"], **kw)


def test_no_call_takes_device_memory():
    s = state()
    for _, call in all_calls(s):  # (first calls load their kernels)
        call()
    torch.cuda.synchronize()
    held, (free, _) = torch.cuda.memory_allocated(), torch.cuda.mem_get_info()
    for _ in range(20):
        for _, call in all_calls(s):
            call()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == held
    assert free - torch.cuda.mem_get_info()[0] < 2 << 20  # nothing that grows with the calls
    assert pa.read_device_error(s["ws"]) == 0


def test_no_call_waits_for_the_gpu():
    s = state()
    for _, call in all_calls(s):
        call()
    a = torch.randn(8192, 8192, device="cuda").bfloat16()
    c = torch.empty_like(a)
    torch.cuda.synchronize()
    for name, call in all_calls(s):
        done = torch.cuda.Event()
        for _ in range(60):  # some 40 ms of work ahead of the call
            torch.mm(a, a, out=c)
        done.record()
        call()
        assert not done.query(), name
        torch.cuda.synchronize()


def test_a_given_stream_gives_what_the_current_one_does():
    a, b = state(), state()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for (name, one), (_, two) in zip(all_calls(a), all_calls(b, side)):
        one()
        two()
        torch.cuda.synchronize()
        for k in ("out", "sums_out", "keep", "new"):
            assert torch.equal(a[k], b[k]), (name, k)
        for k in ("q4", "bf16", "e4m3", "back"):
            for x, y in zip(a[k], b[k]):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (name, k)
