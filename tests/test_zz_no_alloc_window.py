"""The promise of every call, for the sliding-window ones: they take no device memory and do not wait
for the GPU, on the current stream or a given one."""
import pytest
import torch

from paged_kv_cache_309_gb300 import pa
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

B, H, G, D, BS, T, N = 3, 2, 4, 128, 16, 1024, 700


def state():
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(4)
    nb = 3 * B * T // BS
    s = dict(lens=torch.tensor([1000, 37, 640], dtype=torch.int32, device="cuda"))
    wide = torch.randn(N, (H * G + 2 * H) * D, generator=g, device="cuda").bfloat16()
    s["rows"] = [wide[:, i * D:j * D].unflatten(1, (j - i, D))
                 for i, j in ((0, H * G), (H * G, H * G + H), (H * G + H, H * G + 2 * H))]
    s["turned"] = torch.zeros(N, H * G, D, dtype=torch.bfloat16, device="cuda")
    s["cos_sin"] = torch.randn(4096, 64, generator=g, device="cuda")
    s["pos"] = torch.randint(0, 4096, (N,), generator=g, device="cuda")
    s["slots"] = torch.randperm(nb * BS, generator=g, device="cuda")[:N]
    perm = torch.randperm(nb, generator=g, device="cuda").int()
    s["table"] = perm[:B * T // BS].view(B, -1).contiguous()
    s["q"] = torch.randn(B, H * G, D, generator=g, device="cuda").bfloat16()
    s["bf16"] = [torch.randn(nb, BS, H, D, generator=g, device="cuda").bfloat16() for _ in range(2)]
    s["e4m3"] = [c.to(torch.float8_e4m3fn) for c in s["bf16"]]
    s["scales"] = [torch.tensor([x], device="cuda") for x in (0.05, 0.3)]
    s["out"], s["prompt_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["turned"])
    s["starts"] = torch.tensor([0, 400, 437, N], dtype=torch.int32, device="cuda")
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["ws"] = pa.window_decode_workspace(B, H * G, H, D, 500, 4, T)
    return s


def all_calls(s, stream=None):
    kw = dict(stream=stream)
    for cache in ("bf16", "e4m3"):
        sc = dict(zip(("k_scale", "v_scale"), s["scales"])) if cache == "e4m3" else {}
        yield "append " + cache, lambda: pa.pa_rope_and_cache(
            s["turned"], *s["rows"], *s[cache], s["cos_sin"], s["pos"], s["slots"], **sc, **kw)
        for window in (500, 40):  # cut, and whole
            yield "decode " + cache, lambda: pa.pa_paged_window_decode_attention(
                s["out"], s["q"], *s[cache], s["table"], s["lens"], window, 4, D ** -0.5, T, s["ws"], **sc, **kw)
    yield "prefill", lambda: pa.pa_paged_window_prefill_attention(
        s["prompt_out"], s["turned"], *s["bf16"], s["table"], s["starts"], s["lens"], 100, 4, D ** -0.5, 400,
        s["err"], **kw)


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
    assert pa.read_device_error(s["ws"]) == 0 and int(s["err"]) == 0


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
        for k in ("out", "turned", "prompt_out"):
            assert torch.equal(a[k], b[k]), (name, k)
        for k in ("bf16", "e4m3"):
            for x, y in zip(a[k], b[k]):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (name, k)
