"""Thin ctypes binding of libpa.so, same names as the C ABI (include/pa.h).

Argument marshalling only: each function turns torch tensors into device
pointers, sizes and strides, passes the current (or given) CUDA stream and
raises ``PAError`` on a non-OK status.  All computation happens in the CUDA
library; there is no fallback: if ``libpa.so`` is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpa.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "pa.h")

PA_OK, PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_ERR_ALIGN, PA_ERR_WORKSPACE, PA_ERR_CUDA = range(6)
PA_BF16, PA_FP16, PA_FP32, PA_FP8_E4M3, PA_Q4 = range(5)
PA_DEVERR_WAIT_TIMEOUT = 0x1
PA_DEVERR_CONTEXT_CLIPPED = 0x2
PA_DEVERR_SLOT_MISMATCH = 0x4

_TORCH_DTYPE = {torch.bfloat16: PA_BF16, torch.float16: PA_FP16, torch.float32: PA_FP32,
                torch.float8_e4m3fn: PA_FP8_E4M3}

_lib = None


class PAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _load().pa_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: {msg}")


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build the CUDA library first "
                           "(paged_kv_cache_309_gb300.build.build())")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, F32, SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                            ctypes.c_size_t)
    E = ctypes.c_int  # enums
    lib.pa_status_string.argtypes = [E]
    lib.pa_status_string.restype = ctypes.c_char_p
    lib.pa_reshape_and_cache.argtypes = [P, P, E, I64, I32, I32, I64, I64, P, P, E, I64, I32, I64,
                                         P, P, I64, P, P, P]
    lib.pa_reshape_and_cache.restype = E
    lib.pa_concat_mla_k.argtypes = [P, E, P, P, E, I64, I32, I32, I32, I64, I64, I64, I64, I64, P]
    lib.pa_concat_mla_k.restype = E
    lib.pa_concat_and_cache_mla.argtypes = [P, P, E, I64, I32, I32, I64, I64, P, E, I64, I32,
                                            I64, P, P, P]
    lib.pa_concat_and_cache_mla.restype = E
    lib.pa_paged_decode_workspace_size.argtypes = [I32, I32, I32, I32, I32]
    lib.pa_paged_decode_workspace_size.restype = SZ
    lib.pa_paged_decode_attention.argtypes = [P, P, P, P, E, P, P, I32, I32, I32, I32, I32, I32,
                                              I64, F32, I32, P, SZ, P]
    lib.pa_paged_decode_attention.restype = E
    lib.pa_paged_decode_attention_fp8.argtypes = [P, P, P, P, P, P, P, P, I32, I32, I32, I32,
                                                  I32, I32, I64, F32, I32, P, SZ, P]
    lib.pa_paged_decode_attention_fp8.restype = E
    lib.pa_paged_decode_step.argtypes = [P, P, P, P, P, P, P, E, P, P, P, P, I32, I32, I32, I32,
                                         I32, I32, I64, F32, I32, P, SZ, P]
    lib.pa_paged_decode_step.restype = E
    lib.pa_paged_prefill_attention.argtypes = [P, P, P, P, E, P, P, P, I32, I32, I32, I32, I32,
                                               I32, I64, F32, I32, P, P]
    lib.pa_paged_prefill_attention.restype = E
    lib.pa_paged_decode_attention_static.argtypes = [P, P, P, P, E, P, P, I32, I32, I32, I32,
                                                     I32, I32, I64, F32, I32, P, P]
    lib.pa_paged_decode_attention_static.restype = E
    lib.pa_paged_decode_plan.argtypes = [I32, I32, I32, I32, ctypes.POINTER(I32),
                                         ctypes.POINTER(I32)]
    lib.pa_paged_decode_plan.restype = E
    lib.pa_mla_absorb_q.argtypes = [P, P, P, P, I32, I32, I32, I32, I32, P]
    lib.pa_mla_absorb_q.restype = E
    lib.pa_mla_decode_workspace_size.argtypes = [I32, I32, I32]
    lib.pa_mla_decode_workspace_size.restype = SZ
    lib.pa_mla_decode_attention.argtypes = [P, P, P, P, P, I32, I32, I32, I32, I32, I32, I64,
                                            ctypes.c_float, I32, P, SZ, P]
    lib.pa_mla_decode_attention.restype = E
    lib.pa_mla_project_out.argtypes = [P, P, P, I32, I32, I32, I32, P]
    lib.pa_mla_project_out.restype = E
    lib.pa_selftest_bounded_wait.argtypes = [P, P]
    lib.pa_selftest_bounded_wait.restype = E
    lib.pa_reshape_and_cache_q4.argtypes = [P, P, E, I64, I32, I32, I64, I64, P, P, I64, I32, I64,
                                            P, P, I64, P]
    lib.pa_reshape_and_cache_q4.restype = E
    lib.pa_gather_cache_q4.argtypes = [P, P, E, I64, I32, I32, I64, I64, P, P, I64, I32, I64, P, P]
    lib.pa_gather_cache_q4.restype = E
    lib.pa_paged_decode_attention_q4.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32,
                                                 I64, F32, I32, P, SZ, P]
    lib.pa_paged_decode_attention_q4.restype = E
    lib.pa_paged_decode_scored_workspace_size.argtypes = [I32, I32, I32, I32, I32]
    lib.pa_paged_decode_scored_workspace_size.restype = SZ
    lib.pa_paged_decode_attention_scored.argtypes = [P, P, P, I32, I32, P, P, P, E, P, P, P, P, I32,
                                                     I32, I32, I32, I32, I32, I64, F32, I32, P, SZ,
                                                     P]
    lib.pa_paged_decode_attention_scored.restype = E
    lib.pa_evict_select.argtypes = [P, P, P, P, P, I32, I32, I32, I32, I32, I32, P]
    lib.pa_evict_select.restype = E
    lib.pa_evict_select_paged.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, I32, I32,
                                          I64, P]
    lib.pa_evict_select_paged.restype = E
    lib.pa_cache_compact.argtypes = [P, P, I32, P, P, I32, P, I32, P, I32, I32, I32, I32, I64, P]
    lib.pa_cache_compact.restype = E
    lib.pa_rope_and_cache.argtypes = [P, P, P, P, E, I64, I32, I32, I32, I64, I64, I64, I64, P, P,
                                      I64, I32, I32, P, P, E, I64, I32, I64, P, P, I64, P, P, P]
    lib.pa_rope_and_cache.restype = E
    lib.pa_paged_window_decode_workspace_size.argtypes = [I32] * 7
    lib.pa_paged_window_decode_workspace_size.restype = SZ
    lib.pa_paged_window_decode_attention.argtypes = [P, P, P, P, E, P, P, P, P, I32, I32, I32, I32,
                                                     I32, I32, I64, I32, I32, F32, I32, P, SZ, P]
    lib.pa_paged_window_decode_attention.restype = E
    lib.pa_paged_window_prefill_attention.argtypes = [P, P, P, P, E, P, P, P, I32, I32, I32, I32,
                                                      I32, I32, I64, I32, I32, F32, I32, I64, P, P]
    lib.pa_paged_window_prefill_attention.restype = E
    _lib = lib
    return lib


def library():
    """The loaded ctypes library (raises if it was not built)."""
    return _load()


def declared_functions():
    """Names of the functions include/pa.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(pa_[a-z0-9_]+)\s*\(", text)))


def _check(status, where):
    if status != PA_OK:
        raise PAError(status, where)


def _on_device(**tensors):
    """Refuse, before anything is launched, a tensor the kernels cannot use:
    every tensor passed (None is skipped) must be a CUDA tensor on the
    current CUDA device, because the library takes its pointers as device
    addresses of that device (a host or another GPU's pointer would be
    dereferenced as one)."""
    cur = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch tensor")
        device = t.get_device()  # -1 on the host
        if device == cur:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (it is on {t.device})")
        if cur is None:
            cur = torch.cuda.current_device()
        if device != cur:
            raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{cur}")


def _word(t, name):
    """A device word the kernels OR 4-byte error bits into: int32, at least
    one element, on the current device."""
    if t is None:
        return
    _on_device(**{name: t})
    if t.dtype != torch.int32 or t.numel() < 1:
        raise ValueError(f"{name} must be an int32 tensor with at least one element")


def _scales(k_scale, v_scale):
    """k_scale/v_scale: both None, or both one-element float32 device tensors."""
    if (k_scale is None) != (v_scale is None):
        raise ValueError("give both k_scale and v_scale, or neither")
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t is None:
            continue
        _on_device(**{name: t})
        if t.dtype != torch.float32 or t.numel() < 1:
            raise ValueError(f"{name} must be a float32 tensor with at least one element")


def _workspace(t):
    """A decode workspace: a uint8 device tensor on the current device."""
    _on_device(workspace=t)
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:  # the raw handle (a private call) where torch has it: a Stream object costs 3 us
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            return torch.cuda.current_stream().cuda_stream
        return raw(torch.cuda.current_device())
    if stream.device.index != torch.cuda.current_device():
        raise ValueError(f"stream belongs to {stream.device}, not the current device")
    return stream.cuda_stream


def _dtype(t):
    try:
        return _TORCH_DTYPE[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}") from None


def pa_reshape_and_cache(key, value, key_cache, value_cache, slot_mapping,
                         swa_slot_mapping=None, k_scale=None, v_scale=None, stream=None):
    """key/value [N, H, d] (token stride free), caches [num_blocks, bs, H, d]
    (block stride free), slot_mapping [N] int64, optional swa table int64,
    optional k_scale/v_scale one-element float32 device tensors."""
    _on_device(key=key, value=value, key_cache=key_cache, value_cache=value_cache,
               slot_mapping=slot_mapping, swa_slot_mapping=swa_slot_mapping)
    _scales(k_scale, v_scale)
    lib = _load()
    N, H, d = key.shape
    if key.stride(2) != 1 or key.stride(1) != d:
        raise ValueError("key: heads and elements must be contiguous")
    if value is not None and (value.shape != key.shape or value.stride(2) != 1
                              or value.stride(1) != d):
        raise ValueError("value must match key and be contiguous per token")
    nb, bs, Hc, dc = key_cache.shape
    if (Hc, dc) != (H, d) or key_cache.stride(3) != 1 or key_cache.stride(2) != d \
            or key_cache.stride(1) != H * d:
        raise ValueError("key_cache must be [num_blocks, bs, H, d], contiguous inside a block")
    if value_cache is not None and (value_cache.shape != key_cache.shape
                                    or value_cache.stride() != key_cache.stride()
                                    or value_cache.dtype != key_cache.dtype):
        raise ValueError("value_cache must match key_cache")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != N:
        raise ValueError("slot_mapping must be int64 [N]")
    swa_len = 0
    if swa_slot_mapping is not None:
        if swa_slot_mapping.dtype != torch.int64:
            raise ValueError("swa_slot_mapping must be int64")
        swa_len = swa_slot_mapping.numel()
    st = lib.pa_reshape_and_cache(
        _ptr(key), _ptr(value), _dtype(key), N, H, d, key.stride(0),
        0 if value is None else value.stride(0), _ptr(key_cache), _ptr(value_cache),
        _dtype(key_cache), nb, bs, key_cache.stride(0), _ptr(slot_mapping),
        _ptr(swa_slot_mapping), swa_len, _ptr(k_scale), _ptr(v_scale), _stream(stream))
    _check(st, "pa_reshape_and_cache")


def pa_concat_mla_k(k, k_nope, k_rope, stream=None):
    """k [N, H, nope+rope] <- k_nope [N, H, nope] | k_rope [N, 1, rope]."""
    _on_device(k=k, k_nope=k_nope, k_rope=k_rope)
    lib = _load()
    N, H, nope = k_nope.shape
    rope = k_rope.shape[2]
    for t in (k, k_nope, k_rope):
        if t.stride(2) != 1:
            raise ValueError("last dimension must be contiguous")
    if k.shape != (N, H, nope + rope) or k_rope.shape[:2] != (N, 1):
        raise ValueError("shape mismatch")
    if k_rope.dtype != k_nope.dtype:
        raise ValueError("k_nope and k_rope must share a dtype")
    st = lib.pa_concat_mla_k(_ptr(k), _dtype(k), _ptr(k_nope), _ptr(k_rope), _dtype(k_nope), N, H,
                             nope, rope, k.stride(0), k.stride(1), k_nope.stride(0),
                             k_nope.stride(1), k_rope.stride(0), _stream(stream))
    _check(st, "pa_concat_mla_k")


def pa_concat_and_cache_mla(kv_c, k_pe, latent_cache, slot_mapping, scale=None, stream=None):
    """latent_cache [num_blocks, bs, (1,) d_c + d_r] <- [kv_c[t] | k_pe[t]] at
    slot_mapping[t] (int64 [N]; negative or out-of-pool slots skipped);
    kv_c [N, d_c] and k_pe [N, d_r] (token stride free, rows contiguous);
    optional scale: one-element float32 device tensor (x / scale before the
    cast)."""
    _on_device(kv_c=kv_c, k_pe=k_pe, latent_cache=latent_cache, slot_mapping=slot_mapping)
    if scale is not None:
        _on_device(scale=scale)
        if scale.dtype != torch.float32 or scale.numel() < 1:
            raise ValueError("scale must be a float32 tensor with at least one element")
    lib = _load()
    kc = kv_c.view(kv_c.shape[0], -1) if kv_c.dim() == 3 else kv_c
    kp = k_pe.view(k_pe.shape[0], -1) if k_pe.dim() == 3 else k_pe
    N, dc = kc.shape
    dr = kp.shape[1]
    if kp.shape[0] != N or kc.stride(1) != 1 or kp.stride(1) != 1:
        raise ValueError("kv_c [N, d_c] and k_pe [N, d_r] with contiguous rows expected")
    if kp.dtype != kc.dtype:
        raise ValueError("kv_c and k_pe must share a dtype")
    nb, bs = latent_cache.shape[0], latent_cache.shape[1]
    if latent_cache.shape[-1] != dc + dr or latent_cache.numel() != nb * bs * (dc + dr) \
            or not latent_cache.is_contiguous():
        raise ValueError("latent_cache must be [num_blocks, bs, (1,) d_c + d_r], contiguous")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != N:
        raise ValueError("slot_mapping must be int64 [N]")
    st = lib.pa_concat_and_cache_mla(
        _ptr(kc), _ptr(kp), _dtype(kc), N, dc, dr, kc.stride(0), kp.stride(0),
        _ptr(latent_cache), _dtype(latent_cache), nb, bs, bs * (dc + dr), _ptr(slot_mapping),
        _ptr(scale), _stream(stream))
    _check(st, "pa_concat_and_cache_mla")


def pa_paged_decode_plan(num_seqs, num_kv_heads, max_context_len, num_sms=0):
    """(num_splits, tokens_per_split) of the decode split plan."""
    lib = _load()
    a, b = ctypes.c_int32(), ctypes.c_int32()
    _check(lib.pa_paged_decode_plan(num_seqs, num_kv_heads, max_context_len, num_sms,
                                    ctypes.byref(a), ctypes.byref(b)), "pa_paged_decode_plan")
    return a.value, b.value


def pa_paged_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_size,
                                   max_context_len):
    return int(_load().pa_paged_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads,
                                                      head_size, max_context_len))


def decode_workspace(num_seqs, num_q_heads, num_kv_heads, head_size, max_context_len,
                     device=None):
    """A zeroed device workspace of the required size (allocated by torch)."""
    n = pa_paged_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_size,
                                       max_context_len)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def read_device_error(workspace) -> int:
    """The sticky device-side error word (first 4 bytes of the workspace)."""
    return int(workspace[:4].view(torch.int32).item())


def pa_paged_decode_attention(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                              max_context_len, workspace, stream=None, k_scale=None,
                              v_scale=None):
    """out/q [B, H_Q, d] bf16; caches [num_blocks, bs, H_KV, d] bf16 or
    float8_e4m3fn, contiguous; block_tables [B, max_blocks_per_seq] int32;
    context_lens [B] int32.  With k_scale/v_scale (one-element float32 device
    tensors) the e4m3 cache goes through pa_paged_decode_attention_fp8."""
    _on_device(out=out, q=q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
               context_lens=context_lens)
    _workspace(workspace)
    _scales(k_scale, v_scale)
    lib = _load()
    B, HQ, d = q.shape
    nb, bs, HKV, dc = k_cache.shape
    for t, name in ((q, "q"), (out, "out"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                    (block_tables, "block_tables"), (context_lens, "context_lens")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if out.shape != q.shape or v_cache.shape != k_cache.shape or dc != d:
        raise ValueError("shape mismatch")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.numel() != B:
        raise ValueError("block_tables must be [B, max_blocks_per_seq], context_lens [B]")
    if q.dtype != torch.bfloat16 or out.dtype != torch.bfloat16:
        raise ValueError("q and out must be bf16")
    if k_scale is not None or v_scale is not None:
        if k_cache.dtype != torch.float8_e4m3fn:
            raise ValueError("k_scale/v_scale apply to an e4m3 cache")
        st = lib.pa_paged_decode_attention_fp8(
            _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
            _ptr(block_tables), _ptr(context_lens), B, HQ, HKV, d, bs, block_tables.shape[1], nb,
            float(scale), int(max_context_len), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))
        _check(st, "pa_paged_decode_attention_fp8")
        return
    st = lib.pa_paged_decode_attention(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _dtype(k_cache), _ptr(block_tables),
        _ptr(context_lens), B, HQ, HKV, d, bs, block_tables.shape[1], nb, float(scale),
        int(max_context_len), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check(st, "pa_paged_decode_attention")


def pa_paged_decode_attention_static(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                                     max_context_len, error_word=None, stream=None):
    """Decode attention without a caller workspace: the split-K partials go
    to the library's own 16 MiB device scratch (for callers that cannot
    allocate device memory).  error_word: None or a one-element int32 device
    tensor that receives the device-side error bits.  Calls sharing the
    scratch must be ordered on one stream."""
    _on_device(out=out, q=q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
               context_lens=context_lens)
    _word(error_word, "error_word")
    lib = _load()
    B, HQ, d = q.shape
    nb, bs, HKV, dc = k_cache.shape
    for t, name in ((q, "q"), (out, "out"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                    (block_tables, "block_tables"), (context_lens, "context_lens")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if out.shape != q.shape or v_cache.shape != k_cache.shape or dc != d:
        raise ValueError("shape mismatch")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    st = lib.pa_paged_decode_attention_static(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _dtype(k_cache), _ptr(block_tables),
        _ptr(context_lens), B, HQ, HKV, d, bs, block_tables.shape[1], nb, float(scale),
        int(max_context_len), _ptr(error_word), _stream(stream))
    _check(st, "pa_paged_decode_attention_static")


def pa_paged_decode_step(out, q, new_k, new_v, slot_mapping, k_cache, v_cache, block_tables,
                         context_lens, scale, max_context_len, workspace, k_scale=None,
                         v_scale=None, stream=None):
    """One decode step in one launch: new_k/new_v [B, H_KV, d] bf16 are
    written at slot_mapping [B] int64 (bf16 cache, or e4m3 cache with
    k_scale/v_scale), then attention over the cache as in
    pa_paged_decode_attention."""
    _on_device(out=out, q=q, new_k=new_k, new_v=new_v, slot_mapping=slot_mapping,
               k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
               context_lens=context_lens)
    _workspace(workspace)
    _scales(k_scale, v_scale)
    lib = _load()
    B, HQ, d = q.shape
    nb, bs, HKV, dc = k_cache.shape
    for t, name in ((q, "q"), (out, "out"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                    (new_k, "new_k"), (new_v, "new_v"), (block_tables, "block_tables"),
                    (context_lens, "context_lens"), (slot_mapping, "slot_mapping")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if new_k.shape != (B, HKV, d) or new_v.shape != (B, HKV, d) or new_k.dtype != torch.bfloat16:
        raise ValueError("new_k/new_v must be bf16 [B, H_KV, d]")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != B:
        raise ValueError("slot_mapping must be int64 [B]")
    st = lib.pa_paged_decode_step(
        _ptr(out), _ptr(q), _ptr(new_k), _ptr(new_v), _ptr(slot_mapping), _ptr(k_cache),
        _ptr(v_cache), _dtype(k_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_tables),
        _ptr(context_lens), B, HQ, HKV, d, bs, block_tables.shape[1], nb, float(scale),
        int(max_context_len), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check(st, "pa_paged_decode_step")


def pa_paged_prefill_attention(out, q, k_cache, v_cache, block_tables, cu_seqlens_q,
                               context_lens, scale, max_q_len, error_word, stream=None):
    """Causal varlen prefill: q/out [total_new, H_Q, d] bf16, caches
    [num_blocks, bs, H_KV, d] bf16, cu_seqlens_q [B+1] int32, context_lens [B]
    int32 (tokens including the new ones), error_word one int32 on the device."""
    if error_word is None:
        raise ValueError("error_word is required")
    _on_device(out=out, q=q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
               cu_seqlens_q=cu_seqlens_q, context_lens=context_lens)
    _word(error_word, "error_word")
    lib = _load()
    T, HQ, d = q.shape
    nb, bs, HKV, dc = k_cache.shape
    B = context_lens.numel()
    for t, name in ((q, "q"), (out, "out"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                    (block_tables, "block_tables"), (cu_seqlens_q, "cu_seqlens_q"),
                    (context_lens, "context_lens")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if out.shape != q.shape or cu_seqlens_q.numel() != B + 1 or dc != d:
        raise ValueError("shape mismatch")
    if cu_seqlens_q.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("cu_seqlens_q and context_lens must be int32")
    st = lib.pa_paged_prefill_attention(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _dtype(k_cache), _ptr(block_tables),
        _ptr(cu_seqlens_q), _ptr(context_lens), B, HQ, HKV, d, bs, block_tables.shape[1], nb,
        float(scale), int(max_q_len), _ptr(error_word), _stream(stream))
    _check(st, "pa_paged_prefill_attention")


def pa_selftest_bounded_wait(error_word, stream=None):
    """Diagnostic: one CTA's bounded wait on a barrier nothing completes runs
    out (2 s) and sets PA_DEVERR_WAIT_TIMEOUT (1) in error_word, a one-element
    int32 device tensor the caller cleared."""
    if error_word is None:
        raise ValueError("error_word is required")
    _word(error_word, "error_word")
    st = _load().pa_selftest_bounded_wait(_ptr(error_word), _stream(stream))
    _check(st, "pa_selftest_bounded_wait")


# ------------------------------------------------------------- MLA decode --
def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def pa_mla_absorb_q(q_latent, q_nope, q_pe, w_uk, stream=None):
    """q_latent [B, H, d_c + d_r] <- [W_UK_h q_nope[b, h] | q_pe[b, h]];
    q_nope [B, H, d_h], q_pe [B, H, d_r], w_uk [d_c, H * d_h], all bf16."""
    _on_device(q_latent=q_latent, q_nope=q_nope, q_pe=q_pe, w_uk=w_uk)
    B, H, dh = q_nope.shape
    dr = q_pe.shape[2]
    dc = w_uk.shape[0]
    for t in (q_latent, q_nope, q_pe, w_uk):
        _need(t.is_contiguous() and t.dtype == torch.bfloat16, "bf16 contiguous tensors expected")
    _need(q_latent.shape == (B, H, dc + dr) and q_pe.shape[:2] == (B, H)
          and w_uk.shape == (dc, H * dh), "shape mismatch")
    _check(_load().pa_mla_absorb_q(_ptr(q_latent), _ptr(q_nope), _ptr(q_pe), _ptr(w_uk), B, H,
                                   dh, dr, dc, _stream(stream)), "pa_mla_absorb_q")


def pa_mla_decode_workspace_size(num_seqs, num_heads, max_context_len):
    return int(_load().pa_mla_decode_workspace_size(num_seqs, num_heads, max_context_len))


def mla_decode_workspace(num_seqs, num_heads, max_context_len, device=None):
    """A zeroed device workspace for pa_mla_decode_attention (allocated by torch)."""
    n = pa_mla_decode_workspace_size(num_seqs, num_heads, max_context_len)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def pa_mla_decode_attention(out_latent, q_latent, latent_cache, block_tables, context_lens,
                            scale, max_context_len, workspace, latent_dim=512, stream=None):
    """out_latent [B, H, d_c] bf16; q_latent [B, H, d_c + d_r] bf16;
    latent_cache [num_blocks, bs, (1,) d_c + d_r] bf16; block_tables
    [B, max_blocks_per_seq] int32; context_lens [B] int32."""
    _on_device(out_latent=out_latent, q_latent=q_latent, latent_cache=latent_cache,
               block_tables=block_tables, context_lens=context_lens)
    _workspace(workspace)
    B, H, dk = q_latent.shape
    nb, bs = latent_cache.shape[0], latent_cache.shape[1]
    for t, name in ((out_latent, "out_latent"), (q_latent, "q_latent"),
                    (latent_cache, "latent_cache"), (block_tables, "block_tables"),
                    (context_lens, "context_lens")):
        _need(t.is_contiguous(), f"{name} must be contiguous")
    _need(latent_cache.shape[-1] == dk and latent_cache.numel() == nb * bs * dk,
          "latent_cache must be [num_blocks, bs, (1,) d_c + d_r]")
    _need(out_latent.shape == (B, H, latent_dim), "out_latent must be [B, H, d_c]")
    _need(q_latent.dtype == torch.bfloat16 and out_latent.dtype == torch.bfloat16
          and latent_cache.dtype == torch.bfloat16, "bf16 tensors expected")
    _need(block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32,
          "block_tables and context_lens must be int32")
    _need(block_tables.dim() == 2 and block_tables.shape[0] == B and context_lens.numel() == B,
          "block_tables must be [B, max_blocks_per_seq], context_lens [B]")
    st = _load().pa_mla_decode_attention(
        _ptr(out_latent), _ptr(q_latent), _ptr(latent_cache), _ptr(block_tables),
        _ptr(context_lens), B, H, latent_dim, dk - latent_dim, bs, block_tables.shape[1], nb,
        float(scale), int(max_context_len), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "pa_mla_decode_attention")


def pa_mla_project_out(out, out_latent, w_uv, stream=None):
    """out [B, H, d_v] <- out_latent[b, h, :] W_UV_h; out_latent [B, H, d_c],
    w_uv [d_c, H * d_v], all bf16."""
    _on_device(out=out, out_latent=out_latent, w_uv=w_uv)
    B, H, dc = out_latent.shape
    dv = out.shape[2]
    for t in (out, out_latent, w_uv):
        _need(t.is_contiguous() and t.dtype == torch.bfloat16, "bf16 contiguous tensors expected")
    _need(out.shape[:2] == (B, H) and w_uv.shape == (dc, H * dv), "shape mismatch")
    _check(_load().pa_mla_project_out(_ptr(out), _ptr(out_latent), _ptr(w_uv), B, H, dc, dv,
                                      _stream(stream)), "pa_mla_project_out")


def _i32(name, value):
    """value as a C int32; ctypes would keep its low 32 bits without a word."""
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{name} does not fit 32 bits")
    return int(value)


# ------------------------------------------------------------ 4-bit cache --
def q4_row_bytes(head_size):
    """Bytes of a kv head's row in a 4-bit cache: head_size / 2 of codes, then
    an fp16 (scale, minimum) pair for each group of 32 elements."""
    if head_size <= 0 or head_size % 32 != 0:
        raise ValueError("head_size must be a multiple of 32")
    return 5 * head_size // 8


def _q4_shapes(key, value, key_cache, value_cache, slot_mapping):
    """Checks shared by the 4-bit write and gather: (N, H, d, num_blocks, bs)."""
    shape = key.shape
    N, H, d = shape
    if key.stride(2) != 1 or key.stride(1) != d:
        raise ValueError("key: [N, H, d] with heads and elements contiguous expected")
    if (value is None) != (value_cache is None):
        raise ValueError("give both value and value_cache, or neither")
    if value is not None and (value.shape != shape or value.dtype != key.dtype
                              or value.stride(2) != 1 or value.stride(1) != d):
        raise ValueError("value must match key, heads and elements contiguous")
    nb, bs, Hc, rb = key_cache.shape
    strides = key_cache.stride()
    if key_cache.dtype != torch.uint8 or Hc != H or rb != q4_row_bytes(d) \
            or strides[1:] != (H * rb, rb, 1):
        raise ValueError("key_cache must be uint8 [num_blocks, bs, H, 5 * d / 8], contiguous "
                         "inside a block")
    if value_cache is not None and (value_cache.shape != key_cache.shape
                                    or value_cache.stride() != strides
                                    or value_cache.dtype != torch.uint8):
        raise ValueError("value_cache must match key_cache")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != N \
            or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be int64 [N]")
    return N, H, d, nb, bs


def pa_reshape_and_cache_q4(key, value, key_cache, value_cache, slot_mapping,
                            swa_slot_mapping=None, stream=None):
    """key/value [N, H, d] (token stride free) quantised into 4-bit caches
    uint8 [num_blocks, bs, H, 5 * d / 8] (block stride free); slot_mapping [N]
    int64, optional swa table int64.  value and value_cache may be None."""
    _on_device(key=key, value=value, key_cache=key_cache, value_cache=value_cache,
               slot_mapping=slot_mapping, swa_slot_mapping=swa_slot_mapping)
    N, H, d, nb, bs = _q4_shapes(key, value, key_cache, value_cache, slot_mapping)
    swa_len = 0
    if swa_slot_mapping is not None:
        if swa_slot_mapping.dtype != torch.int64 or not swa_slot_mapping.is_contiguous():
            raise ValueError("swa_slot_mapping must be int64, contiguous")
        swa_len = swa_slot_mapping.numel()
    st = _load().pa_reshape_and_cache_q4(
        _ptr(key), _ptr(value), _dtype(key), N, H, d, key.stride(0),
        0 if value is None else value.stride(0), _ptr(key_cache), _ptr(value_cache), nb, bs,
        key_cache.stride(0), _ptr(slot_mapping), _ptr(swa_slot_mapping), swa_len,
        _stream(stream))
    _check(st, "pa_reshape_and_cache_q4")


def pa_gather_cache_q4(key, value, key_cache, value_cache, slot_mapping, stream=None):
    """key/value [N, H, d] bf16, fp16 or fp32 (written) <- the rows of the
    4-bit caches at slot_mapping [N] int64; rows of negative or out-of-pool
    slots are left as they were.  value and value_cache may be None."""
    _on_device(key=key, value=value, key_cache=key_cache, value_cache=value_cache,
               slot_mapping=slot_mapping)
    N, H, d, nb, bs = _q4_shapes(key, value, key_cache, value_cache, slot_mapping)
    st = _load().pa_gather_cache_q4(
        _ptr(key), _ptr(value), _dtype(key), N, H, d, key.stride(0),
        0 if value is None else value.stride(0), _ptr(key_cache), _ptr(value_cache), nb, bs,
        key_cache.stride(0), _ptr(slot_mapping), _stream(stream))
    _check(st, "pa_gather_cache_q4")


def _decode_shapes(out, q, k_cache, v_cache, block_tables, context_lens, workspace):
    """Checks shared by the calls below: (B, H_Q, H_KV, d, block_size, num_blocks)."""
    _on_device(out=out, q=q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
               context_lens=context_lens, workspace=workspace)
    B, HQ, d = q.shape
    shape = k_cache.shape
    nb, bs, HKV, row = shape
    kind = k_cache.dtype
    if not (q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous()
            and v_cache.is_contiguous() and block_tables.is_contiguous()
            and context_lens.is_contiguous() and workspace.is_contiguous()):
        raise ValueError("out, q, caches, block_tables, context_lens and workspace must be "
                         "contiguous")
    if q.dtype != torch.bfloat16 or out.dtype != torch.bfloat16 or out.shape != q.shape:
        raise ValueError("q and out must be bf16 [B, H_Q, d]")
    if v_cache.dtype != kind or v_cache.shape != shape:
        raise ValueError("v_cache must match k_cache")
    if row != (q4_row_bytes(d) if kind == torch.uint8 else d):
        raise ValueError("cache rows must be d elements, or 5 * d / 8 bytes of a 4-bit cache "
                         "(uint8)")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.numel() != B:
        raise ValueError("block_tables must be [B, max_blocks_per_seq], context_lens [B]")
    return B, HQ, HKV, d, bs, nb


def pa_paged_decode_attention_q4(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                                 max_context_len, workspace, stream=None):
    """out/q [B, H_Q, 128] bf16; 4-bit caches uint8 [num_blocks, bs, H_KV, 80],
    contiguous; block_tables [B, max_blocks_per_seq] int32; context_lens [B]
    int32; workspace from decode_workspace."""
    B, HQ, HKV, d, bs, nb = _decode_shapes(out, q, k_cache, v_cache, block_tables, context_lens,
                                           workspace)
    if k_cache.dtype != torch.uint8:
        raise ValueError("a 4-bit cache (uint8 rows) is expected")
    max_context_len = _i32("max_context_len", max_context_len)
    st = _load().pa_paged_decode_attention_q4(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        B, HQ, HKV, d, bs, block_tables.shape[1], nb, float(scale),
        max_context_len,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "pa_paged_decode_attention_q4")


# ------------------------------------------------ attention weights, eviction --
def pa_paged_decode_scored_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_size,
                                          max_context_len):
    max_context_len = _i32("max_context_len", max_context_len)
    return int(_load().pa_paged_decode_scored_workspace_size(num_seqs, num_q_heads, num_kv_heads,
                                                             head_size, max_context_len))


def decode_scored_workspace(num_seqs, num_q_heads, num_kv_heads, head_size, max_context_len,
                            device=None):
    """A zeroed device workspace for pa_paged_decode_attention_scored (allocated by torch)."""
    n = pa_paged_decode_scored_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_size,
                                              max_context_len)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def _sums(sums, sums_out, B, H):
    """Checks of the accumulated weights (their device apart): tokens per row."""
    shape = sums.shape
    if len(shape) != 3 or shape[0] != B or shape[1] != H or sums.dtype != torch.float32 \
            or not sums.is_contiguous():
        raise ValueError("sums must be float32 [B, H_KV, tokens], contiguous")
    if sums_out is not None and sums_out is not sums and (
            sums_out.shape != shape or sums_out.dtype != torch.float32
            or not sums_out.is_contiguous()):
        raise ValueError("sums_out must match sums")
    return shape[2]


def pa_paged_decode_attention_scored(out, sums_out, sums, num_new, q, k_cache, v_cache,
                                     block_tables, context_lens, scale, max_context_len, workspace,
                                     k_scale=None, v_scale=None, stream=None):
    """Decode attention (bf16, float8_e4m3fn with optional scales, or uint8
    4-bit caches) that also adds each token's attention weight, summed over a
    kv head's query heads: sums_out [B, H_KV, T] <- sums + weights, the last
    num_new tokens of a sequence starting from 0.  sums_out may be sums.  While
    the workspace's error word holds a wait timeout, no sum is written.
    workspace from decode_scored_workspace."""
    B, HQ, HKV, d, bs, nb = _decode_shapes(out, q, k_cache, v_cache, block_tables, context_lens,
                                           workspace)
    _on_device(sums=sums, sums_out=sums_out)
    if sums_out is None:
        raise ValueError("sums_out is required")
    tokens = _sums(sums, sums_out, B, HKV)
    if k_scale is not None or v_scale is not None:
        _scales(k_scale, v_scale)
        if k_cache.dtype != torch.float8_e4m3fn:
            raise ValueError("k_scale/v_scale apply to an e4m3 cache")
    if num_new < 0:
        raise ValueError("num_new must not be negative")
    max_context_len = _i32("max_context_len", max_context_len)
    dtype = PA_Q4 if k_cache.dtype == torch.uint8 else _dtype(k_cache)
    st = _load().pa_paged_decode_attention_scored(
        _ptr(out), _ptr(sums_out), _ptr(sums), tokens, min(int(num_new), 2 ** 31 - 1),
        _ptr(q), _ptr(k_cache), _ptr(v_cache), dtype, _ptr(k_scale), _ptr(v_scale),
        _ptr(block_tables), _ptr(context_lens), B, HQ, HKV, d, bs, block_tables.shape[1], nb,
        float(scale), max_context_len, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "pa_paged_decode_attention_scored")


def pa_evict_select(keep, new_lens, sums_out, sums, context_lens, budget, num_sink, num_recent,
                    stream=None):
    """keep [B, H_KV, budget] int32 <- the tokens of each row to keep, ascending,
    -1 behind them: the first num_sink and last num_recent, then the largest
    sums [B, H_KV, T] float32 (ties to the lowest token); new_lens [B] int32 <-
    their number; sums_out (None, sums itself or another like it) <- their sums."""
    _on_device(keep=keep, new_lens=new_lens, sums=sums, sums_out=sums_out,
               context_lens=context_lens)
    B, H, tokens, num_sink, num_recent = _select_shapes(keep, new_lens, sums_out, sums,
                                                        context_lens, budget, num_sink, num_recent)
    _check(_load().pa_evict_select(_ptr(keep), _ptr(new_lens), _ptr(sums_out), _ptr(sums),
                                   _ptr(context_lens), B, H, tokens, budget, num_sink,
                                   num_recent, _stream(stream)), "pa_evict_select")


def pa_evict_select_paged(keep, new_lens, sums_out, sums, context_lens, block_tables, budget,
                          num_sink, num_recent, block_size, num_blocks, stream=None):
    """pa_evict_select where block_tables [B, max_blocks_per_seq] int32 may hold
    dropped blocks (ids outside [0, num_blocks)): their tokens are never kept."""
    _on_device(keep=keep, new_lens=new_lens, sums=sums, sums_out=sums_out,
               context_lens=context_lens, block_tables=block_tables)
    B, H, tokens, num_sink, num_recent = _select_shapes(keep, new_lens, sums_out, sums,
                                                        context_lens, budget, num_sink, num_recent)
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 \
            or block_tables.shape[0] != B or not block_tables.is_contiguous():
        raise ValueError("block_tables must be int32 [B, max_blocks_per_seq], contiguous")
    block_size = _i32("block_size", block_size)
    if not 0 <= num_blocks < 2 ** 63:
        raise ValueError("num_blocks must be from 0 to 2^63 - 1")
    _check(_load().pa_evict_select_paged(
        _ptr(keep), _ptr(new_lens), _ptr(sums_out), _ptr(sums), _ptr(context_lens),
        _ptr(block_tables), B, H, tokens, budget, num_sink, num_recent, block_size,
        block_tables.shape[1], int(num_blocks), _stream(stream)), "pa_evict_select_paged")


def _select_shapes(keep, new_lens, sums_out, sums, context_lens, budget, num_sink, num_recent):
    """Checks shared by both choices: (B, H_KV, tokens, num_sink, num_recent)."""
    if keep.dtype != torch.int32 or keep.dim() != 3 or not keep.is_contiguous():
        raise ValueError("keep must be int32 [B, H_KV, budget], contiguous")
    B, H, width = keep.shape
    if width != budget:
        raise ValueError("keep must be [B, H_KV, budget]")
    tokens = _sums(sums, sums_out, B, H)
    for t, name in ((new_lens, "new_lens"), (context_lens, "context_lens")):
        if t.dtype != torch.int32 or t.numel() != B or not t.is_contiguous():
            raise ValueError(f"{name} must be int32 [B]")
    return B, H, tokens, _i32("num_sink", num_sink), _i32("num_recent", num_recent)


def pa_cache_compact(k_cache, v_cache, keep, keep_lens, src_block_tables, dst_block_tables,
                     stream=None):
    """Row j of each (sequence, kv head), read through dst_block_tables, <- its
    row keep[b, g, j], read through src_block_tables, for j < keep_lens[b];
    caches [num_blocks, bs, H_KV, row] of any type (v_cache may be None), rows
    of a multiple of 16 bytes.  In place: pass one table twice (keep
    ascending)."""
    _on_device(k_cache=k_cache, v_cache=v_cache, keep=keep, keep_lens=keep_lens,
               src_block_tables=src_block_tables, dst_block_tables=dst_block_tables)
    if k_cache.dim() != 4 or not k_cache.is_contiguous():
        raise ValueError("k_cache must be [num_blocks, bs, H_KV, row], contiguous")
    if v_cache is not None and (v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype
                                or not v_cache.is_contiguous()):
        raise ValueError("v_cache must match k_cache")
    nb, bs, H, row = k_cache.shape
    if keep.dtype != torch.int32 or keep.dim() != 3 or keep.shape[1] != H \
            or not keep.is_contiguous():
        raise ValueError("keep must be int32 [B, H_KV, n], contiguous")
    B = keep.shape[0]
    if keep_lens.dtype != torch.int32 or keep_lens.numel() != B or not keep_lens.is_contiguous():
        raise ValueError("keep_lens must be int32 [B]")
    for t, name in ((src_block_tables, "src_block_tables"), (dst_block_tables, "dst_block_tables")):
        if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != B or not t.is_contiguous():
            raise ValueError(f"{name} must be int32 [B, blocks], contiguous")
    _check(_load().pa_cache_compact(
        _ptr(k_cache), _ptr(v_cache), row * k_cache.element_size(), _ptr(keep), _ptr(keep_lens),
        keep.shape[2], _ptr(src_block_tables), src_block_tables.shape[1], _ptr(dst_block_tables),
        dst_block_tables.shape[1], B, H, bs, nb, _stream(stream)), "pa_cache_compact")


# --------------------------------------------------------- sliding window --
# These calls come once per layer and token, where the host's time is what counts: their checks
# read each tensor's properties once, and the messages are made where a check failed.
def _all_here(*tensors):
    """Whether every tensor is a CUDA tensor on the current device: that device, else -1."""
    try:
        cur = tensors[0].get_device()
        for t in tensors:
            if t.get_device() != cur:
                return -1
    except AttributeError:
        return -1
    return cur if cur >= 0 and cur == torch.cuda.current_device() else -1


def _stream_on(device, stream):
    """_stream for a device already known to be the current one."""
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(device)
    return _stream(stream)


def pa_rope_and_cache(q_out, q, key, value, key_cache, value_cache, cos_sin, positions,
                      slot_mapping, interleaved=False, swa_slot_mapping=None, k_scale=None,
                      v_scale=None, stream=None):
    """q_out <- q [N, H_Q, d] rotated by position; key [N, H, d] rotated and
    value [N, H, d] written to the caches [num_blocks, bs, H, d] (block stride
    free) at slot_mapping [N] int64.  cos_sin [max_positions, rot_dim] float32
    holds each position's cosines, then its sines; positions [N] int64; the
    first rot_dim elements of a head turn, as pairs (i, i + rot_dim / 2) or,
    interleaved, (2 i, 2 i + 1).  q, q_out, key and value share a dtype and have
    free token strides; q_out may be q.  Optional swa table int64,
    k_scale/v_scale one-element float32 device tensors."""
    device = _all_here(q, q_out, key, value, key_cache, value_cache, cos_sin, positions,
                       slot_mapping)
    if device < 0:
        _on_device(q_out=q_out, q=q, key=key, value=value, key_cache=key_cache,
                   value_cache=value_cache, cos_sin=cos_sin, positions=positions,
                   slot_mapping=slot_mapping)
    kind, shape, cache_shape = q.dtype, key.shape, key_cache.shape
    N, HQ, d = q_shape = q.shape
    H = shape[1]
    sq, s1, s2 = q.stride()
    so, s3, s4 = q_out.stride()
    sk, s5, s6 = key.stride()
    sv, s7, s8 = value.stride()
    if not (s2 == s4 == s6 == s8 == 1 and (s1 == s3 == d or HQ == 1) and (s5 == s7 == d or H == 1)):
        raise ValueError("q_out, q, key and value: heads and elements must be contiguous")
    if q_out.dtype != kind or key.dtype != kind or value.dtype != kind:
        raise ValueError("q_out, key and value must share q's dtype")
    if q_out.shape != q_shape or shape != (N, H, d) or value.shape != shape:
        raise ValueError("q_out must match q; key and value must be [N, H, d]")
    nb, bs, Hc, dc = cache_shape
    strides = key_cache.stride()
    sb, r1, r2, r3 = strides
    if Hc != H or dc != d or r3 != 1 or r2 != d or r1 != H * d:
        raise ValueError("key_cache must be [num_blocks, bs, H, d], contiguous inside a block")
    cache_kind = key_cache.dtype
    if value_cache.shape != cache_shape or value_cache.stride() != strides \
            or value_cache.dtype != cache_kind:
        raise ValueError("value_cache must match key_cache")
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be float32 [max_positions, rot_dim], contiguous")
    if positions.dtype != torch.int64 or positions.numel() != N or not positions.is_contiguous():
        raise ValueError("positions must be int64 [N]")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != N \
            or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be int64 [N]")
    swa = ks = vs = None
    swa_len = 0
    if swa_slot_mapping is not None:
        _on_device(swa_slot_mapping=swa_slot_mapping)
        if swa_slot_mapping.dtype != torch.int64 or not swa_slot_mapping.is_contiguous():
            raise ValueError("swa_slot_mapping must be int64, contiguous")
        swa, swa_len = swa_slot_mapping.data_ptr(), swa_slot_mapping.numel()
    if k_scale is not None or v_scale is not None:
        _scales(k_scale, v_scale)
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    most, rot = cos_sin.shape
    st = _load().pa_rope_and_cache(
        q_out.data_ptr(), q.data_ptr(), key.data_ptr(), value.data_ptr(), _dtype(q), N, HQ, H, d,
        so, sq, sk, sv, cos_sin.data_ptr(), positions.data_ptr(), most, _i32("rot_dim", rot),
        1 if interleaved else 0, key_cache.data_ptr(), value_cache.data_ptr(), _dtype(key_cache),
        nb, bs, sb, slot_mapping.data_ptr(), swa, swa_len, ks, vs, _stream_on(device, stream))
    if st != PA_OK:
        raise PAError(st, "pa_rope_and_cache")


def pa_paged_window_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_size, window,
                                          num_sink, max_context_len):
    window, num_sink = _i32("window", window), _i32("num_sink", num_sink)
    return int(_load().pa_paged_window_decode_workspace_size(
        num_seqs, num_q_heads, num_kv_heads, head_size, window, num_sink,
        _i32("max_context_len", max_context_len)))


def window_decode_workspace(num_seqs, num_q_heads, num_kv_heads, head_size, window, num_sink,
                            max_context_len, device=None):
    """A zeroed device workspace for pa_paged_window_decode_attention (allocated by torch)."""
    n = pa_paged_window_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_size,
                                              window, num_sink, max_context_len)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def _window_shapes(out, q, k_cache, v_cache, block_tables, context_lens, others):
    """Checks shared by the window attention calls: (device, B, H_Q, H_KV, d, block_size,
    num_blocks, max_blocks_per_seq)."""
    device = _all_here(q, out, k_cache, v_cache, block_tables, context_lens, *others)
    if device < 0:
        _on_device(out=out, q=q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
                   context_lens=context_lens)
    q_shape, shape, kind = q.shape, k_cache.shape, k_cache.dtype
    _, HQ, d = q_shape
    nb, bs, HKV, row = shape
    if not (q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous()
            and v_cache.is_contiguous() and block_tables.is_contiguous()
            and context_lens.is_contiguous()):
        raise ValueError("out, q, caches, block_tables and lengths must be contiguous")
    if q.dtype != torch.bfloat16 or out.dtype != torch.bfloat16 or out.shape != q_shape:
        raise ValueError("q and out must be bf16 and of one shape")
    if v_cache.dtype != kind or v_cache.shape != shape or row != d:
        raise ValueError("v_cache must match k_cache, rows of d elements")
    B = context_lens.numel()
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be [B, max_blocks_per_seq], context_lens [B]")
    return device, B, HQ, HKV, d, bs, nb, block_tables.shape[1]


def pa_paged_window_decode_attention(out, q, k_cache, v_cache, block_tables, context_lens, window,
                                     num_sink, scale, max_context_len, workspace, k_scale=None,
                                     v_scale=None, stream=None):
    """Decode attention (bf16 caches, or float8_e4m3fn with optional scales)
    over each sequence's last `window` tokens and its first num_sink; other
    arguments as for pa_paged_decode_attention, workspace from
    window_decode_workspace."""
    device, B, HQ, HKV, d, bs, nb, width = _window_shapes(out, q, k_cache, v_cache, block_tables,
                                                          context_lens, (workspace,))
    if device < 0 or not workspace.is_contiguous():
        _workspace(workspace)
    if q.shape[0] != B:
        raise ValueError("q must be [B, H_Q, d]")
    ks = vs = None
    if k_scale is not None or v_scale is not None:
        _scales(k_scale, v_scale)
        if k_cache.dtype != torch.float8_e4m3fn:
            raise ValueError("k_scale/v_scale apply to an e4m3 cache")
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    st = _load().pa_paged_window_decode_attention(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _dtype(k_cache), ks,
        vs, block_tables.data_ptr(), context_lens.data_ptr(), B, HQ, HKV, d, bs, width, nb,
        _i32("window", window), _i32("num_sink", num_sink), float(scale),
        _i32("max_context_len", max_context_len), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_on(device, stream))
    if st != PA_OK:
        raise PAError(st, "pa_paged_window_decode_attention")


def pa_paged_window_prefill_attention(out, q, k_cache, v_cache, block_tables, cu_seqlens_q,
                                      context_lens, window, num_sink, scale, max_q_len,
                                      error_word, stream=None):
    """Causal varlen prefill where the query at position p sees tokens
    t <= p with t > p - window or t < num_sink; out shares no memory with q;
    other arguments as for pa_paged_prefill_attention."""
    if error_word is None:
        raise ValueError("error_word is required")
    device, B, HQ, HKV, d, bs, nb, width = _window_shapes(
        out, q, k_cache, v_cache, block_tables, context_lens, (cu_seqlens_q, error_word))
    if device < 0:
        _on_device(cu_seqlens_q=cu_seqlens_q)
    if device < 0 or error_word.dtype != torch.int32 or error_word.numel() < 1:
        _word(error_word, "error_word")
    if cu_seqlens_q.dtype != torch.int32 or cu_seqlens_q.numel() != B + 1 \
            or not cu_seqlens_q.is_contiguous():
        raise ValueError("cu_seqlens_q must be int32 [B + 1]")
    st = _load().pa_paged_window_prefill_attention(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _dtype(k_cache),
        block_tables.data_ptr(), cu_seqlens_q.data_ptr(), context_lens.data_ptr(), B, HQ, HKV, d,
        bs, width, nb, _i32("window", window), _i32("num_sink", num_sink), float(scale),
        _i32("max_q_len", max_q_len), q.shape[0], error_word.data_ptr(),
        _stream_on(device, stream))
    if st != PA_OK:
        raise PAError(st, "pa_paged_window_prefill_attention")
