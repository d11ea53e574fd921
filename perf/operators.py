"""Cases of the long-context cache operators: the 4-bit cache (write, read back, decode attention),
decode attention that accumulates each cached token's weight, and eviction by that weight.

4-bit rows: a kv head's row of d elements is d/2 code bytes (element 2i in the low nibble of byte i) followed by
one (scale, minimum) pair of fp16 for each group of 32 elements; an element stands for minimum + scale * code.
"""
import math

import torch

own = False

GROUP = 32
HEAD = 128
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


def listed():
    return [
        # one decode step of a batch: each sequence's newest token, written and read back
        {"name": "write_step", "op": "write", "tokens": 64, "heads": 8, "block": 16, "src": "bf16", "out": "fp32",
         "swa": 0, "pad": 0},
        # a long prompt's cache write with padded positions, read back as bf16 for the attention of its next chunk
        {"name": "write_prompt", "op": "write", "tokens": 32768, "heads": 8, "block": 16, "src": "bf16", "out": "bf16",
         "swa": 0, "pad": 0},
        # an odd number of tokens and heads out of a wider fp32 projection (strided rows), through a sliding-window table
        {"name": "write_window", "op": "write", "tokens": 5001, "heads": 5, "block": 64, "src": "fp32", "out": "fp16",
         "swa": 4096, "pad": 64},
        # reading a cached prefix back as bf16 rows
        {"name": "read_prefix", "op": "read", "tokens": 65536, "heads": 8, "block": 16, "out": "bf16"},
        # the smallest decode batch: a few tokens a sequence, one of them empty
        {"name": "decode_tiny", "op": "decode", "cache": "q4", "seqs": 4, "lo": 0, "hi": 64, "kv_heads": 8, "group": 2,
         "block": 16, "holes": False},
        # an ordinary decode batch of ragged lengths
        {"name": "decode_batch", "op": "decode", "cache": "q4", "seqs": 64, "lo": 512, "hi": 4096, "kv_heads": 8,
         "group": 2, "block": 16, "holes": False},
        # few sequences of very long contexts: the context is split over the GPU
        {"name": "decode_long", "op": "decode", "cache": "q4", "seqs": 8, "lo": 32768, "hi": 131072, "kv_heads": 8,
         "group": 4, "block": 16, "holes": False},
        # the weight-accumulating decode step over an e4m3 cache, ragged batch with a missing block
        {"name": "scored_batch_e4m3", "op": "scored", "cache": "e4m3", "seqs": 64, "lo": 512, "hi": 4096, "kv_heads": 8,
         "group": 2, "block": 16, "holes": True, "new": 1},
        # the same over the 4-bit cache, one sequence, wide groups
        {"name": "scored_one_q4", "op": "scored", "cache": "q4", "seqs": 1, "lo": 9001, "hi": 9001, "kv_heads": 4,
         "group": 8, "block": 64, "holes": False, "new": 9001},
        # and over bf16 at long contexts
        {"name": "scored_long_bf16", "op": "scored", "cache": "bf16", "seqs": 8, "lo": 32768, "hi": 131072,
         "kv_heads": 8, "group": 4, "block": 16, "holes": False, "new": 1},
        # a batch over its budget by one chunk: select and move rows to new blocks
        {"name": "evict_batch", "op": "evict", "seqs": 16, "lo": 1800, "hi": 2304, "budget": 2048, "sink": 4,
         "recent": 256, "kv_heads": 8, "row": 128, "latent": False, "block": 16},
        # very long contexts cut down to a quarter
        {"name": "evict_long", "op": "evict", "seqs": 8, "lo": 32768, "hi": 131072, "budget": 16384, "sink": 16,
         "recent": 1024, "kv_heads": 8, "row": 128, "latent": False, "block": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "scored", "scored", "evict", "evict"])
    heads = rng.choice([1, 2, 3, 4, 5, 8])
    block = rng.choice([8, 16, 32, 64, 128, 256])
    if op == "write":
        return {"op": op, "tokens": _log(rng, 1, 32768), "heads": heads, "block": block,
                "src": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "out": rng.choice(["bf16", "fp16", "fp32"]),
                "swa": rng.choice([0, 0, 2048]), "pad": rng.choice([0, 8, 128])}
    if op == "read":
        return {"op": op, "tokens": _log(rng, 1, 65536), "heads": heads, "block": block,
                "out": rng.choice(["bf16", "fp16", "fp32"])}
    seqs = _log(rng, 1, 64)
    most = min(131072, 4_000_000 // (seqs * heads))
    hi = _log(rng, 1, most)
    lo = rng.choice([0, hi // 8, hi // 2, hi])
    if op in ("decode", "scored"):
        c = {"op": op, "cache": "q4" if op == "decode" else rng.choice(["q4", "bf16", "e4m3"]), "seqs": seqs, "lo": lo,
             "hi": hi, "kv_heads": heads, "group": rng.choice([1, 2, 4, 8, 16]), "block": block,
             "holes": rng.random() < 0.25}
        if op == "scored":
            c["new"] = rng.choice([0, 1, 1, 17, hi])
        return c
    budget = max(1, int(hi * rng.choice([0.1, 0.25, 0.5, 0.9, 1.1])))
    latent = rng.random() < 0.25
    return {"op": op, "seqs": seqs, "lo": lo, "hi": hi, "budget": budget, "sink": min(4, budget // 4),
            "recent": budget // rng.choice([2, 4, 8]), "kv_heads": 1 if latent else heads,
            "row": 576 if latent else 128, "latent": latent, "block": block}


# ---------------------------------------------------------------- inputs --
def _lens(case):
    """The batch's context lengths, spread evenly from lo to hi (their order comes from the seed)."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _table(lens, block, spare, gen):
    """Shuffled physical blocks for sequences of these lengths: block table (int32), number of blocks."""
    need = [(n + block - 1) // block for n in lens]
    width = max(1, max(need))
    total = sum(need) + spare
    perm = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    start = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda").unsqueeze(1)
    col = torch.arange(width, device="cuda").unsqueeze(0)
    table = perm[(start + col).clamp(max=total - 1)]
    inside = col < torch.tensor(need, device="cuda").unsqueeze(1)
    return torch.where(inside, table, torch.zeros_like(table)).contiguous(), total, perm[sum(need):]


def _q4_rows(x):
    """Rows of 4-bit groups (uint8) that stand for x [..., d]."""
    code, scale, low = _quantise(x)
    return _pack(code, scale, low)


def _q4_pool(blocks, block, heads, gen):
    x = torch.randn((blocks, block, heads, HEAD), generator=gen, device="cuda", dtype=torch.float16)
    return torch.cat([_q4_rows(part) for part in x.split(max(1, 100_000_000 // (block * heads * HEAD)))])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, block = case["op"], case["block"]
    st = dict(case=dict(case))
    if op in ("write", "read"):
        n, h = case["tokens"], case["heads"]
        slots = (n + block - 1) // block * block + block
        where = torch.randperm(slots, generator=gen, device="cuda")[:n]
        st["k_out"] = torch.zeros((n, h, HEAD), dtype=_TYPES[case["out"]], device="cuda")
        st["v_out"] = torch.zeros_like(st["k_out"])
        if op == "read":
            st["k_cache"] = _q4_pool(slots // block, block, h, gen)
            st["v_cache"] = _q4_pool(slots // block, block, h, gen)
            st["read_slots"] = where
            return st
        # key rows lie in a wider row, as in a fused projection's output
        wide = h * HEAD + case["pad"]
        for name in ("key", "value"):
            x = torch.randn((n, wide), generator=gen, device="cuda").to(_TYPES[case["src"]])
            st[name] = x[:, :h * HEAD].unflatten(1, (h, HEAD))
        if n > 1:
            where = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.05, torch.full_like(where, -1), where)
        st["slots"], st["swa"], st["read_slots"] = where, None, where
        if case["swa"]:
            # the last `swa` tokens keep a slot of the window's pool, older ones none
            swa = torch.full((slots,), -1, dtype=torch.int64, device="cuda")
            last = where[-case["swa"]:]
            last = last[last >= 0]
            swa[last] = torch.randperm(slots, generator=gen, device="cuda")[:last.numel()]
            st["swa"] = swa
            st["read_slots"] = torch.where(where >= 0, swa[where.clamp(min=0)], where)
        row = 5 * HEAD // 8
        st["k_cache"] = torch.zeros((slots // block, block, h, row), dtype=torch.uint8, device="cuda")
        st["v_cache"] = torch.zeros_like(st["k_cache"])
        return st
    lens = _lens(case)
    order = torch.randperm(len(lens), generator=gen, device="cuda").tolist()
    lens = [lens[i] for i in order]
    h = case["kv_heads"]
    kept = [min(n, case["budget"]) for n in lens] if op == "evict" else []
    spare = sum((n + block - 1) // block for n in kept) + 3
    table, blocks, rest = _table(lens, block, spare, gen)
    st["max_len"] = max(1, max(lens))
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["table"] = table
    if op == "evict":
        # weights as attention leaves them: few heavy tokens, many light ones, a fifth never looked at
        sums = torch.exp(2 * torch.randn((len(lens), h, st["max_len"]), generator=gen, device="cuda"))
        st["sums"] = torch.where(torch.rand(sums.shape, generator=gen, device="cuda") < 0.2,
                                 torch.zeros_like(sums), sums)
        st["sums_out"] = torch.zeros((len(lens), h, st["max_len"]), device="cuda")
        st["keep"] = torch.zeros((len(lens), h, case["budget"]), dtype=torch.int32, device="cuda")
        st["new_lens"] = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
        need = [(n + block - 1) // block for n in kept]
        width = max(1, max(need))
        dst = torch.zeros((len(lens), width), dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            dst[i, :n] = rest[at:at + n]
            at += n
        st["new_table"] = dst
        shape = (blocks, block, h, case["row"])
        st["k_cache"] = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        st["v_cache"] = None if case["latent"] else torch.randn(shape, generator=gen, device="cuda",
                                                                dtype=torch.bfloat16)
        return st
    hq = h * case["group"]
    st["scale"] = 1 / math.sqrt(HEAD)
    st["q"] = torch.randn((len(lens), hq, HEAD), generator=gen, device="cuda").to(torch.bfloat16)
    st["out"] = torch.zeros_like(st["q"])
    if case["holes"]:
        # one block in 16 is gone from the pool (its tokens drop out)
        gone = torch.rand(table.shape, generator=gen, device="cuda") < 1 / 16
        st["table"] = torch.where(gone, torch.full_like(table, -1), table)
    st["k_scale"] = st["v_scale"] = None
    if case["cache"] == "q4":
        st["k_cache"] = _q4_pool(blocks, block, h, gen)
        st["v_cache"] = _q4_pool(blocks, block, h, gen)
    else:
        shape = (blocks, block, h, HEAD)
        k = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        v = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        if case["cache"] == "e4m3":
            st["k_scale"] = torch.tensor([0.05], device="cuda")
            st["v_scale"] = torch.tensor([0.05], device="cuda")
            k, v = (k / st["k_scale"]).to(torch.float8_e4m3fn), (v / st["v_scale"]).to(torch.float8_e4m3fn)
        st["k_cache"], st["v_cache"] = k, v
    if op == "scored":
        st["sums"] = torch.exp(2 * torch.randn((len(lens), h, st["max_len"]), generator=gen, device="cuda"))
        st["sums_out"] = torch.zeros_like(st["sums"])
    return st


# ------------------------------------------------------------ plain forms --
def _quantise(x):
    """Codes, scale and minimum of each group of 32 (the last dimension split in groups), in 32 bits."""
    x = x.float().unflatten(-1, (-1, GROUP))
    fine = torch.isfinite(x).all(-1, keepdim=True)
    x = torch.where(fine, x, torch.zeros_like(x))
    low = x.amin(-1, keepdim=True).clamp(-65504, 65504).half().float()
    span = x.amax(-1, keepdim=True) - low
    scale = (span / torch.full_like(span, 15.0)).clamp(0, 1023).half().float()
    code = torch.round((x - low) / torch.where(scale > 0, scale, torch.ones_like(scale))).clamp(0, 15)
    code = torch.where(scale > 0, code, torch.zeros_like(code)).to(torch.uint8)
    nan = torch.full_like(low, float("nan"))
    return code, torch.where(fine, scale, nan).half(), torch.where(fine, low, nan).half()


def _pack(code, scale, low):
    code = code.flatten(-2)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    meta = torch.cat([scale, low], -1).contiguous().view(torch.uint8).flatten(-2)
    return torch.cat([packed, meta], -1)


def _unpack(rows):
    """The values that rows of 4-bit groups stand for, in 32 bits."""
    d = rows.shape[-1] * 8 // 5
    packed, meta = rows[..., :d // 2], rows[..., d // 2:].contiguous()
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).unflatten(-1, (-1, GROUP)).float()
    meta = meta.view(torch.float16).float().unflatten(-1, (-1, 2))
    return (code * meta[..., 0:1] + meta[..., 1:2]).flatten(-2)


def _cached(pool, scale, table, rows, inside):
    """A cache's values [B, T, H, d] in 32 bits at these logical rows; zeros where there is no token."""
    block = pool.shape[1]
    ids = torch.gather(table, 1, rows // block)
    there = inside & (ids >= 0) & (ids < pool.shape[0])
    at = torch.where(there, ids.long() * block + rows % block, torch.zeros_like(rows))
    x = pool.flatten(0, 1)[at]
    x = _unpack(x) if pool.dtype == torch.uint8 else x.float()
    if scale is not None:
        x = x * scale
    return torch.where(there[..., None, None], x, torch.zeros_like(x)), there


def _attend(st):
    """Attention outputs in 32 bits and the weights [B, H_KV, G, T]."""
    q, lens = st["q"], st["lens"].long()
    rows = torch.arange(st["max_len"], device="cuda").expand(len(lens), -1)
    inside = rows < lens[:, None]
    k, there = _cached(st["k_cache"], st["k_scale"], st["table"], rows, inside)
    heads = k.shape[2]
    qs = q.float().unflatten(1, (heads, -1))
    score = torch.matmul(qs, k.permute(0, 2, 3, 1)) * st["scale"]
    del k
    score = torch.where(there[:, None, None], score, torch.full_like(score, float("-inf")))
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    del score
    total = weight.sum(-1, keepdim=True)
    weight = weight / torch.where(total > 0, total, torch.ones_like(total))
    v, _ = _cached(st["v_cache"], st["v_scale"], st["table"], rows, inside)
    out = torch.matmul(weight, v.permute(0, 2, 1, 3)).flatten(1, 2)
    return out, weight, rows, inside


def _select(st):
    """The kept tokens of each row, ascending (-1 behind them), their number and their sums."""
    case, sums, lens = st["case"], st["sums"], st["lens"].long()
    t = torch.arange(sums.shape[2], device="cuda").expand_as(sums)
    n = lens[:, None, None]
    first = (t < case["sink"]) | (t >= n - case["recent"])
    worth = torch.where(first, torch.full_like(sums, float("inf")), sums)
    worth = torch.where(t < n, worth, torch.full_like(sums, float("-inf")))
    order = torch.sort(worth, dim=-1, descending=True, stable=True).indices
    new_lens = lens.clamp(max=case["budget"])
    best = order[..., :case["budget"]]
    rank = torch.arange(best.shape[-1], device="cuda").expand_as(best)
    live = rank < new_lens[:, None, None]
    best = torch.where(live, best, torch.full_like(best, sums.shape[2])).sort(-1).values
    keep = torch.full_like(st["keep"], -1)
    keep[..., :best.shape[-1]] = torch.where(live, best, torch.full_like(best, -1)).int()
    compact = torch.gather(sums, 2, best.clamp(max=sums.shape[2] - 1))
    sums_out = torch.zeros_like(sums)
    sums_out[..., :best.shape[-1]] = torch.where(live, compact, torch.zeros_like(compact))
    return keep, new_lens.int(), sums_out


def _move(st, pool, keep):
    """Kept rows copied to the new blocks of the pool."""
    block = pool.shape[1]
    seq, head, j = torch.nonzero(keep >= 0, as_tuple=True)
    old = keep[seq, head, j].long()
    src = st["table"][seq, old // block].long() * block + old % block
    dst = st["new_table"][seq, j // block].long() * block + j % block
    flat = pool.flatten(0, 1)
    flat[dst, head] = flat[src, head]
    return pool


# -------------------------------------------------------------------- run --
def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        from paged_kv_cache_309_gb300 import pa
    if op in ("write", "read"):
        if own:
            if op == "write":
                pa.pa_reshape_and_cache_q4(st["key"], st["value"], st["k_cache"], st["v_cache"], st["slots"],
                                           st["swa"])
            pa.pa_gather_cache_q4(st["k_out"], st["v_out"], st["k_cache"], st["v_cache"], st["read_slots"])
            return {"key": st["k_out"], "value": st["v_out"]}
        kc, vc = st["k_cache"].flatten(0, 1), st["v_cache"].flatten(0, 1)
        to = st["read_slots"]
        there = to >= 0
        if op == "write":
            kc[to[there]] = _q4_rows(st["key"][there])
            vc[to[there]] = _q4_rows(st["value"][there])
        at = to.clamp(min=0)
        k, v = _unpack(kc[at]), _unpack(vc[at])
        return {"key": torch.where(there[:, None, None], k, torch.zeros_like(k)).to(st["k_out"].dtype),
                "value": torch.where(there[:, None, None], v, torch.zeros_like(v)).to(st["v_out"].dtype)}
    if op == "evict":
        if own:
            pa.pa_evict_select(st["keep"], st["new_lens"], st["sums_out"], st["sums"], st["lens"], case["budget"],
                               case["sink"], case["recent"])
            pa.pa_cache_compact(st["k_cache"], st["v_cache"], st["keep"], st["new_lens"], st["table"],
                                st["new_table"])
            keep, new_lens, sums = st["keep"], st["new_lens"], st["sums_out"]
            k, v = st["k_cache"], st["v_cache"]
        else:
            keep, new_lens, sums = _select(st)
            k = _move(st, st["k_cache"], keep)
            v = None if st["v_cache"] is None else _move(st, st["v_cache"], keep)
        got = {"keep": keep, "new_lens": new_lens, "sums": sums, "k_cache": k}
        return got if v is None else {**got, "v_cache": v}
    if own:
        b, hq, d = st["q"].shape
        if "workspace" not in st:  # a user's program keeps it beside its tables
            make = pa.decode_scored_workspace if op == "scored" else pa.decode_workspace
            st["workspace"] = make(b, hq, case["kv_heads"], d, st["max_len"])
        if op == "scored":
            pa.pa_paged_decode_attention_scored(
                st["out"], st["sums_out"], st["sums"], case["new"], st["q"], st["k_cache"], st["v_cache"],
                st["table"], st["lens"], st["scale"], st["max_len"], st["workspace"], k_scale=st["k_scale"],
                v_scale=st["v_scale"])
            return {"out": st["out"], "sums": st["sums_out"]}
        pa.pa_paged_decode_attention_q4(st["out"], st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                                        st["scale"], st["max_len"], st["workspace"])
        return {"out": st["out"]}
    out, weight, rows, inside = _attend(st)
    out = out.to(torch.bfloat16)
    if op == "decode":
        return {"out": out}
    # a token that came with the last `new` ones has no sum yet
    fresh = rows >= st["lens"].long()[:, None] - case["new"]
    sums = torch.where(fresh[:, None], torch.zeros_like(st["sums"]), st["sums"]) + weight.sum(2)
    return {"out": out, "sums": torch.where(inside[:, None], sums, torch.zeros_like(sums))}


# ------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    row = 5 * HEAD // 8
    if op in ("write", "read"):
        n, h = case["tokens"], case["heads"]
        there = n
        if op == "write":
            live = n * 0.95 if n > 1 else n
            there = min(live, case["swa"] * 0.95) if case["swa"] else live
        read_back = there * h * (row + HEAD * _BYTES[case["out"]]) * 2 + 8 * n
        if op == "read":
            return {"bytes": int(read_back), "flops": int(2 * there * h * HEAD * 2)}
        write = there * h * (HEAD * _BYTES[case["src"]] + row) * 2 + 8 * n
        return {"bytes": int(write + read_back), "flops": int(there * h * HEAD * 2 * 8)}
    lens = _lens(case)
    total, h = sum(lens), case["kv_heads"]
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        pools = 1 if case["latent"] else 2
        return {"bytes": total * h * 4 + len(lens) * h * case["budget"] * 4 + kept * h * 4
                + kept * h * case["row"] * 2 * 2 * pools, "flops": total * h}
    hq = h * case["group"]
    tokens = row if case["cache"] == "q4" else HEAD * _BYTES[case["cache"]]
    size = total * h * tokens * 2 + len(lens) * hq * HEAD * 4 + total // case["block"] * 4
    flops = 4 * hq * HEAD * total
    if op == "scored":
        old = sum(max(0, n - case["new"]) for n in lens)
        size += (total + old) * h * 4
        flops += hq * total
    return {"bytes": size, "flops": flops}


# ------------------------------------------------------------------ exact --
def _exact_groups(x):
    """Quantised and restored in 64 bits, from the definition; x [n, h, d] finite."""
    g = x.double().reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    low = g.min(-1).values.clamp(-65504, 65504).to(torch.float16).double()
    step = ((g.max(-1).values - low) / 15).clamp(0, 1023).to(torch.float16).double()
    code = ((g - low[..., None]) / step[..., None]).round().clamp(0, 15)
    code = torch.where(step[..., None] > 0, code, torch.zeros_like(code))
    return (low[..., None] + step[..., None] * code).reshape(x.shape)


def _exact_rows(raw):
    """Packed rows restored in 64 bits."""
    d = raw.shape[-1] * 8 // 5
    pairs = raw[..., d // 2:].contiguous().view(torch.float16).double()
    step, low = pairs[..., 0::2], pairs[..., 1::2]
    value = torch.empty(*raw.shape[:-1], d, dtype=torch.float64, device=raw.device)
    value[..., 0::2] = (raw[..., :d // 2] % 16).double()
    value[..., 1::2] = (raw[..., :d // 2] // 16).double()
    return value * step.repeat_interleave(GROUP, -1) + low.repeat_interleave(GROUP, -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("write", "read"):
        live = st["read_slots"] >= 0
        found = {}
        for name, cache in (("key", "k_cache"), ("value", "v_cache")):
            x = torch.zeros(st["k_out"].shape, dtype=torch.float64, device="cuda")
            if op == "write":
                x[live] = _exact_groups(st[name][live])
            else:
                x = _exact_rows(st[cache].reshape(-1, *st[cache].shape[2:])[st["read_slots"]])
            found[name] = x
        return found
    lens = st["lens"].tolist()
    if op == "evict":
        import numpy as np
        sums = st["sums"].double().cpu().numpy()
        got = np.zeros(sums.shape)
        for b, n in enumerate(lens):
            for h in range(sums.shape[1]):
                at = np.arange(n)
                free = (at >= case["sink"]) & (at < n - case["recent"])
                order = np.lexsort((at, -sums[b, h, :n], free))
                kept = np.sort(order[:case["budget"]])
                got[b, h, :len(kept)] = sums[b, h, kept]
        made = {"keep": None, "new_lens": None, "sums": torch.from_numpy(got).cuda(), "k_cache": None}
        return made if st["v_cache"] is None else {**made, "v_cache": None}
    block, heads = case["block"], case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    sums = torch.zeros(len(lens), heads, st["max_len"], dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        at = torch.arange(n, device="cuda")
        blk = st["table"][b].long()[at // block]
        live = blk >= 0
        if op == "scored":
            old = n - case["new"]
            if old > 0:
                sums[b, :, :old] = st["sums"][b, :, :old].double()
        if not bool(live.any()):
            continue
        slot = blk[live] * block + at[live] % block
        for h in range(heads):
            k, v = (st[c].reshape(-1, heads, st[c].shape[-1])[slot, h] for c in ("k_cache", "v_cache"))
            if case["cache"] == "q4":
                k, v = _exact_rows(k), _exact_rows(v)
            else:
                k, v = k.double(), v.double()
            if st["k_scale"] is not None:
                k, v = k * st["k_scale"].double(), v * st["v_scale"].double()
            qs = st["q"][b, h * case["group"]:(h + 1) * case["group"]].double()
            p = torch.softmax(qs @ k.T * st["scale"], -1)
            out[b, h * case["group"]:(h + 1) * case["group"]] = p @ v
            if op == "scored":
                sums[b, h, at[live]] += p.sum(0)
    return {"out": out, "sums": sums} if op == "scored" else {"out": out}
