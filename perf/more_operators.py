"""Cases of the sliding-window path: queries and keys rotated by position with the keys and values appended to the paged
cache, and attention over that cache with a sliding window and a few first tokens that stay visible, for single
tokens and for prompts.

A query at position p of its sequence sees token t where t <= p and (t > p - window or t < sink).
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


def listed():
    return [
        # one decode step of a batch: each sequence's newest token
        {"name": "append_step", "op": "append", "tokens": 64, "q_heads": 16, "kv_heads": 8, "head": 128, "rot": 128,
         "pairs": False, "block": 16, "src": "bf16", "cache": "bf16", "scaled": False, "swa": 0},
        # a long prompt out of a fused projection (strided rows), with padded positions
        {"name": "append_prompt", "op": "append", "tokens": 32768, "q_heads": 32, "kv_heads": 8, "head": 128,
         "rot": 128, "pairs": False, "block": 16, "src": "bf16", "cache": "bf16", "scaled": False, "swa": 0},
        # an e4m3 cache behind a sliding-window slot table: odd numbers, neighbouring pairs, a part of the head rotated
        {"name": "append_window_e4m3", "op": "append", "tokens": 5001, "q_heads": 10, "kv_heads": 5, "head": 96,
         "rot": 32, "pairs": True, "block": 64, "src": "fp16", "cache": "e4m3", "scaled": True, "swa": 4096},
        # a prompt's chunk in fp32 with wide heads
        {"name": "append_fp32", "op": "append", "tokens": 2047, "q_heads": 7, "kv_heads": 1, "head": 256, "rot": 256,
         "pairs": False, "block": 32, "src": "fp32", "cache": "bf16", "scaled": False, "swa": 0},
        # the smallest decode batch: a few tokens a sequence, one of them empty
        {"name": "decode_tiny", "op": "decode", "cache": "bf16", "seqs": 4, "lo": 0, "hi": 64, "q_heads": 16,
         "kv_heads": 8, "block": 16, "window": 32, "sink": 4, "holes": False},
        # an ordinary decode batch of ragged lengths
        {"name": "decode_batch", "op": "decode", "cache": "bf16", "seqs": 64, "lo": 512, "hi": 4096, "q_heads": 16,
         "kv_heads": 8, "block": 16, "window": 1024, "sink": 4, "holes": False},
        # few sequences of very long contexts under a wide window
        {"name": "decode_long", "op": "decode", "cache": "bf16", "seqs": 8, "lo": 32768, "hi": 131072, "q_heads": 32,
         "kv_heads": 8, "block": 16, "window": 16384, "sink": 64, "holes": False},
        # an e4m3 cache with scales, wide groups, a window that starts inside a block, missing blocks
        {"name": "decode_batch_e4m3", "op": "decode", "cache": "e4m3", "seqs": 64, "lo": 512, "hi": 8192,
         "q_heads": 32, "kv_heads": 4, "block": 64, "window": 2000, "sink": 5, "holes": True},
        # a few short questions, one of a single token, some behind a cached prefix
        {"name": "prefill_tiny", "op": "prefill", "seqs": 3, "new_lo": 1, "new_hi": 40, "before": 300, "q_heads": 16,
         "kv_heads": 8, "block": 16, "window": 128, "sink": 4, "holes": False},
        # chunked prefill: the next 512 tokens of long prompts
        {"name": "prefill_chunk", "op": "prefill", "seqs": 8, "new_lo": 512, "new_hi": 512, "before": 6000,
         "q_heads": 16, "kv_heads": 8, "block": 16, "window": 1024, "sink": 4, "holes": False},
        # fresh prompts of 8192 tokens
        {"name": "prefill_prompts", "op": "prefill", "seqs": 4, "new_lo": 8192, "new_hi": 8192, "before": 0,
         "q_heads": 32, "kv_heads": 8, "block": 16, "window": 4096, "sink": 4, "holes": False},
        # ragged prompts under a narrow window without first tokens, many heads to a kv head
        {"name": "prefill_narrow", "op": "prefill", "seqs": 5, "new_lo": 1000, "new_hi": 6001, "before": 0,
         "q_heads": 16, "kv_heads": 2, "block": 64, "window": 250, "sink": 0, "holes": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill"])
    block = rng.choice([8, 16, 32, 64, 128, 256])
    if op == "append":
        head = rng.choice([32, 64, 96, 128, 128, 192, 256])
        heads = rng.choice([1, 2, 3, 4, 5, 8])
        cache = rng.choice(["bf16", "bf16", "fp16", "fp32", "e4m3"])
        group = rng.choice([1, 2, 4, 7, 8])
        return {"op": op, "tokens": _log(rng, 1, min(32768, 32768 * 48 * 64 // (head * heads * (group + 2)))),
                "q_heads": heads * group, "kv_heads": heads, "head": head,
                "rot": rng.choice([head, head, head // 2, 32, 16]), "pairs": rng.random() < 0.4, "block": block,
                "src": rng.choice(["bf16", "bf16", "fp16"]), "cache": cache,
                "scaled": cache == "e4m3" or rng.random() < 0.15, "swa": rng.choice([0, 0, 0, 2048])}
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 8, 16])
    case = {"op": op, "q_heads": kv_heads * group, "kv_heads": kv_heads, "block": block,
            "window": _log(rng, 1, 16384), "sink": rng.choice([0, 0, 1, 4, 4, 16, 64, 130]),
            "holes": rng.random() < 0.2}
    if op == "decode":
        seqs = _log(rng, 1, 64)
        hi = _log(rng, 1, min(131072, 4_000_000 // (seqs * kv_heads)))
        return {**case, "cache": rng.choice(["bf16", "bf16", "e4m3"]), "seqs": seqs,
                "lo": rng.choice([0, hi // 8, hi // 2, hi]), "hi": hi}
    seqs = _log(rng, 1, 16)
    new_hi = _log(rng, 1, max(1, min(8192, 131072 // case["q_heads"]) // seqs))
    return {**case, "seqs": seqs, "new_hi": new_hi, "new_lo": rng.choice([1, max(1, new_hi // 2), new_hi]),
            "before": rng.choice([0, 0, 17, 1000, 5000])}


# ---------------------------------------------------------------- inputs --
def _spread(n, lo, hi):
    """n lengths spread evenly from lo to hi."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _table(lens, block, gen):
    """Shuffled physical blocks for sequences of these lengths: block table (int32), number of blocks."""
    need = [(n + block - 1) // block for n in lens]
    total = sum(need) + 3
    perm = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    start = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda").unsqueeze(1)
    col = torch.arange(max(1, max(need)), device="cuda").unsqueeze(0)
    table = perm[(start + col).clamp(max=total - 1)]
    inside = col < torch.tensor(need, device="cuda").unsqueeze(1)
    return torch.where(inside, table, torch.zeros_like(table)).contiguous(), total


def _lens(case):
    """New tokens and context lengths (the new ones included) of the sequences."""
    n = case["seqs"]
    if case["op"] == "decode":
        return [1] * n, _spread(n, case["lo"], case["hi"])
    new = _spread(n, case["new_lo"], case["new_hi"])
    return new, [a + b for a, b in zip(new, _spread(n, 0, case["before"]))]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=dict(case))

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    if case["op"] == "append":
        n, hq, h, d, rot = (case[k] for k in ("tokens", "q_heads", "kv_heads", "head", "rot"))
        # queries, keys and values lie side by side in the output of a fused projection
        wide = normal(n, (hq + 2 * h) * d, dtype=_TYPES[case["src"]])
        st["q"] = wide[:, :hq * d].unflatten(1, (hq, d))
        st["key"] = wide[:, hq * d:(hq + h) * d].unflatten(1, (h, d))
        st["value"] = wide[:, (hq + h) * d:].unflatten(1, (h, d))
        st["q_out"] = torch.zeros((n, hq, d), dtype=wide.dtype, device="cuda")
        # cosines, then sines, of every position's angles
        most = 131072
        angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -2.0 * torch.arange(rot // 2, device="cuda", dtype=torch.float64) / rot)
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        if n > 512:  # a prompt (its chunk behind others), else a batch of sequences' newest tokens
            first = int(torch.randint(0, most - n, (1,), generator=gen, device="cuda"))
            st["positions"] = torch.arange(first, first + n, device="cuda")
        else:
            st["positions"] = torch.randint(0, most, (n,), generator=gen, device="cuda")
        slots = (n + case["block"] - 1) // case["block"] * case["block"] + case["block"]
        where = torch.randperm(slots, generator=gen, device="cuda")[:n]
        if n > 64:
            where = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.05, torch.full_like(where, -1), where)
        st["slots"], st["swa"] = where, None
        if case["swa"]:
            # the last `swa` tokens keep a slot of the window's pool, older ones none
            st["swa"] = torch.full((slots,), -1, dtype=torch.int64, device="cuda")
            last = where[-case["swa"]:]
            last = last[last >= 0]
            st["swa"][last] = torch.randperm(slots, generator=gen, device="cuda")[:last.numel()]
        shape = (slots // case["block"], case["block"], h, d)
        st["k_cache"] = normal(*shape, dtype=_TYPES[case["cache"]])
        st["v_cache"] = normal(*shape, dtype=_TYPES[case["cache"]])
        st["k_scale"] = torch.tensor([0.05], device="cuda") if case["scaled"] else None
        st["v_scale"] = torch.tensor([0.03], device="cuda") if case["scaled"] else None
        return st
    new, lens = _lens(case)
    order = torch.randperm(len(lens), generator=gen, device="cuda").tolist()
    new, lens = [new[i] for i in order], [lens[i] for i in order]
    hq, h, block = case["q_heads"], case["kv_heads"], case["block"]
    st["table"], blocks = _table(lens, block, gen)
    if case["holes"]:
        # one block in 16 is gone from the pool (its tokens drop out)
        gone = torch.rand(st["table"].shape, generator=gen, device="cuda") < 1 / 16
        st["table"] = torch.where(gone, torch.full_like(st["table"], -1), st["table"])
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["max_len"], st["max_new"] = max(1, max(lens)), max(new)
    st["scale"] = 1 / math.sqrt(128)
    st["q"] = normal(sum(new), hq, 128)
    st["out"] = torch.zeros_like(st["q"])
    st["k_scale"] = st["v_scale"] = None
    for name in ("k_cache", "v_cache"):
        x = torch.randn((blocks, block, h, 128), generator=gen, device="cuda", dtype=torch.bfloat16)
        if case.get("cache") == "e4m3":
            st[name[0] + "_scale"] = torch.tensor([0.05], device="cuda")
            x = (x / st[name[0] + "_scale"]).to(torch.float8_e4m3fn)
        st[name] = x
    if case["op"] == "prefill":
        st["starts"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        st["error"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------ plain forms --
def _rotated(x, cos, sin, rot, pairs):
    """The first rot elements of each head rotated by the token's angles, the rest as they are; in 32 bits."""
    x = x.float()
    turned = x[..., :rot]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if pairs else (turned[..., :rot // 2], turned[..., rot // 2:])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], -1).flatten(-2) if pairs else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _stored(x, scale, dtype):
    if scale is not None:
        x = x / scale
    if dtype == torch.float8_e4m3fn:
        x = x.clamp(-448, 448)
    return x.to(dtype)


def _cached(pool, scale, table, rows, inside):
    """A cache's values [B, H, T, d] in 32 bits at these logical rows [B, T]; zeros where there is no token."""
    block = pool.shape[1]
    ids = torch.gather(table, 1, (rows // block).clamp(max=table.shape[1] - 1))
    there = inside & (ids >= 0)
    at = torch.where(there, ids.long() * block + rows % block, torch.zeros_like(rows))
    x = pool.flatten(0, 1)[at].float()
    if scale is not None:
        x = x * scale
    return torch.where(there[..., None, None], x, torch.zeros_like(x)).transpose(1, 2), there


def _softmax(score, seen):
    """Weights of the seen scores in their place; a row that sees nothing has none."""
    score.masked_fill_(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    total = score.sum(-1, keepdim=True)
    return score.div_(torch.where(total > 0, total, torch.ones_like(total)))


def _decode(st):
    """One query a sequence over the rows that it sees: the first ones, then the window."""
    case, lens = st["case"], st["lens"].long()[:, None]
    sink = min(case["sink"], st["max_len"])
    wide = min(case["window"], st["max_len"])
    first = torch.arange(sink, device="cuda").expand(len(lens), -1)
    low = (lens - case["window"]).clamp(min=0)
    last = low + torch.arange(wide, device="cuda")
    rows = torch.cat([first, last], 1)
    inside = torch.cat([(first < lens) & (first < low), last < lens], 1)
    k, there = _cached(st["k_cache"], st["k_scale"], st["table"], rows, inside)
    q = st["q"].float().unflatten(1, (k.shape[1], -1))
    weight = _softmax(torch.matmul(q, k.transpose(2, 3)) * st["scale"], there[:, None, None])
    v, _ = _cached(st["v_cache"], st["v_scale"], st["table"], rows, inside)
    return torch.matmul(weight, v).flatten(1, 2).to(st["out"].dtype)


def _prefill(st):
    """The new tokens of every sequence, padded to one length, over the padded rows of its context."""
    case, lens, starts = st["case"], st["lens"].long()[:, None], st["starts"].long()
    new = (starts[1:] - starts[:-1])[:, None]
    rows = torch.arange(st["max_len"], device="cuda").expand(len(lens), -1)
    k, there = _cached(st["k_cache"], st["k_scale"], st["table"], rows, rows < lens)
    j = torch.arange(st["max_new"], device="cuda")[None]
    real = j < new
    at = torch.where(real, starts[:-1, None] + j, torch.zeros_like(j))
    pos = (lens - new + j)[:, :, None]
    t = rows[:, None, :]
    seen = there[:, None, :] & (t <= pos) & ((t > pos - case["window"]) | (t < case["sink"]))
    heads = k.shape[1]
    q = st["q"][at].float().unflatten(2, (heads, -1)).permute(0, 2, 3, 1, 4)
    score = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).mul_(st["scale"])
    weight = _softmax(score.unflatten(2, q.shape[2:4]), seen[:, None, None])
    v, _ = _cached(st["v_cache"], st["v_scale"], st["table"], rows, rows < lens)
    out = torch.matmul(weight.flatten(2, 3), v).unflatten(2, q.shape[2:4])
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3)[real].to(st["out"].dtype)


# -------------------------------------------------------------------- run --
def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        from paged_kv_cache_309_gb300 import pa
    if op == "append":
        if own:
            pa.pa_rope_and_cache(st["q_out"], st["q"], st["key"], st["value"], st["k_cache"], st["v_cache"],
                                 st["cos_sin"], st["positions"], st["slots"], interleaved=case["pairs"],
                                 swa_slot_mapping=st["swa"], k_scale=st["k_scale"], v_scale=st["v_scale"])
            return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
        at = st["cos_sin"][st["positions"]][:, None]
        cos, sin = at[..., :case["rot"] // 2], at[..., case["rot"] // 2:]
        to = st["slots"]
        if st["swa"] is not None:
            to = torch.where(to >= 0, st["swa"][to.clamp(min=0)], to)
        live = to >= 0
        key = _rotated(st["key"], cos, sin, case["rot"], case["pairs"])
        st["k_cache"].flatten(0, 1)[to[live]] = _stored(key, st["k_scale"], st["k_cache"].dtype)[live]
        st["v_cache"].flatten(0, 1)[to[live]] = _stored(st["value"].float(), st["v_scale"], st["v_cache"].dtype)[live]
        return {"q": _rotated(st["q"], cos, sin, case["rot"], case["pairs"]).to(st["q"].dtype),
                "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    if not own:
        return {"out": _decode(st) if op == "decode" else _prefill(st)}
    if op == "decode":
        if "workspace" not in st:  # a user's program keeps it beside its tables
            st["workspace"] = pa.window_decode_workspace(case["seqs"], case["q_heads"], case["kv_heads"], 128,
                                                         case["window"], case["sink"], st["max_len"])
        pa.pa_paged_window_decode_attention(st["out"], st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                                            case["window"], case["sink"], st["scale"], st["max_len"],
                                            st["workspace"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    else:
        pa.pa_paged_window_prefill_attention(st["out"], st["q"], st["k_cache"], st["v_cache"], st["table"],
                                             st["starts"], st["lens"], case["window"], case["sink"], st["scale"],
                                             st["max_new"], st["error"])
    return {"out": st["out"]}


# ------------------------------------------------------------------- work --
def _below(p, case):
    """How many tokens a query at position p sees."""
    w, s = case["window"], case["sink"]
    return p + 1 if p < w else w + min(s, p + 1 - w)


def work(case):
    if case["op"] == "append":
        n, hq, h, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head"]
        live = n * 0.95 if n > 64 else n
        if case["swa"]:
            live = min(live, case["swa"] * 0.95)
        size = n * hq * d * 2 * _BYTES[case["src"]] + n * (case["rot"] * 4 + 16)
        size += live * 2 * h * d * (_BYTES[case["src"]] + _BYTES[case["cache"]])
        return {"bytes": int(size), "flops": int((n * hq + live * h) * case["rot"] * 3)}
    new, lens = _lens(case)
    row = 2 * case["kv_heads"] * 128 * _BYTES[case.get("cache", "bf16")]
    size, pairs = sum(new) * case["q_heads"] * 128 * 4, 0
    for n, length in zip(new, lens):
        if length == 0:
            continue
        first = length - n
        pairs += sum(_below(p, case) for p in range(first, length))
        read = min(length, n - 1 + case["window"])
        size += (read + min(case["sink"], length - read)) * row
    return {"bytes": int(size), "flops": int(4 * pairs * case["q_heads"] * 128)}


# ------------------------------------------------------------------ exact --
def _turn(x, positions, table, pairs):
    """Rotation as a complex product, in 64 bits."""
    rot = table.shape[1]
    angle = table.double()[positions]
    factor = torch.complex(angle[:, :rot // 2], angle[:, rot // 2:])[:, None, :]
    y = x.double().clone()
    if pairs:
        y[..., :rot] = torch.view_as_real(torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous())
                                          * factor).flatten(-2)
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * factor
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        got = {"q": _turn(st["q"], st["positions"], st["cos_sin"], case["pairs"])}
        slot = st["slots"].clone()
        if st["swa"] is not None:
            slot[slot >= 0] = st["swa"][slot[slot >= 0]]
        keep = torch.nonzero(slot >= 0).flatten()
        for name, src in (("k", _turn(st["key"], st["positions"], st["cos_sin"], case["pairs"])),
                          ("v", st["value"].double())):
            if st[name + "_scale"] is not None:
                src = src / st[name + "_scale"].double()
            if case["cache"] == "e4m3":
                src = src.clamp(-448, 448)
            cache = st[name + "_cache"].double()
            cache.view(-1, *cache.shape[2:]).index_copy_(0, slot[keep], src[keep])
            got[name + "_cache"] = cache
        return got
    lens, block = st["lens"].tolist(), case["block"]
    starts = st["starts"].tolist() if case["op"] == "prefill" else list(range(len(lens) + 1))
    group = case["q_heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(lens):
        if length == 0:
            continue
        new = starts[b + 1] - starts[b]
        t = torch.arange(length, device="cuda")
        blk = st["table"][b].long()[t // block]
        slot = blk.clamp(min=0) * block + t % block
        for i in range(0, new, 1024):
            m = min(1024, new - i)
            p = length - new + i + torch.arange(m, device="cuda")
            low = max(0, int(length - new + i) - case["window"] + 1)
            pick = (t <= length - new + i + m - 1) & ((t >= low) | (t < case["sink"]))
            tok = t[pick]
            hide = (tok[None] > p[:, None]) | ((tok[None] <= p[:, None] - case["window"])
                                               & (tok[None] >= case["sink"])) | (blk[pick] < 0)[None]
            none = hide.all(1)
            for h in range(case["kv_heads"]):
                k, v = (st[c].reshape(-1, case["kv_heads"], 128)[slot[pick], h].double()
                        for c in ("k_cache", "v_cache"))
                if st["k_scale"] is not None:
                    k, v = k * st["k_scale"].double(), v * st["v_scale"].double()
                rows = slice(starts[b] + i, starts[b] + i + m)
                q = st["q"][rows, h * group:(h + 1) * group].double()
                s = torch.einsum("mgd,td->gmt", q, k) * st["scale"]
                w = torch.softmax(s.masked_fill(hide[None], float("-inf")), -1)
                w = w.masked_fill(none[None, :, None], 0)
                out[rows, h * group:(h + 1) * group] = torch.einsum("gmt,td->mgd", w, v)
    return {"out": out}
