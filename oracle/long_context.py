"""Plain numpy forms of the long-context cache operators (test infrastructure,
as the rest of this package): the 4-bit rows, decode attention with each
token's weight, the choice of the tokens to keep and the moving of their rows.

Rows are formed in fp32 exactly as the format says (IEEE, round to nearest
even), so the bytes of a cache can be compared; attention is in double.
"""
import numpy as np

GROUP = 32


def q4_quantise(x):
    """uint8 rows [..., 5 * d / 8] of float32 values x [..., d]."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], np.float32(0), g)
    m = np.clip(g.min(-1), np.float32(-65504), np.float32(65504)).astype(np.float16)
    mf = m.astype(np.float32)
    s = np.clip((g.max(-1) - mf) / np.float32(15), 0, 1023).astype(np.float16)
    sf = s.astype(np.float32)
    y = (g - mf[..., None]) / np.where(sf > 0, sf, np.float32(1))[..., None]
    code = np.where(sf[..., None] > 0, np.clip(np.rint(y), 0, 15), 0).astype(np.uint8)
    s = np.where(bad, np.float16(np.nan), s)
    m = np.where(bad, np.float16(np.nan), m)
    code = np.where(bad[..., None], 0, code).astype(np.uint8).reshape(x.shape)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    pairs = np.stack([s, m], -1).reshape(*x.shape[:-1], x.shape[-1] // GROUP * 2)
    return np.concatenate([packed, pairs.view(np.uint8)], -1)


def q4_restore(rows):
    """float64 values of uint8 rows."""
    d = rows.shape[-1] * 8 // 5
    packed = rows[..., :d // 2]
    pairs = np.ascontiguousarray(rows[..., d // 2:]).view(np.float16).astype(np.float64)
    code = np.empty(rows.shape[:-1] + (d,))
    code[..., 0::2] = packed & 15
    code[..., 1::2] = packed >> 4
    return code * np.repeat(pairs[..., 0::2], GROUP, -1) + np.repeat(pairs[..., 1::2], GROUP, -1)


def q4_write(key, cache, slots, swa=None):
    """key [N, H, d] float32 into cache [nb, bs, H, rb] (in place)."""
    flat = cache.reshape(-1, *cache.shape[2:])
    rows = q4_quantise(key)
    for t, s in enumerate(slots):
        if s >= 0 and swa is not None:
            s = swa[s] if s < len(swa) else -1
        if 0 <= s < len(flat):
            flat[s] = rows[t]


def decode(q, k, v, table, lens, block, scale, limit=None):
    """Attention of q [B, HQ, d] over pools k, v [nb, bs, HKV, d] (float64):
    outputs [B, HQ, d] and weights [B, HKV, T] summed over each kv head's
    query heads (T the longest length; 0 for dropped blocks)."""
    B, HQ, d = q.shape
    nb, bs, H, _ = k.shape
    G = HQ // H
    L = [max(0, min(int(n), table.shape[1] * bs, limit if limit is not None else 1 << 62))
         for n in lens]
    out = np.zeros((B, HQ, d))
    sums = np.zeros((B, H, max(1, max(L, default=1))))
    for b in range(B):
        t = np.arange(L[b])
        blk = table[b][t // bs].astype(np.int64)
        t = t[(blk >= 0) & (blk < nb)]
        blk = blk[(blk >= 0) & (blk < nb)]
        if t.size == 0:
            continue
        kk, vv = k[blk, t % bs], v[blk, t % bs]
        for h in range(HQ):
            s = kk[:, h // G] @ q[b, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[b, h] = p @ vv[:, h // G]
            sums[b, h // G, t] += p
    return out, sums


def evict_select(sums, lens, budget, sink, recent, table=None, block=1, num_blocks=0):
    """keep [B, H, budget] int32 (-1 behind the kept), new_lens [B].  With a
    table, tokens of blocks outside the pool or past it do not take part."""
    B, H, T = sums.shape
    keep = np.full((B, H, budget), -1, np.int32)
    new = np.zeros(B, np.int32)
    for b in range(B):
        L = max(0, min(int(lens[b]), T))
        there = range(L)
        if table is not None:
            there = [t for t in there if t // block < table.shape[1]
                     and 0 <= table[b, t // block] < num_blocks]
        new[b] = min(len(there), budget)
        for h in range(H):
            def rank(t):
                x = float(sums[b, h, t])
                free = sink <= t < L - recent
                return (free, np.isnan(x), 0.0 if np.isnan(x) else -x, t)
            order = sorted(there, key=rank)
            keep[b, h, :new[b]] = sorted(order[:budget])
    return keep, new


def compact(cache, keep, keep_lens, src_table, dst_table):
    """Rows of cache [nb, bs, H, ...] moved (in place), in the order of j."""
    nb, bs = cache.shape[:2]
    for b in range(keep.shape[0]):
        for g in range(keep.shape[1]):
            for j in range(min(int(keep_lens[b]), keep.shape[2])):
                t = int(keep[b, g, j])
                if t < 0 or t // bs >= src_table.shape[1] or j // bs >= dst_table.shape[1]:
                    continue
                s, d = int(src_table[b, t // bs]), int(dst_table[b, j // bs])
                if 0 <= s < nb and 0 <= d < nb:
                    cache[d, j % bs, g] = cache[s, t % bs, g]
