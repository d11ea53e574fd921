"""Plain forms of the sliding-window operators in numpy, from their definitions
(include/pa.h): rotation by position in 64 bits, and attention rows over the
tokens that a window and a few first tokens leave."""
import numpy as np


def rotate(x, cos_sin, positions, interleaved):
    """x [N, H, d] with the first cos_sin.shape[1] elements of a head turned, in 64 bits, and the
    sum of the magnitudes of each element's terms."""
    x = np.asarray(x, np.float64)
    rot = cos_sin.shape[1]
    cs = np.asarray(cos_sin, np.float64)[positions]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y, size = x.copy(), np.abs(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
    size[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, size


def rotate_f32(x, cos_sin, positions, interleaved):
    """The same with every product and sum rounded to fp32."""
    x = np.asarray(x, np.float32)
    rot = cos_sin.shape[1]
    c, s = cos_sin[positions][:, None, :rot // 2], cos_sin[positions][:, None, rot // 2:]
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y = x.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def slots(slot_mapping, swa, num_slots):
    """Each token's slot, -1 where it has none."""
    out = []
    for s in slot_mapping:
        if swa is not None and s >= 0:
            s = swa[s] if s < len(swa) else -1
        out.append(int(s) if 0 <= s < num_slots else -1)
    return out


def visible(pos, window, num_sink):
    """The tokens that the query at position pos sees."""
    t = np.arange(max(0, pos + 1))
    return t[(t > pos - window) | (t < num_sink)]


def row(q, k_cache, v_cache, table, tokens, scale):
    """Attention of q [G, d] over these tokens of one kv head's pool [num_blocks, bs, d], in 64
    bits: output [G, d], weighted magnitudes [G, d], largest |score| bound and sum of |v|."""
    d = q.shape[-1]
    bs = k_cache.shape[1]
    blocks = np.asarray(table)[tokens // bs] if len(tokens) else np.zeros(0, int)
    there = (blocks >= 0) & (blocks < k_cache.shape[0])
    blocks, offs = blocks[there], tokens[there] % bs
    if not len(blocks):
        z = np.zeros((q.shape[0], d))
        return z, z, 0.0, 0.0
    k, v = k_cache[blocks, offs].astype(np.float64), v_cache[blocks, offs].astype(np.float64)
    q = q.astype(np.float64)
    s = scale * q @ k.T
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    size = abs(scale) * (np.abs(q) @ np.abs(k).T).max()
    return p @ v, p @ np.abs(v), size, np.abs(v).sum(0).max()


def decode(q, k_cache, v_cache, tables, lens, window, num_sink, scale):
    """Every row of a batch: q [B, H_Q, d], caches [num_blocks, bs, H_KV, d] -> what row() gives."""
    group = q.shape[1] // k_cache.shape[2]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    size, total = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    for b, n in enumerate(lens):
        t = visible(int(n) - 1, window, num_sink)
        for g in range(k_cache.shape[2]):
            h = slice(g * group, (g + 1) * group)
            out[b, h], mag[b, h], size[b, h], total[b, h] = row(
                q[b, h], k_cache[:, :, g], v_cache[:, :, g], tables[b], t, scale)
    return out, mag, size, total


def prefill(q, k_cache, v_cache, tables, starts, lens, window, num_sink, scale, rows=None):
    """Rows of a prompt batch: q [T, H_Q, d] -> what row() gives; rows: which of the T (all)."""
    group = q.shape[1] // k_cache.shape[2]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    size, total = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    for b, n in enumerate(lens):
        new = int(starts[b + 1] - starts[b])
        for j in range(new):
            i = int(starts[b]) + j
            if rows is not None and i not in rows:
                continue
            t = visible(int(n) - new + j, window, num_sink)
            for g in range(k_cache.shape[2]):
                h = slice(g * group, (g + 1) * group)
                out[i, h], mag[i, h], size[i, h], total[i, h] = row(
                    q[i, h], k_cache[:, :, g], v_cache[:, :, g], tables[b], t, scale)
    return out, mag, size, total
