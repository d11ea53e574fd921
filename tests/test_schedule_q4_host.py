"""Host model of the cut the 4-bit decode kernel derives on the GPU.

Units of 64 tokens lie end to end; unit t of sequence b sits at cost
t + kPC (b + 1); the line of length total = units + kPC B is cut into
parts = min(chunks, total) equal parts.  A chunk starts at the first unit
whose cost reaches ceil(k total / parts), found as the first non-empty
sequence whose last unit reaches it (its first unit, where sequences stay
whole).  Partial slots: c - 1 for a piece that goes on from chunk c - 1,
chunks - 1 + (b or the chunk) for a split sequence's first piece.  Also the
host's bound on the chunks by the workspace's partial rows.
"""
import numpy as np
import pytest


def launch_chunks(slots_on_gpu, heads, seqs, num_splits):
    chunks, rows = slots_on_gpu // heads, seqs * num_splits - -(-seqs // 128)
    whole = num_splits == 1
    if whole:
        chunks = min(chunks, seqs)
    elif chunks - 1 + min(seqs, chunks - 1) > rows:
        chunks = rows - seqs + 1 if seqs < rows - seqs else rows // 2 + 1
    chunks = max(1, min(chunks, 32767))
    return chunks, chunks - 1 + min(seqs, chunks - 1), whole


def pieces(lens, chunks, whole, kpc):
    """Every chunk's pieces (b, first unit, end unit) as the kernel walks them."""
    n = [(max(0, x) + 63) // 64 for x in lens]
    B, units = len(n), sum(n)
    total = units + kpc * B
    parts = min(total, chunks)
    pre = np.concatenate([[0], np.cumsum(n)]).astype(int)

    def start(k):
        if k >= parts:
            return units
        x = -(-k * total // parts)
        for b in range(B):
            if n[b] and pre[b] + (0 if whole else n[b] - 1) + kpc * (b + 1) >= x:
                return int(pre[b]) if whole else max(x - kpc * (b + 1), int(pre[b]))
        return units
    out = []
    for c in range(chunks):
        lo, hi = start(c), start(c + 1)
        out.append([(b, max(lo, int(pre[b])), min(hi, int(pre[b + 1]))) for b in range(B)
                    if max(lo, int(pre[b])) < min(hi, int(pre[b + 1]))])
    return out, n, pre, total, parts


def check(lens, slots_on_gpu, heads, num_splits, kpc=2):
    B = len(lens)
    chunks, slots, whole = launch_chunks(slots_on_gpu, heads, B, num_splits)
    assert slots <= B * num_splits - -(-B // 128) or whole
    got, n, pre, total, parts = pieces(lens, chunks, whole, kpc)
    used, seen = set(), np.zeros(sum(n), int)
    count = {}
    for c, ps in enumerate(got):
        for b, lo, hi in ps:
            seen[lo:hi] += 1
            count.setdefault(b, []).append(c)
    assert (seen == 1).all()
    for b, cs in count.items():
        if whole:
            assert len(cs) == 1
            continue
        c_first = (int(pre[b]) + kpc * (b + 1)) * parts // total
        c_last = (int(pre[b]) + n[b] - 1 + kpc * (b + 1)) * parts // total
        assert cs == list(range(c_first, c_last + 1)), (b, cs, c_first, c_last)
        if c_last > c_first:
            for c in cs:
                s = c - 1 if c > c_first else chunks - 1 + (b if B <= chunks - 1 else c_first)
                assert 0 <= s < slots and s not in used
                used.add(s)


@pytest.mark.parametrize("heads", [1, 3, 8, 40])
def test_cut_invariants(heads):
    rng = np.random.default_rng(heads)
    for case in range(150):
        B = int(rng.integers(1, 130))
        top = int(rng.choice([1, 64, 65, 300, 4096, 30000]))
        lens = rng.integers(0, top + 1, B).tolist()
        if case % 5 == 0:
            lens[int(rng.integers(B))] = 60000
        splits = int(rng.choice([1, 2, 3, 10, 76, 1000]))
        check(lens, int(rng.choice([8, 304, 456])), heads, splits)


def test_cut_of_batches_of_one_and_of_many():
    for L in (1, 64, 65, 128, 9001, 131072):
        for splits in (1, 2, 141, 1216):
            check([L], 456, 4, splits)
            check([L, 0, 1], 456, 8, splits)
    check([1] * 2000, 456, 8, 2)
    check([0] * 50, 456, 8, 2)
    check([0] * 50, 456, 8, 1)
