"""Oracle: attention of several new tokens per sequence over the paged cache,
and the norm and rotation of query and key heads (fp64).

TEST INFRASTRUCTURE ONLY (see the package docstring).

Chunk attention.  Row i of a sequence's n new tokens is position
p = L - n + i; it sees position t when t < L and, under the causal mask,
t <= p and (with a window w) t > p - w.  Its output is the softmax-weighted
sum of the visible positions' values, zeros where it sees none: the
definition of attention, with the positions found through the block table as
in attention.py.  Positions that a row does not see are left out before any
product, so nothing they hold can reach it.

Norm and rotation.  y = x w / sqrt(mean(x^2) + eps); a pair (a, b) turns by
its angle as the complex number a + ib does.
"""

import numpy as np

from .attention import token_location


def gather_positions(cache, table_row, positions, kv_head):
    """fp64 [len(positions)][D]: rows of one KV head, found one by one."""
    bs = cache.shape[2]
    out = np.empty((len(positions), cache.shape[3]), dtype=np.float64)
    for k, t in enumerate(positions):
        blk, off = token_location(table_row, t, bs)
        if not 0 <= blk < cache.shape[0]:
            raise ValueError(f"position {t}: physical block {blk} outside the pool")
        out[k] = cache[blk, kv_head, off]
    return out


def visible(length, n, i, causal, window):
    """The positions that row i of n sees, as a range."""
    if not causal:
        return range(0, length)
    p = length - n + i
    first = max(0, p - window + 1) if window else 0
    return range(min(first, max(p + 1, 0)), max(p + 1, 0))


def paged_chunk_attention(query, key_cache, value_cache, block_tables, context_lens, query_starts, scale,
                          causal=True, window=0):
    """-> (out, spread, reach, count, top), fp64.

    out [T][H][D]; rows of no sequence stay NaN.  For error bounds: spread
    [T][H][D] = sum_t softmax_t |v_t|, reach [T][H] = the largest
    scale * sum_i |q_i k_t,i| over the visible t, count [T][H] = how many
    positions the row sees, top [T][H][D] = the largest |v_t|.
    """
    num_tokens, heads, d = query.shape
    group = heads // key_cache.shape[1]
    out = np.full(query.shape, np.nan)
    spread = np.zeros(query.shape)
    top = np.zeros(query.shape)
    reach = np.zeros((num_tokens, heads))
    count = np.zeros((num_tokens, heads))
    for s in range(len(context_lens)):
        lo, hi = int(query_starts[s]), int(query_starts[s + 1])
        n, length = hi - lo, int(context_lens[s])
        if n == 0:
            continue
        seen = [visible(length, n, i, causal, window) for i in range(n)]
        first = min((r.start for r in seen if len(r)), default=0)
        last = max((r.stop for r in seen if len(r)), default=0)
        for kvh in range(key_cache.shape[1]):
            keys = gather_positions(key_cache, block_tables[s], range(first, last), kvh)
            values = gather_positions(value_cache, block_tables[s], range(first, last), kvh)
            for i, r in enumerate(seen):
                k, v = keys[r.start - first:r.stop - first], values[r.start - first:r.stop - first]
                for h in range(kvh * group, (kvh + 1) * group):
                    if len(r) == 0:
                        out[lo + i, h] = 0.0
                        continue
                    q = query[lo + i, h].astype(np.float64)
                    with np.errstate(invalid="ignore", over="ignore"):
                        x = scale * (k @ q)
                        w = np.exp(x - x.max())
                        w /= w.sum()
                        out[lo + i, h] = w @ v
                        spread[lo + i, h] = w @ np.abs(v)
                        top[lo + i, h] = np.abs(v).max(axis=0)
                        reach[lo + i, h] = scale * np.max(np.abs(k) @ np.abs(q))
                    count[lo + i, h] = len(r)
    return out, spread, reach, count, top


def norm_rope(x, weight, eps, positions, cos_sin, interleaved):
    """x [T][heads][D] -> (y, size) fp64: y normed (weight not None) and
    rotated (cos_sin not None, [P][rot]); size = |a| + |b| of each element's
    pair (|y| where nothing is rotated), for error bounds."""
    y = np.asarray(x, dtype=np.float64).copy()
    if weight is not None:
        mean = (y * y).mean(axis=-1, keepdims=True)
        with np.errstate(divide="ignore", invalid="ignore"):
            y = y / np.sqrt(mean + eps) * np.asarray(weight, dtype=np.float64)
    size = np.abs(y)
    if cos_sin is None or cos_sin.shape[1] == 0:
        return y, size
    rot = cos_sin.shape[1]
    half = rot // 2
    if interleaved:
        first, second = np.arange(0, rot, 2), np.arange(1, rot, 2)
    else:
        first, second = np.arange(half), np.arange(half, rot)
    row = np.asarray(cos_sin, dtype=np.float64)[np.asarray(positions)]
    turn = (row[:, :half] + 1j * row[:, half:])[:, None, :]
    z = (y[..., first] + 1j * y[..., second]) * turn
    both = np.abs(y[..., first]) + np.abs(y[..., second])
    y[..., first], y[..., second] = z.real, z.imag
    size[..., first] = both
    size[..., second] = both
    return y, size
