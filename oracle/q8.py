"""Oracle: the 8-bit cache, its decode, and the choice of blocks (fp64).

TEST INFRASTRUCTURE ONLY (see the package docstring).

A block and KV head holds codes of one scale a / M: a the largest magnitude it
holds, M = 127 (int8) or 448 (e4m3).  New rows x become the code nearest to
M x / a, ties to even; where they raise a from a0, the rows before them become
the code nearest to code * a0 / a.  The decode is the definition of attention on
codes times scales; a block list leaves the positions of other blocks out.
"""

import numpy as np

TOP = {"int8": 127.0, "e4m3": 448.0}


def e4m3_values():
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3
    mantissa bits; exponent 0 has no leading one; the last code of each sign is
    NaN (there are no infinities)."""
    values = np.empty(256)
    for code in range(256):
        exponent, mantissa = (code >> 3) & 15, code & 7
        v = mantissa * 2.0 ** -9 if exponent == 0 else (8 + mantissa) * 2.0 ** (exponent - 10)
        if code & 127 == 127:
            v = np.nan
        values[code] = -v if code & 128 else v
    return values


def round_e4m3(y):
    """Nearest e4m3 value, ties to even, past the largest: the largest."""
    y = np.asarray(y, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        exponent = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
        step = np.exp2(np.minimum(exponent, 8) - 3)
        return np.clip(np.rint(y / step) * step, -448.0, 448.0)


def round_codes(y, kind):
    """Exact quotients -> code values (fp64)."""
    if kind == "int8":
        return np.where(np.isnan(y), 0.0, np.clip(np.rint(y), -127, 127))
    return round_e4m3(y)


def write(codes, scales, rows, tables, lens, starts, kind):
    """codes [NB][Hkv][bs][D] and scales [NB][Hkv] (fp64, changed in place) after
    the write of rows [T][Hkv][D]; starts None: one row per sequence."""
    top, bs, hkv = TOP[kind], codes.shape[2], codes.shape[1]
    for s, length in enumerate(lens):
        lo, hi = (s, s + 1) if starts is None else (int(starts[s]), int(starts[s + 1]))
        length, n = int(length), hi - lo
        positions = [p for p in range(length - n, length) if p >= 0]
        for block in sorted({p // bs for p in positions}):
            inside = [p for p in positions if p // bs == block]
            phys = int(tables[s][block])
            first = inside[0] % bs
            for h in range(hkv):
                new = np.array([rows[lo + p - (length - n), h] for p in inside], dtype=np.float64)
                finite = np.abs(new[np.isfinite(new)])
                a0 = float(np.float16(np.float32(scales[phys, h]) * np.float32(top))) if first else 0.0
                a = max(a0, finite.max() if finite.size else 0.0)
                by = a if a > 0 else 1.0
                if first and a > a0:
                    codes[phys, h, :first] = round_codes(codes[phys, h, :first] * a0 / by, kind)
                codes[phys, h, first:first + len(inside)] = round_codes(top * new / by, kind)
                if not first or a > a0:
                    scales[phys, h] = float(np.float32(a) / np.float32(top))


def key_bounds(bounds, keys, tables, lens, starts):
    """bounds [NB][Hkv][2][D] (fp64, changed in place) of the blocks that hold new
    tokens; keys [NB][Hkv][bs][D] fp64."""
    bs = keys.shape[2]
    for s, length in enumerate(lens):
        n = 1 if starts is None else int(starts[s + 1]) - int(starts[s])
        for block in sorted({p // bs for p in range(int(length) - n, int(length)) if p >= 0}):
            phys = int(tables[s][block])
            seen = keys[phys, :, :min(bs, int(length) - block * bs)]
            bounds[phys, :, 0], bounds[phys, :, 1] = seen.max(axis=1), seen.min(axis=1)


def select(query, bounds, tables, lens, block_size, keep, first, last):
    """-> selected [N][Hkv][keep] (ascending, then -1), num_selected [N][Hkv]."""
    n, hkv = len(lens), bounds.shape[1]
    group = query.shape[1] // hkv
    selected = np.full((n, hkv, keep), -1, np.int64)
    number = np.zeros((n, hkv), np.int64)
    for s in range(n):
        blocks = -(-int(lens[s]) // block_size)
        for h in range(hkv):
            score = []
            for b in range(blocks):
                hi, lo = bounds[int(tables[s][b]), h]
                best = -np.inf
                for q in query[s, h * group:(h + 1) * group].astype(np.float64):
                    with np.errstate(invalid="ignore"):
                        x = np.sum(np.where(np.isnan(q), q, np.maximum(q, 0)) * hi + np.minimum(q, 0) * lo)
                    best = max(best, x if np.isfinite(x) else np.inf)
                score.append(best)
            kept = set(range(blocks)) if blocks <= keep else set(range(first)) | set(range(blocks - last, blocks))
            for b in sorted(range(blocks), key=lambda b: (-score[b], b)):
                if len(kept) >= min(keep, blocks):
                    break
                kept.add(b)
            number[s, h] = len(kept)
            selected[s, h, :len(kept)] = sorted(kept)
    return selected, number


def decode(query, keys, values, tables, lens, scale, lists=None):
    """keys, values [NB][Hkv][bs][D] fp64 (codes times scales) -> (out, spread,
    reach, count, top): the output [N][H][D] and, for error bounds, sum_t w_t
    |v_t|, the largest scale * sum_i |q_i k_t,i|, the positions seen, the largest
    |v_t|.  lists[s][h]: the logical blocks to look at."""
    n, heads, d = query.shape
    hkv, bs = keys.shape[1], keys.shape[2]
    group = heads // hkv
    out, spread, top = np.zeros(query.shape), np.zeros(query.shape), np.zeros(query.shape)
    reach, count = np.zeros((n, heads)), np.zeros((n, heads))
    for s in range(n):
        length = int(lens[s])
        for kvh in range(hkv):
            blocks = range(-(-length // bs)) if lists is None else lists[s][kvh]
            at = [(int(tables[s][b]), o) for b in blocks for o in range(bs) if b * bs + o < length]
            if not at:
                continue
            phys, off = np.array(at).T
            k, v = keys[phys, kvh, off], values[phys, kvh, off]
            for h in range(kvh * group, (kvh + 1) * group):
                q = query[s, h].astype(np.float64)
                x = scale * (k @ q)
                w = np.exp(x - x.max())
                w /= w.sum()
                out[s, h] = w @ v
                spread[s, h] = w @ np.abs(v)
                top[s, h] = np.abs(v).max(axis=0)
                reach[s, h] = scale * np.max(np.abs(k) @ np.abs(q))
                count[s, h] = len(at)
    return out, spread, reach, count, top
