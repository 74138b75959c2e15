"""Pins of oracle/q8.py: worked values and invariants."""

import numpy as np
import pytest

from oracle import q8 as Q
from oracle.attention import paged_decode_attention


def test_e4m3_values():
    v = Q.e4m3_values()
    assert v[0] == 0 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7e] == 448.0
    assert np.isnan(v[0x7f]) and np.isnan(v[0xff]) and v[0xb8] == -1.0
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.int64).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, v, equal_nan=True)


def test_round_e4m3():
    v = Q.e4m3_values()
    finite = np.unique(v[np.isfinite(v)])
    assert np.array_equal(Q.round_e4m3(finite), finite)
    middle = (finite[1:] + finite[:-1]) / 2
    for lo, mid, hi in zip(finite[:-1], middle, finite[1:]):
        even = [x for x in (lo, hi) if not (np.flatnonzero(v == x)[0] & 1)]
        assert Q.round_e4m3(mid) == even[0]
        assert Q.round_e4m3(np.nextafter(mid, -1e9)) == lo and Q.round_e4m3(np.nextafter(mid, 1e9)) == hi
    assert Q.round_e4m3(1e9) == 448 and Q.round_e4m3(-1e9) == -448


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_write_by_hand(kind):
    """Block size 8; a row of magnitude 2, then one of 4 in the same block: the
    first row's codes halve, the scale doubles."""
    top = Q.TOP[kind]
    codes, scales = np.zeros((2, 1, 8, 4)), np.zeros((2, 1))
    tables = [[1]]
    Q.write(codes, scales, np.array([[[2.0, -1.0, 0.5, 0.0]]]), tables, [1], None, kind)
    assert scales[1, 0] == float(np.float32(2 / top))
    assert codes[1, 0, 0, 0] == top and codes[1, 0, 0, 3] == 0
    Q.write(codes, scales, np.array([[[1.0, -4.0, 0.0, 3.0]]]), tables, [2], None, kind)
    assert scales[1, 0] == float(np.float32(4 / top))
    first = [64, -32, 16, 0] if kind == "int8" else [224, -112, 56, 0]  # 63.5 and -31.75 (of -64), 15.875 (of 32)
    assert codes[1, 0, 0].tolist() == first
    assert codes[1, 0, 1, 1] == -top
    assert (codes[0] == 0).all() and (codes[1, 0, 2:] == 0).all()
    # the block's first position again: a fresh block, whatever the scale was
    Q.write(codes, scales, np.array([[[0.5, 0, 0, 0]]]), tables, [1], None, kind)
    assert scales[1, 0] == float(np.float32(0.5 / top)) and codes[1, 0, 0, 0] == top


def test_written_values_are_near():
    rng = np.random.default_rng(0)
    rows = rng.standard_normal((40, 2, 16)).astype(np.float16)
    tables = [[2, 0, 3], [1, 4, 5]]
    for kind, bound in (("int8", lambda a, x: a / 127 / 2), ("e4m3", lambda a, x: np.maximum(x * 2.0 ** -4, a / 448 * 2.0 ** -10))):
        codes, scales = np.zeros((6, 2, 8, 16)), np.zeros((6, 2))
        Q.write(codes, scales, rows, tables, [17, 23], [0, 17, 40], kind)
        for s, (lo, n) in enumerate(((0, 17), (17, 23))):
            for p in range(n):
                b = tables[s][p // 8]
                got = codes[b, :, p % 8] * scales[b][:, None]
                x = rows[lo + p].astype(np.float64)
                a = scales[b][:, None] * Q.TOP[kind]
                assert (np.abs(got - x) <= bound(a, np.abs(x)) * (1 + 1e-6)).all()


def test_decode_is_the_decode():
    """Scales of one and no list: the fp16 decode's oracle; a list of every block
    in any order: the same; identical keys: the mean of the listed values."""
    rng = np.random.default_rng(1)
    kc, vc = rng.standard_normal((9, 2, 8, 16)), rng.standard_normal((9, 2, 8, 16))
    q = rng.standard_normal((3, 4, 16))
    tables, lens = np.array([[3, 1, 0, -1], [8, 4, 5, 6], [2, -1, -1, -1]]), np.array([20, 32, 1])
    ref = paged_decode_attention(q, kc, vc, tables, lens, 0.25)
    out = Q.decode(q, kc, vc, tables, lens, 0.25)[0]
    assert np.allclose(out, ref, rtol=0, atol=1e-12)
    lists = [[[2, 0, 1]] * 2, [[3, 2, 1, 0]] * 2, [[0]] * 2]
    assert np.allclose(Q.decode(q, kc, vc, tables, lens, 0.25, lists)[0], ref, rtol=0, atol=1e-12)
    kc[:] = 1.0
    out = Q.decode(q, kc, vc, tables, lens, 0.25, [[[2]] * 2, [[1, 3]] * 2, [[]] * 2])[0]
    assert np.allclose(out[0, 0], vc[0, 0, :4].mean(axis=0))
    assert np.allclose(out[1, 3], np.concatenate([vc[4, 1], vc[6, 1]]).mean(axis=0))
    assert (out[2] == 0).all()


def test_bounds_hold_and_selection():
    rng = np.random.default_rng(2)
    keys = rng.standard_normal((8, 1, 8, 16))
    tables, lens = [[7, 3, 0, 1, 5, 2]], [44]
    bounds = np.zeros((8, 1, 2, 16))
    Q.key_bounds(bounds, keys, tables, lens, [0, 44])
    assert (bounds[4] == 0).all() and (bounds[6] == 0).all()
    assert np.array_equal(bounds[2, 0, 0], keys[2, 0, :4].max(axis=0))
    q = rng.standard_normal((1, 2, 16))
    score = {}
    for b, phys in enumerate(tables[0]):
        seen = keys[phys, 0, :min(8, 44 - 8 * b)]
        score[b] = max((np.maximum(q[0, h] * bounds[phys, 0, 0], q[0, h] * bounds[phys, 0, 1])).sum() for h in range(2))
        assert (seen @ q[0].T).max() <= score[b] + 1e-12
    kept, number = Q.select(q, bounds, tables, lens, 8, 4, 1, 1)
    middle = sorted(sorted(range(1, 5), key=lambda b: -score[b])[:2])
    assert number[0, 0] == 4 and kept[0, 0].tolist() == [0] + middle + [5]
    bounds[:] = 1.0  # ties: the lowest index
    assert Q.select(q, bounds, tables, lens, 8, 4, 0, 1)[0][0, 0].tolist() == [0, 1, 2, 5]
    assert Q.select(q, bounds, tables, [13], 8, 4, 0, 1)[0][0, 0].tolist() == [0, 1, -1, -1]
    bounds[1, 0, 0, 3] = np.nan  # not finite: the largest
    assert Q.select(q, bounds, tables, lens, 8, 2, 0, 1)[0][0, 0].tolist() == [3, 5]
