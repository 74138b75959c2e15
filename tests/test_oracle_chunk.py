"""Pins of the chunk-attention and norm-and-rotation oracle."""

import math

import numpy as np
import pytest

from oracle import attention as OA
from oracle import chunk as OK


def _case(rng, n, length, hkv=2, group=2, d=8, bs=4):
    nb = -(-max(length, 1) // bs) + 2
    table = rng.permutation(nb)[None].astype(np.int64)
    kc, vc = rng.standard_normal((2, nb, hkv, bs, d))
    q = rng.standard_normal((n, hkv * group, d))
    return q, kc, vc, table


@pytest.mark.parametrize("n,length", [(1, 1), (1, 13), (5, 5), (4, 11)])
def test_each_row_is_a_decode_of_its_prefix(n, length):
    rng = np.random.default_rng(n * 100 + length)
    q, kc, vc, table = _case(rng, n, length)
    out, _, _, count, _ = OK.paged_chunk_attention(q, kc, vc, table, [length], [0, n], 0.3)
    for i in range(n):
        ref = OA.paged_decode_attention_one(q[i], kc, vc, table[0], length - n + i + 1, 0.3)
        assert np.allclose(out[i], ref, rtol=0, atol=1e-14)
        assert (count[i] == length - n + i + 1).all()


def test_window_of_one_returns_the_rows_own_value():
    rng = np.random.default_rng(3)
    q, kc, vc, table = _case(rng, 6, 9)
    out, *_ = OK.paged_chunk_attention(q, kc, vc, table, [9], [0, 6], 0.3, window=1)
    for i in range(6):
        blk, off = OA.token_location(table[0], 3 + i, 4)
        assert np.array_equal(out[i], np.repeat(vc[blk, :, off], 2, axis=0))


def test_without_the_causal_mask_every_row_sees_all():
    rng = np.random.default_rng(4)
    q, kc, vc, table = _case(rng, 7, 3)   # more queries than positions
    out, *_ = OK.paged_chunk_attention(q, kc, vc, table, [3], [0, 7], 0.3, causal=False)
    for i in range(7):
        assert np.allclose(out[i], OA.paged_decode_attention_one(q[i], kc, vc, table[0], 3, 0.3), atol=1e-14)


def test_rows_that_see_nothing_are_zero_and_rows_outside_are_untouched():
    rng = np.random.default_rng(5)
    q, kc, vc, table = _case(rng, 8, 3)
    out, *_ = OK.paged_chunk_attention(q, kc, vc, table, [3], [1, 6], 0.3)   # 5 rows, 3 positions
    assert np.isnan(out[0]).all() and np.isnan(out[6:]).all()
    assert (out[1:3] == 0).all() and np.isfinite(out[3:6]).all()


def test_hidden_positions_do_not_reach_a_row():
    rng = np.random.default_rng(6)
    q, kc, vc, table = _case(rng, 4, 8)
    clean, *_ = OK.paged_chunk_attention(q, kc, vc, table, [8], [0, 4], 0.3)
    blk, off = OA.token_location(table[0], 7, 4)
    kc[blk, :, off], vc[blk, :, off] = np.nan, np.inf
    out, *_ = OK.paged_chunk_attention(q, kc, vc, table, [8], [0, 4], 0.3)
    assert np.array_equal(out[:3], clean[:3]) and np.isnan(out[3]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance_only(interleaved):
    rng = np.random.default_rng(7)
    d, rot = 16, 16
    angle = np.arange(64)[:, None] * 100.0 ** (-np.arange(rot // 2) / (rot // 2))
    table = np.concatenate([np.cos(angle), np.sin(angle)], axis=1)
    x, y = rng.standard_normal((2, 1, 1, d))
    dots = []
    for base in (0, 11, 40):
        a, _ = OK.norm_rope(x, None, 0.0, [base], table, interleaved)
        b, _ = OK.norm_rope(y, None, 0.0, [base + 5], table, interleaved)
        assert math.isclose(np.linalg.norm(a), np.linalg.norm(x), rel_tol=1e-12)
        dots.append(float((a * b).sum()))
    assert np.allclose(dots, dots[0], atol=1e-12)


def test_quarter_turn_swaps_the_pairs():
    table = np.array([[0.0, 0.0, 1.0, 1.0]])   # cos 0, sin 1
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    half, _ = OK.norm_rope(x, None, 0.0, [0], table, False)
    pairs, _ = OK.norm_rope(x, None, 0.0, [0], table, True)
    assert half.ravel().tolist() == [-3.0, -4.0, 1.0, 2.0, 9.0]
    assert pairs.ravel().tolist() == [-2.0, 1.0, -4.0, 3.0, 9.0]


def test_norm_by_hand():
    y, _ = OK.norm_rope(np.array([[[3.0, 4.0]]]), np.array([1.0, 2.0]), 0.0, None, None, False)
    r = math.sqrt(12.5)
    assert np.allclose(y.ravel(), [3 / r, 8 / r])
    z, _ = OK.norm_rope(np.zeros((1, 1, 2)), np.ones(2), 1e-6, None, None, False)
    assert (z == 0).all()
