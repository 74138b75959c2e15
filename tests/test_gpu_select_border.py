"""The choice of blocks where scores are alike to many digits, against integers:
an fp16 value is a multiple of 2^-24, so a score is a whole number of 2^-48 and
Python holds it exactly."""

import numpy as np
import pytest
import torch

import test_gpu_q8 as G
import test_gpu_select as S

pytestmark = pytest.mark.gpu
pkv = G.pkv


def whole(x):
    """fp16 values as whole numbers of 2^-24 (Python's)."""
    return (x.astype(np.float64) * 2.0 ** 24).astype(np.int64).astype(object)


def exact_scores(q, bounds, table, kvh):
    """Scores of one sequence's blocks, in 2^-48: q [H][D], bounds [NB][Hkv][2][D]."""
    group = q.shape[0] // bounds.shape[1]
    b = whole(bounds[table, kvh])
    best = None
    for h in whole(q[kvh * group:(kvh + 1) * group]):
        x = (np.where(h >= 0, h, 0) * b[:, 0] + np.where(h < 0, h, 0) * b[:, 1]).sum(axis=1)
        best = x if best is None else np.maximum(best, x)
    return best.tolist()


def check(pkv, q, bounds, tables, lens, bs, keep, first=0, last=0):
    selected, number = S.select(pkv, q, bounds, tables, lens, bs, keep, first, last)
    for s in range(len(lens)):
        blocks = -(-int(lens[s]) // bs)
        for k in range(bounds.shape[1]):
            assert number[s, k] == min(blocks, keep)
            if blocks <= keep:
                continue
            score = exact_scores(q[s], bounds, tables[s, :blocks], k)
            kept = set(range(first)) | set(range(blocks - last, blocks))
            for b in sorted(range(blocks), key=lambda b: (-score[b], b)):
                if len(kept) >= keep:
                    break
                kept.add(b)
            assert selected[s, k].tolist() == sorted(kept)


def wider(tables, columns):
    return np.concatenate([tables, np.full((len(tables), columns), -1, np.int32)], axis=1)


# more columns than 4096 take the kernels whose scores are in global memory
@pytest.mark.parametrize("columns", [0, 5000])
@pytest.mark.parametrize("blocks", [40, 128, 400, 2500])
@pytest.mark.parametrize("h,d", [(1, 64), (4, 128), (11, 64)])
def test_large_terms_that_cancel(pkv, h, d, blocks, columns):
    """A pair of channels at +3e6 and -3e6 in every score; blocks differ by fp16's
    smallest steps in one of eight other channels."""
    q, bounds, tables, lens = S.make(1, h, 1, d, 8, [8 * blocks, 8 * blocks - 5])
    rng = np.random.default_rng(blocks + d)
    bounds[:] = bounds[0]
    q[:, :, 0], q[:, :, 1] = 1750.0, 1750.0
    bounds[:, :, :, 0], bounds[:, :, :, 1] = 1750.0, -1750.0
    bounds[:, :, :, 2:10] = 0
    bounds[np.arange(len(bounds)), :, :, rng.integers(2, 10, len(bounds))] = \
        (rng.integers(-8, 9, (len(bounds), 1, 1)) * 2.0 ** -24).astype(np.float16)
    check(pkv, q, bounds, wider(tables, columns), lens, 8, blocks // 2)
    check(pkv, q, bounds, wider(tables, columns), lens, 8, blocks // 3, 2, 5)


@pytest.mark.parametrize("columns", [0, 5000])
@pytest.mark.parametrize("blocks", [60, 500])
@pytest.mark.parametrize("h,d", [(1, 64), (4, 128), (16, 128)])
def test_the_same_terms_in_another_order(pkv, h, d, blocks, columns):
    """Equal scores whose terms, of very different sizes, stand in other channels:
    the lowest index wins."""
    q, bounds, tables, lens = S.make(2, h, 1, d, 8, [8 * blocks])
    rng = np.random.default_rng(blocks + d)
    q = np.array([60000.0, 37.0, 0.011, 3e-6] * (d // 64)) * rng.choice([-1, 1, 0.9], (1, h, d // 16))
    q = np.broadcast_to(q[..., None], (1, h, d // 16, 16)).reshape(1, h, d).astype(np.float16)
    for few in range(5):  # five sets of blocks with equal scores
        x = rng.standard_normal((1, 2, d // 16, 16)).astype(np.float16)
        x = np.stack([np.maximum(x[:, 0], x[:, 1]), np.minimum(x[:, 0], x[:, 1])], axis=1)
        for b in range(few, len(bounds), 5):
            order = np.argsort(rng.random((1, 1, d // 16, 16)), axis=3)
            bounds[b] = np.take_along_axis(x, np.broadcast_to(order, x.shape), axis=3).reshape(1, 2, d)
    for keep in (1, 7, blocks // 10 + 1, blocks // 2):
        check(pkv, q, bounds, wider(tables, columns), lens, 8, keep)


@pytest.mark.parametrize("blocks", [100, 600])
def test_the_smallest_and_the_largest_terms(pkv, blocks):
    """Terms from 2^-48 to 2^32 in one score: the whole range counts."""
    q, bounds, tables, lens = S.make(3, 2, 1, 64, 8, [8 * blocks])
    rng = np.random.default_rng(blocks)
    bounds[:] = 0
    q[:] = 65504.0
    q[:, :, 32:] = 2.0 ** -24
    bounds[:, :, :, :16], bounds[:, :, :, 16:32] = 65504.0, -65504.0
    steps = rng.integers(-3, 4, (len(bounds), 1, 1, 32))
    bounds[:, :, :, 32:] = steps * 2.0 ** -24
    check(pkv, q, bounds, tables, lens, 8, blocks // 2)


@pytest.mark.parametrize("columns", [0, 5000])
@pytest.mark.parametrize("blocks", [100, 900])
@pytest.mark.parametrize("h,d", [(1, 64), (4, 128)])
def test_fp16_values_of_every_size(pkv, h, d, blocks, columns):
    """Queries and bounds of random bits, and the same with the large ones in pairs
    that cancel."""
    q, bounds, tables, lens = S.make(6, h, 1, d, 8, [8 * blocks])
    rng = np.random.default_rng(blocks + d)

    def bits(shape):
        sign, size = rng.integers(0, 2, shape) << 15, rng.integers(0, 0x7c00, shape)
        return (sign | size).astype(np.uint16).view(np.float16)

    q, bounds = bits(q.shape), bits(bounds.shape)
    bounds = np.stack([np.maximum(bounds[:, :, 0], bounds[:, :, 1]), np.minimum(bounds[:, :, 0], bounds[:, :, 1])], axis=2)
    check(pkv, q, bounds, wider(tables, columns), lens, 8, blocks // 2)
    bounds[...] = bounds[:, :, :1]  # hi = lo
    q[:, :, 1::2] = q[:, :, ::2]
    small = (np.abs(bounds[..., 1::2].astype(np.float64)) < 2.0 ** -8)
    bounds[..., 1::2] = np.where(small, bounds[..., 1::2], -bounds[..., ::2])
    bounds[..., ::2] = np.where(small, np.float16(2.0 ** -24), bounds[..., ::2])
    check(pkv, q, bounds, wider(tables, columns), lens, 8, blocks // 2)
