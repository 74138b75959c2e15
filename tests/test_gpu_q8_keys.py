"""The int8 decode's scores are products of the queries and the codes, and off by
no more than such products are: nothing that cancels is added to them."""

import numpy as np
import pytest
import torch

import test_gpu_q8 as G

pytestmark = pytest.mark.gpu
pkv = G.pkv


def strict(c, out):
    """Within the tolerance of the decode's tests, without its part for int8 (256 steps of the scale)."""
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    ref, spread, reach, count, top = c.oracle()
    got = out.float().cpu().numpy().astype(np.float64)
    over = np.abs(got - ref) / G.bound(ref, spread, reach, count, top, c.d)
    assert over.max() <= 1.0, (over.max(), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("h,hkv,d,bs,lens", [(1, 1, 64, 16, [300, 40, 7]), (8, 2, 128, 16, [500, 1200, 3]),
                                            (16, 1, 64, 64, [900, 130]), (4, 4, 128, 8, [77, 2000, 9])])
def test_large_queries_where_the_codes_are_zero(pkv, h, hkv, d, bs, lens):
    """A block's scale is that of an outlier channel, whose query is zero; the
    channels with large queries are below half a code."""
    c = G.Case(1, "int8", h, hkv, d, bs, lens, q_std=1.0)
    q = c.q.reshape(len(lens), h, d)
    q[:, :, d // 2:] = (c.rng.standard_normal((len(lens), h, d - d // 2)) * 3000).astype(np.float16)
    q[:, :, 0] = 0
    keys = c.pools[0]
    keys[..., 1:d // 2] = np.clip(np.round(keys[..., 1:d // 2] / 40), -4, 4)
    keys[..., d // 2:] = 0
    keys[..., 0] = 127
    c.gpu()
    strict(c, c.call(pkv))
    c.pick(9, "any").gpu()
    strict(c, c.call(pkv))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,hkv", [(2, 2), (8, 1), (12, 1)])
def test_ordinary_codes(pkv, h, hkv, d):
    c = G.Case(2, "int8", h, hkv, d, 16, [1, 900, 33, 2500]).gpu()
    strict(c, c.call(pkv))


def test_every_code(pkv):
    """Each of -128 to 127 in every channel, keys and values."""
    for d in (64, 128):
        c = G.Case(3, "int8", 4, 1, d, 16, [256], q_std=0.05)
        for pool, turn in zip(c.pools, (1, 3)):
            t = np.arange(256).reshape(16, 1, 16, 1)
            pool[c.tables[0, :16]] = (t * turn + np.arange(d)) % 256 - 128
        c.gpu()
        strict(c, c.call(pkv))
