"""GPU parity of the norm with rotation where a lane group takes four heads
(65536 lanes and more), for every number of lanes per head; tolerances are
those of test_gpu_rope.py."""

import numpy as np
import pytest
import torch

from oracle import cache_ops as OC
from pkv_testlib import bits16
from test_gpu_rope import Case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from paged_kv_cache_152_gb300 import build
    build.build()
    import paged_kv_cache_152_gb300 as m
    m.load()
    return m


# tokens, query and KV heads (no multiples of four, mostly), head_dim, rotated part: 8, 16 and 32 lanes per head
SHAPES = [(1500, 5, 3, 40, 32), (2000, 6, 2, 64, 64), (700, 7, 3, 128, 128), (900, 5, 2, 80, 48), (1100, 3, 1, 128, 0),
          (600, 5, 1, 256, 64), (500, 6, 3, 200, 96), (400, 9, 2, 256, 256)]


def many(t, h, hkv, d, kinds):
    return t * (h + kinds * hkv) * (8 if d <= 64 else 16 if d <= 128 else 32) >= 65536


@pytest.mark.parametrize("t,h,hkv,d,rot", SHAPES)
@pytest.mark.parametrize("norm", ["both", "key", "none"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_plain_and_in_place(pkv, t, h, hkv, d, rot, norm, interleaved):
    assert many(t, h, hkv, d, 1)
    c = Case(21, t, h, hkv, d, rot, norm).gpu()
    qo, ko = torch.full_like(c.tq, 7.0), torch.full_like(c.tk, 7.0)
    pkv.qk_norm_rope(qo, ko, c.tq, c.tk, interleaved=interleaved, eps=1e-5, status=c.status, **c.kw)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    check(qo, c.q, c.wq, 1e-5, c.pos, c.cs, interleaved)
    check(ko, c.k, c.wk, 1e-5, c.pos, c.cs, interleaved)
    pkv.qk_norm_rope(c.tq, c.tk, c.tq, c.tk, interleaved=interleaved, eps=1e-5, status=c.status, **c.kw)
    torch.cuda.synchronize()
    assert torch.equal(c.tq, qo) and torch.equal(c.tk, ko)
    assert np.array_equal(bits16(c.tv), bits16(c.v))


@pytest.mark.parametrize("t,h,hkv,d,rot", SHAPES + [(7, 32, 8, 128, 128), (33, 3, 1, 96, 96), (9, 4, 4, 256, 64)])
@pytest.mark.parametrize("bs", [8, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_into_the_cache(pkv, t, h, hkv, d, rot, bs, interleaved):
    """Keys within the bound, values bit for bit, every other slot untouched,
    padding slots skipped (the last three shapes: one head per group)."""
    c = Case(22, t, h, hkv, d, rot, bs=bs)
    c.slots[::5] = -1
    c.gpu()
    qo = torch.full_like(c.tq, 7.0)
    pkv.qk_norm_rope_and_cache(qo, c.tq, c.tk, c.tv, c.tkc, c.tvc, c.tslots, interleaved=interleaved, status=c.status,
                               **c.kw)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    check(qo, c.q, c.wq, 1e-6, c.pos, c.cs, interleaved)
    vc = c.vc.copy()
    OC.reshape_and_cache(c.v, c.v, np.zeros_like(vc), vc, c.slots)
    assert np.array_equal(bits16(c.tvc), bits16(vc))
    flat = c.tkc.transpose(1, 2).reshape(-1, hkv, d)
    rows = np.nonzero(c.slots >= 0)[0]
    got = torch.zeros_like(c.tk)
    got[rows] = flat[c.slots[rows]]
    check(got, c.k, c.wk, 1e-6, c.pos, c.cs, interleaved, rows)
    other = np.setdiff1d(np.arange(flat.shape[0]), c.slots)
    before = c.kc.transpose(0, 2, 1, 3).reshape(-1, hkv, d)
    assert np.array_equal(bits16(flat)[other], bits16(before)[other])


def test_bad_device_data_is_reported(pkv):
    """A position or a slot outside its range concerns its own token only,
    also where four heads go together."""
    c = Case(23, 700, 7, 3, 128, 128).gpu()
    good = torch.empty_like(c.tq)
    kc0, vc0 = c.tkc.clone(), c.tvc.clone()
    pkv.qk_norm_rope_and_cache(good, c.tq, c.tk, c.tv, c.tkc, c.tvc, c.tslots, status=c.status, **c.kw)
    pos, slots = c.kw["positions"].clone(), c.tslots.clone()
    pos[3], slots[698] = 5000, c.kc.shape[0] * 16
    qo = torch.full_like(c.tq, 7.0)
    kc, vc = kc0.clone(), vc0.clone()
    pkv.qk_norm_rope_and_cache(qo, c.tq, c.tk, c.tv, kc, vc, slots, status=c.status, **dict(c.kw, positions=pos))
    torch.cuda.synchronize()
    assert int(c.status.item()) == pkv.PKV_ERR_OUT_OF_RANGE
    rest = np.setdiff1d(np.arange(700), [3])
    assert (qo[3] == 7.0).all() and torch.equal(qo[rest], good[rest])
    for now, before, full in ((kc, kc0, c.tkc), (vc, vc0, c.tvc)):
        now, before, full = (x.transpose(1, 2).reshape(-1, 3, 128) for x in (now, before, full))
        bad = c.slots[[3, 698]]
        assert torch.equal(now[bad], before[bad])
        kept = np.setdiff1d(c.slots, bad)
        assert torch.equal(now[kept], full[kept])


def test_slots_far_into_a_large_pool(pkv):
    """Element offsets past 2^32 in each cache."""
    t, hkv, bs, d = 700, 3, 16, 128
    nb = (1 << 32) // (hkv * bs * d) + 60
    c = Case(24, t, 7, hkv, d, d).gpu()
    kc = torch.empty((nb, hkv, bs, d), dtype=torch.float16, device="cuda")
    vc = torch.empty_like(kc)
    slots = torch.arange(nb * bs - t, nb * bs, device="cuda")
    qo = torch.empty_like(c.tq)
    pkv.qk_norm_rope_and_cache(qo, c.tq, c.tk, c.tv, kc, vc, slots, status=c.status, **c.kw)
    tail = -(-t // bs)
    check(kc[-tail:].transpose(1, 2).reshape(-1, hkv, d)[-t:], c.k, c.wk, 1e-6, c.pos, c.cs, False)
    assert torch.equal(vc[-tail:].transpose(1, 2).reshape(-1, hkv, d)[-t:], c.tv)
    check(qo, c.q, c.wq, 1e-6, c.pos, c.cs, False)
    assert int(c.status.item()) == 0
