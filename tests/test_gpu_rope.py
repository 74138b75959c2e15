"""GPU parity of the query/key norm with rotation (and its cache write) with
the fp64 oracle.

Tolerance, per element: fp32 arithmetic of about a dozen roundings (the sum of
at most 256 squares counts as 256 of 2^-24 halved by the square root, the
rest as single ones), 2^-16 of |a| + |b| of the element's pair in all, and the
rounding of the result to fp16, 2^-11 of it, 2^-25 below the normal range.
"""

import numpy as np
import pytest
import torch

from oracle import cache_ops as OC
from oracle import chunk as OK
from pkv_testlib import bits16

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


def table(reach, rot, base=10000.0):
    angle = np.arange(reach)[:, None] * base ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)


def check(got, x, weight, eps, positions, cos_sin, interleaved, rows=slice(None)):
    ref, size = OK.norm_rope(x, weight, eps, positions, cos_sin, interleaved)
    got = got.float().cpu().numpy().astype(np.float64)
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2.0 ** -16 * size
    assert np.isfinite(got[rows]).all()
    over = (np.abs(got - ref) / tol)[rows]
    assert over.max(initial=0.0) <= 1.0, over.max()


class Case:
    def __init__(self, seed, t, h, hkv, d, rot, norm="both", bs=16, std=2.0, reach=5000):
        rng = np.random.default_rng(seed)
        self.q = (rng.standard_normal((t, h, d)) * std).astype(np.float16)
        self.k = (rng.standard_normal((t, hkv, d)) * std).astype(np.float16)
        self.v = (rng.standard_normal((t, hkv, d)) * std).astype(np.float16)
        self.wq = (1 + 0.2 * rng.standard_normal(d)).astype(np.float16) if norm in ("both", "query") else None
        self.wk = (1 + 0.2 * rng.standard_normal(d)).astype(np.float16) if norm in ("both", "key") else None
        self.cs = table(reach, rot) if rot else None
        self.pos = rng.integers(0, reach, t) if rot else None
        nb = -(-max(t, 1) // bs) + 2
        self.kc = rng.standard_normal((nb, hkv, bs, d)).astype(np.float16)
        self.vc = rng.standard_normal((nb, hkv, bs, d)).astype(np.float16)
        self.slots = rng.permutation(nb * bs)[:t].astype(np.int64)

    def gpu(self):
        def up(x):
            return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
        # the three as views of one buffer, tokens strided
        t, h, d = self.q.shape
        hkv = self.k.shape[1]
        fused = torch.zeros(t, (h + 2 * hkv) * d + 8, dtype=torch.float16, device="cuda")
        self.tq = fused[:, :h * d].view(t, h, d)
        self.tk = fused[:, h * d:(h + hkv) * d].view(t, hkv, d)
        self.tv = fused[:, (h + hkv) * d:(h + 2 * hkv) * d].view(t, hkv, d)
        for a, b in ((self.tq, self.q), (self.tk, self.k), (self.tv, self.v)):
            a.copy_(up(b))
        self.kw = dict(positions=up(self.pos), cos_sin=up(self.cs), query_weight=up(self.wq), key_weight=up(self.wk))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.tslots, self.tkc, self.tvc = up(self.slots), up(self.kc), up(self.vc)
        return self


SHAPES = [(1, 8, 8, 64, 64), (1, 1, 1, 8, 0), (7, 32, 8, 128, 128), (5, 4, 2, 128, 64), (3, 6, 2, 80, 32),
          (33, 3, 1, 96, 96), (9, 4, 4, 256, 64), (2, 5, 1, 256, 256), (300, 7, 1, 16, 16), (4, 2, 2, 24, 16),
          (1025, 16, 2, 64, 32), (70, 8, 8, 120, 112)]


@pytest.mark.parametrize("t,h,hkv,d,rot", SHAPES)
@pytest.mark.parametrize("norm", ["both", "query", "none"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_plain(pkv, t, h, hkv, d, rot, norm, interleaved):
    c = Case(1, t, h, hkv, d, rot, norm).gpu()
    qo, ko = torch.full_like(c.tq, 7.0), torch.full_like(c.tk, 7.0)
    pkv.qk_norm_rope(qo, ko, c.tq, c.tk, interleaved=interleaved, eps=1e-5, status=c.status, **c.kw)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    check(qo, c.q, c.wq, 1e-5, c.pos, c.cs, interleaved)
    check(ko, c.k, c.wk, 1e-5, c.pos, c.cs, interleaved)


@pytest.mark.parametrize("t,h,hkv,d,rot", SHAPES)
@pytest.mark.parametrize("bs", [8, 16, 128])
def test_into_the_cache(pkv, t, h, hkv, d, rot, bs):
    """Keys within the bound, values bit for bit, every other slot untouched,
    padding slots skipped."""
    c = Case(2, t, h, hkv, d, rot, bs=bs)
    c.slots[::5] = -1
    c.gpu()
    qo = torch.full_like(c.tq, 7.0)
    pkv.qk_norm_rope_and_cache(qo, c.tq, c.tk, c.tv, c.tkc, c.tvc, c.tslots, status=c.status, **c.kw)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    check(qo, c.q, c.wq, 1e-6, c.pos, c.cs, False)
    vc = c.vc.copy()
    OC.reshape_and_cache(c.v, c.v, np.zeros_like(vc), vc, c.slots)
    assert np.array_equal(bits16(c.tvc), bits16(vc))
    flat = c.tkc.transpose(1, 2).reshape(-1, hkv, d)
    rows = np.nonzero(c.slots >= 0)[0]
    got = torch.zeros_like(c.tk)
    got[rows] = flat[c.slots[rows]]
    check(got, c.k, c.wk, 1e-6, c.pos, c.cs, False, rows)
    other = np.setdiff1d(np.arange(flat.shape[0]), c.slots)
    before = c.kc.transpose(0, 2, 1, 3).reshape(-1, hkv, d)
    assert np.array_equal(bits16(flat)[other], bits16(before)[other])


@pytest.mark.parametrize("d,rot", [(128, 128), (80, 48), (256, 256)])
def test_in_place(pkv, d, rot):
    c = Case(3, 50, 6, 2, d, rot).gpu()
    pkv.qk_norm_rope(c.tq, c.tk, c.tq, c.tk, status=c.status, **c.kw)
    torch.cuda.synchronize()
    check(c.tq, c.q, c.wq, 1e-6, c.pos, c.cs, False)
    check(c.tk, c.k, c.wk, 1e-6, c.pos, c.cs, False)
    assert np.array_equal(bits16(c.tv), bits16(c.v))


def test_zero_heads_large_and_small_values(pkv):
    c = Case(4, 6, 4, 2, 64, 64)
    c.q[0], c.q[1], c.q[2] = 0.0, 65504.0, 6e-8
    c.k[0, 0], c.k[0, 1] = 0.0, 65504.0
    c.gpu()
    qo, ko = torch.empty_like(c.tq), torch.empty_like(c.tk)
    pkv.qk_norm_rope(qo, ko, c.tq, c.tk, **c.kw)
    check(qo, c.q, c.wq, 1e-6, c.pos, c.cs, False)
    check(ko, c.k, c.wk, 1e-6, c.pos, c.cs, False)
    assert (qo[0] == 0).all()


def test_a_head_that_is_not_finite_stays_alone(pkv):
    c = Case(5, 5, 4, 2, 128, 128).gpu()
    clean = torch.empty_like(c.tq)
    ko = torch.empty_like(c.tk)
    pkv.qk_norm_rope(clean, ko, c.tq, c.tk, **c.kw)
    c.tq[2, 1, 7] = float("inf")
    c.tq[3, 0, 0] = float("nan")
    got = torch.empty_like(c.tq)
    pkv.qk_norm_rope(got, ko, c.tq, c.tk, **c.kw)
    mask = torch.ones(5, 4, dtype=torch.bool, device="cuda")
    mask[2, 1] = mask[3, 0] = False
    assert torch.equal(got[mask], clean[mask])
    assert got[2, 1].isnan().any() and got[3, 0].isnan().all()


def test_far_positions(pkv):
    """The last row of a long table; the table is fp32, so the result is exact
    in what the table holds."""
    c = Case(6, 4, 2, 1, 128, 128, reach=200000)
    c.pos = np.array([0, 199999, 131072, 65537])
    c.gpu()
    qo, ko = torch.empty_like(c.tq), torch.empty_like(c.tk)
    pkv.qk_norm_rope(qo, ko, c.tq, c.tk, **c.kw)
    check(qo, c.q, c.wq, 1e-6, c.pos, c.cs, False)


def test_slots_far_into_a_large_pool(pkv):
    """Element offsets past 2^32 in each cache."""
    hkv, bs, d = 8, 16, 128
    nb = (1 << 32) // (hkv * bs * d) + 4
    c = Case(7, 40, 8, hkv, d, d).gpu()
    kc = torch.empty((nb, hkv, bs, d), dtype=torch.float16, device="cuda")
    vc = torch.empty_like(kc)
    first = nb * bs - 40
    slots = torch.arange(first, nb * bs, device="cuda")
    qo = torch.empty_like(c.tq)
    pkv.qk_norm_rope_and_cache(qo, c.tq, c.tk, c.tv, kc, vc, slots, status=c.status, **c.kw)
    got = kc[-4:].transpose(1, 2).reshape(-1, hkv, d)[-40:]
    check(got, c.k, c.wk, 1e-6, c.pos, c.cs, False)
    assert torch.equal(vc[-4:].transpose(1, 2).reshape(-1, hkv, d)[-40:], c.tv)
    assert int(c.status.item()) == 0


def test_bad_device_data_is_reported(pkv):
    """A position outside the table: nothing of that token is written.  A slot
    outside the pool: its key and value are not."""
    c = Case(8, 6, 4, 2, 64, 64).gpu()
    for bad in (-1, 5000, 1 << 40):
        c.status.zero_()
        pos = c.kw["positions"].clone()
        pos[2] = bad
        qo = torch.full_like(c.tq, 7.0)
        kc, vc = c.tkc.clone(), c.tvc.clone()
        pkv.qk_norm_rope_and_cache(qo, c.tq, c.tk, c.tv, kc, vc, c.tslots, status=c.status, **dict(c.kw, positions=pos))
        torch.cuda.synchronize()
        assert int(c.status.item()) == pkv.PKV_ERR_OUT_OF_RANGE
        assert (qo[2] == 7.0).all() and (qo[3] != 7.0).any()
        slot = int(c.slots[2])
        assert torch.equal(kc[slot // 16, :, slot % 16], c.tkc[slot // 16, :, slot % 16])
        assert torch.equal(vc[slot // 16, :, slot % 16], c.tvc[slot // 16, :, slot % 16])
    for bad in (c.kc.shape[0] * 16, 1 << 50):
        c.status.zero_()
        slots = c.tslots.clone()
        slots[1] = bad
        qo = torch.full_like(c.tq, 7.0)
        kc, vc = c.tkc.clone(), c.tvc.clone()
        pkv.qk_norm_rope_and_cache(qo, c.tq, c.tk, c.tv, kc, vc, slots, status=c.status, **c.kw)
        torch.cuda.synchronize()
        assert int(c.status.item()) == pkv.PKV_ERR_OUT_OF_RANGE
        check(qo, c.q, c.wq, 1e-6, c.pos, c.cs, False)
        slot = int(c.slots[1])
        assert torch.equal(kc[slot // 16, :, slot % 16], c.tkc[slot // 16, :, slot % 16])


def test_graph_and_other_stream(pkv):
    c = Case(9, 17, 8, 2, 128, 128).gpu()
    qo, ko = torch.empty_like(c.tq), torch.empty_like(c.tk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.qk_norm_rope(qo, ko, c.tq, c.tk, stream=side, **c.kw)
    side.synchronize()
    check(qo, c.q, c.wq, 1e-6, c.pos, c.cs, False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.qk_norm_rope(qo, ko, c.tq, c.tk, **c.kw)
    c.pos = (c.pos + 1234) % 5000
    c.kw["positions"].copy_(torch.from_numpy(c.pos))
    g.replay()
    torch.cuda.synchronize()
    check(qo, c.q, c.wq, 1e-6, c.pos, c.cs, False)
    check(ko, c.k, c.wk, 1e-6, c.pos, c.cs, False)


def test_no_tokens(pkv):
    c = Case(10, 0, 4, 2, 64, 64).gpu()
    pkv.qk_norm_rope(torch.empty_like(c.tq), torch.empty_like(c.tk), c.tq, c.tk, **c.kw)
    pkv.qk_norm_rope_and_cache(torch.empty_like(c.tq), c.tq, c.tk, c.tv, c.tkc, c.tvc, c.tslots, **c.kw)
