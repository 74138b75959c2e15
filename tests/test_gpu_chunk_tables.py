"""GPU checks of the chunk attention with block tables far wider than the
contexts, as a server keeps them: the work split then computes in 64 bits."""

import numpy as np
import pytest
import torch

from test_gpu_chunk import Case

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


def fits_32(c, hkv, group, positions):
    """The split's rule, from its description: items times the table's length
    plus 256 times KV heads below 2^29."""
    items = c.rows // (2 * (128 // group)) + len(c.lens)
    return items < (1 << 29) // (positions + 256) // hkv


SEQS = [(1, 900), (70, 500), (200, 210), (5, 1300), (0, 40), (30, 20), (1, 1), (300, 2300)]


@pytest.mark.parametrize("h,hkv,d,bs,columns", [(8, 2, 128, 128, 1 << 18), (4, 4, 64, 16, 1 << 21),
                                                (16, 1, 128, 64, 1 << 21)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 90), (True, 1000), (False, 0)])
def test_wide_tables(pkv, h, hkv, d, bs, columns, causal, window):
    """The same bits as with narrow tables, which the oracle is compared with:
    the split depends on the lengths alone."""
    c = Case(40, h, hkv, d, bs, SEQS, causal=causal, window=window, before=1, behind=2).gpu()
    expect = c.oracle()
    narrow = c.t["tables"]
    wide = torch.full((len(SEQS), columns), -1, dtype=torch.int32, device="cuda")
    wide[:, :narrow.shape[1]] = narrow
    assert fits_32(c, hkv, h // hkv, narrow.shape[1] * bs) and not fits_32(c, hkv, h // hkv, columns * bs)
    for num_ctas in (0, 1, 5, 40, 601):
        c.t["tables"] = narrow
        small = c.call(pkv, out=torch.full_like(c.out, -77.0), num_ctas=num_ctas)
        c.check(small, expect)
        c.t["tables"] = wide
        large = c.call(pkv, out=torch.full_like(c.out, -77.0), num_ctas=num_ctas)
        torch.cuda.synchronize()
        assert torch.equal(small, large) and int(c.status.item()) == 0


def test_many_sequences_and_wide_tables(pkv):
    """Runs of several sequences per thread, found again unit by unit."""
    rng = np.random.default_rng(41)
    seqs = [(int(n), int(n + x)) for n, x in zip(rng.integers(0, 4, 1500), rng.integers(0, 60, 1500))]
    c = Case(41, 2, 2, 64, 8, seqs).gpu()
    assert not fits_32(c, 2, 1, (1 << 15) * 8)
    small = c.call(pkv)
    c.check(small)
    wide = torch.full((len(seqs), 1 << 15), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.t["tables"].shape[1]] = c.t["tables"]
    c.t["tables"] = wide
    large = c.call(pkv, out=torch.full_like(c.out, -77.0))
    torch.cuda.synchronize()
    assert torch.equal(small, large) and int(c.status.item()) == 0
