"""What the 8-bit cache's and the selected blocks' calls report, and what they
leave alone."""

import numpy as np
import pytest
import torch

import test_gpu_q8 as G
import test_gpu_select as S

pytestmark = pytest.mark.gpu
pkv = G.pkv

# of three sequences' rows, 140 in all
DECREASING = ([0, 100, 10, 140], [0, 30, 29, 140], [90, 140, 0, 140], [0, 140, 140, 2], [140, 80, 20, 0], [0, 139, 0, 0],
              [140, 140, 0, 0])


@pytest.mark.parametrize("starts", DECREASING)
def test_query_starts_that_decrease(pkv, starts):
    """Reported by the write and by the bounds, and no block outside the tables is touched."""
    for kind in G.EIGHT:
        w = G.Write(28, kind, 2, 64, 16, [150, 145, 141], [50, 50, 40]).gpu()
        w.t["starts"].copy_(torch.tensor(starts, dtype=torch.int32))
        w.call(pkv)
        torch.cuda.synchronize()
        assert int(w.status.item()) == pkv.PKV_ERR_OUT_OF_RANGE
        outside = np.setdiff1d(np.arange(w.codes[0].shape[0]), w.tables[w.tables >= 0])
        assert len(outside)
        for codes, scale, cache, gpu_scale in zip(w.codes, w.scales, (w.t["kc"], w.t["vc"]), (w.t["ks"], w.t["vs"])):
            assert np.array_equal(G.from_gpu(cache)[outside], codes[outside])
            assert np.array_equal(gpu_scale.cpu().numpy()[outside], scale[outside])
        bounds = torch.full((w.codes[0].shape[0], 2, 2, 64), 7.0, dtype=torch.float16, device="cuda")
        w.status.zero_()
        pkv.block_key_bounds(bounds, w.t["kc"], w.t["tables"], w.t["lens"], w.t["starts"], 140, key_scale=w.t["ks"],
                             status=w.status)
        torch.cuda.synchronize()
        assert int(w.status.item()) == pkv.PKV_ERR_OUT_OF_RANGE
        assert bool((bounds[torch.from_numpy(outside).cuda()] == 7).all())


def test_query_starts_in_order_are_not_reported(pkv):
    """Rows before the first and behind the last, sequences without rows, many sequences."""
    for n in (1, 3, 700, 4096):
        rng = np.random.default_rng(n)
        new = rng.integers(0, 4, n)
        w = G.Write(29, "int8", 1, 64, 8, [int(x) + int(y) for x, y in zip(new, rng.integers(0, 9, n))],
                    [int(x) for x in new], before=3, behind=2).gpu()
        w.call(pkv)
        w.check()


@pytest.mark.parametrize("kind", G.ALL)
@pytest.mark.parametrize("count", [1, -1, 9])
@pytest.mark.parametrize("where", [(1, 0), (1, 2), (3, 1)])
def test_lists_of_empty_contexts(pkv, kind, count, where):
    """Entries that count where the context has no block are one too many; the
    output is zeros."""
    c = G.Case(9, kind, 6, 3, 64, 16, [100, 0, 50, 0]).pick(3).gpu()
    c.check(c.call(pkv))
    c.t["number"][where] = count
    c.check(c.call(pkv), status=pkv.PKV_ERR_OUT_OF_RANGE)
    assert bool((c.out[1] == 0).all()) and bool((c.out[3] == 0).all())
    c.status.zero_()
    c.t["number"][where] = 0
    c.t["lens"][0] = -3
    c.lens = np.array([0, 0, 50, 0], np.int32)
    c.t["number"][0] = 0
    c.lists[0] = [[], [], []]
    c.check(c.call(pkv), status=pkv.PKV_ERR_OUT_OF_RANGE)


def test_the_longest_list(pkv):
    """max_selected 2^31 - 1, where an index that goes on by a CTA's threads passes 31 bits."""
    keep = (1 << 31) - 1
    c = G.Case(19, "fp16", 4, 1, 64, 16, [100]).pick(7).gpu()
    selected = torch.full((1, 1, keep), 5, dtype=torch.int32, device="cuda")
    number = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    bounds = torch.zeros(c.pools[0].shape[0], 1, 2, 64, dtype=torch.float16, device="cuda")
    pkv.select_blocks(selected, number, c.t["q"], bounds, c.t["tables"], c.t["lens"], 16, status=c.status)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0 and int(number.item()) == 7
    assert selected[0, 0, :7].tolist() == list(range(7))
    assert int(selected[0, 0, 7:].amax().item()) == -1 and int(selected[0, 0, 7:].amin().item()) == -1
    c.t["selected"], c.t["number"] = selected, number
    c.lists = [[list(range(7))]]
    c.check(c.call(pkv))


def test_numbers_past_32_bits_are_refused(pkv):
    """An argument that does not fit the library's 32 bits is not taken for the
    part of it that does."""
    far = 1 << 32
    q, bounds, tables, lens = S.make(1, 2, 1, 64, 16, [16 * 30, 16 * 20])
    t = [torch.from_numpy(x).cuda() for x in (q, bounds, tables, lens)]
    selected = torch.full((2, 1, 6), -9, dtype=torch.int32, device="cuda")
    number = torch.full((2, 1), -9, dtype=torch.int32, device="cuda")
    for bad in (dict(first_blocks=far + 1), dict(last_blocks=far), dict(first_blocks=-far), dict(block_size=far + 16)):
        kw = dict(block_size=16, first_blocks=1, last_blocks=2)
        kw.update(bad)
        with pytest.raises((ValueError, OverflowError, pkv.PkvError)):
            pkv.select_blocks(selected, number, *t, **kw)
    torch.cuda.synchronize()
    assert bool((selected == -9).all())
    w = G.Write(26, "int8", 2, 64, 16, [40, 20], [30, 20]).gpu()
    out = torch.full((w.codes[0].shape[0], 2, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    with pytest.raises((ValueError, OverflowError, pkv.PkvError)):
        pkv.block_key_bounds(out, w.t["kc"], w.t["tables"], w.t["lens"], w.t["starts"], far + 5, key_scale=w.t["ks"])
    torch.cuda.synchronize()
    assert bool((out == 7).all())
    c = G.Case(9, "fp16", 4, 2, 64, 16, [100, 50]).pick(3).gpu()
    with pytest.raises((ValueError, OverflowError, pkv.PkvError)):
        c.call(pkv, num_ctas=far + 3)
