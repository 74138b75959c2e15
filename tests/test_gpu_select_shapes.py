"""The choice of blocks over every way that its work is laid out: few and many
(sequence, KV head) pairs, clusters of one to eight CTAs, tables much wider than
the contexts and past what one CTA's shared memory holds; and the decode, the
write and the bounds with wide tables."""

import numpy as np
import pytest
import torch

import test_gpu_q8 as G
import test_gpu_select as S

pytestmark = pytest.mark.gpu
pkv = G.pkv


def choose(q, bounds, tables, lens, bs, keep, first, last):
    """The definition in 64 bits, for inputs without ties."""
    n, hkv = len(lens), bounds.shape[1]
    group = q.shape[1] // hkv
    selected, number = np.full((n, hkv, keep), -1, np.int64), np.zeros((n, hkv), np.int64)
    q = q.astype(np.float64)
    for s in range(n):
        blocks = -(-int(lens[s]) // bs)
        b = bounds[tables[s, :blocks]].astype(np.float64)
        for k in range(hkv):
            h = q[s, k * group:(k + 1) * group]
            score = (np.maximum(h, 0) @ b[:, k, 0].T + np.minimum(h, 0) @ b[:, k, 1].T).max(axis=0) if blocks else []
            if blocks <= keep:
                kept = np.arange(blocks)
            else:
                middle = np.arange(first, blocks - last)
                need = keep - first - last
                ranked = middle[np.argsort(-score[middle], kind="stable")]
                if 0 < need:  # rounding does not decide
                    assert score[ranked[need - 1]] - score[ranked[need]] > 1e-9
                kept = np.sort(np.concatenate([np.arange(first), ranked[:need], np.arange(blocks - last, blocks)]))
            selected[s, k, :len(kept)], number[s, k] = kept, len(kept)
    return selected, number


def check(pkv, c, bs, keep, first, last, columns=0, poison=-1):
    q, bounds, tables, lens = c
    wide = np.concatenate([tables, np.full((len(tables), columns), poison, np.int32)], axis=1)
    got = S.select(pkv, q, bounds, wide, lens, bs, keep, first, last)
    ref = choose(q, bounds, tables, lens, bs, keep, first, last)
    assert np.array_equal(got[1], ref[1]) and np.array_equal(got[0], ref[0])


@pytest.mark.parametrize("group", [1, 4, 8, 9, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_more_blocks_than_the_first_kernel_holds(pkv, d, group):
    """About 5000 blocks with scores of their own, beside short contexts."""
    lens = [8 * 5000 - 3, 8 * 4097, 8 * 900, 5, 0, 8 * 40, 8 * 41]
    c = S.make(1, 2 * group, 2, d, 8, lens)
    check(pkv, c, 8, 40, 1, 2)
    check(pkv, c, 8, 700, 3, 0)


@pytest.mark.parametrize("columns", [513, 1025, 2049, 4097, 9000, 70000])
@pytest.mark.parametrize("d,h,hkv", [(64, 2, 2), (128, 8, 2), (128, 16, 1)])
def test_tables_much_wider_than_the_contexts(pkv, d, h, hkv, columns):
    c = S.make(2, h, hkv, d, 16, [16 * 300, 1, 16 * 77 + 5, 16 * 12, 0])
    check(pkv, c, 16, 12, 1, 2, columns)
    check(pkv, c, 16, 64, 0, 0, columns, poison=1 << 30)


# a segment is a sequence and KV head: 80, 200 and 700 of them
@pytest.mark.parametrize("n,hkv", [(10, 8), (80, 1), (25, 8), (200, 1), (88, 8), (700, 1)])
@pytest.mark.parametrize("group,d", [(1, 64), (4, 128), (12, 128)])
def test_many_segments(pkv, n, hkv, group, d):
    rng = np.random.default_rng(n)
    blocks = rng.integers(100, 700, n)
    blocks[0], blocks[n // 2] = 0, 3
    c = S.make(3, group * hkv, hkv, d, 8, [int(8 * x - r) if x else 0 for x, r in zip(blocks, rng.integers(0, 8, n))])
    check(pkv, c, 8, 50, 2, 3)


@pytest.mark.parametrize("blocks", [200, 700, 1500, 3900, 4600])
@pytest.mark.parametrize("d", [64, 128])
def test_hundreds_of_unequal_scores_at_the_border(pkv, d, blocks):
    """One outlier channel makes the fp32 scores' error bound wider than the scores
    lie apart, so that most blocks are scored again."""
    c = S.make(4, 4, 1, d, 8, [8 * blocks, 8 * (blocks // 3)])
    c[0][:, :, 7] = 3.0
    c[1][:, :, :, 7] = 30000.0
    for keep in (20, 150, blocks // 2):
        check(pkv, c, 8, keep, 1, 2)


@pytest.mark.parametrize("kind", G.ALL)
@pytest.mark.parametrize("columns", [1, 300, 5000])
def test_the_other_calls_with_wide_tables(pkv, kind, columns):
    """Decode, write and bounds: the same however wide the table is."""
    c = G.Case(5, kind, 8, 2, 128, 16, [300, 0, 77, 1], columns=columns)
    if kind == "fp16":
        c.pick(6)
    c.gpu()
    c.check(c.call(pkv))
    if kind == "fp16":
        return
    w = G.Write(6, kind, 2, 128, 16, [300, 77, 1], [40, 77, 1])
    w.tables = np.concatenate([w.tables, np.full((3, columns), -1, np.int32)], axis=1)
    w.gpu()
    w.call(pkv)
    w.check()
    bounds = torch.zeros(w.codes[0].shape[0], 2, 2, 128, dtype=torch.float16, device="cuda")
    pkv.block_key_bounds(bounds, w.t["kc"], w.t["tables"], w.t["lens"], w.t["starts"], 118, key_scale=w.t["ks"],
                         status=w.status)
    ref = np.zeros(bounds.shape)
    G.Q.key_bounds(ref, w.codes[0] * w.scales[0].astype(np.float64)[:, :, None, None], w.tables, w.lens, w.starts)
    torch.cuda.synchronize()
    assert int(w.status.item()) == 0
    assert (np.abs(bounds.double().cpu().numpy() - ref) <= np.abs(ref) * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25).all()


@pytest.mark.parametrize("kind", G.ALL)
def test_bounds_of_moved_blocks(pkv, kind):
    """Blocks swapped out, and in again to other places: their bounds go along as
    a pool of their own, or are made anew from query_starts over the whole contexts."""
    hkv, d, bs, lens = 2, 64, 16, [100, 16, 49]
    rng, keys, scale, tables = S.pool(7, kind, hkv, d, bs, lens)
    nb = keys.shape[0]
    cache = [G.to_gpu(keys, kind) for _ in range(2)]
    scales = [torch.zeros(nb, 4, device="cuda") for _ in range(2)]
    if scale is not None:
        for x in scales:
            x[:, :hkv] = torch.from_numpy(scale).cuda()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda")
    key_scale = None if scale is None else scales[0][:, :hkv]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def build(table):
        out = torch.zeros(nb, hkv, 2, d, dtype=torch.float16, device="cuda")
        pkv.block_key_bounds(out, cache[0], torch.from_numpy(table).cuda(), ln, starts, sum(lens), key_scale=key_scale,
                             status=status)
        return out

    # two layers' bounds, which one call moves as it does keys and values
    bounds = [build(tables), build(tables) * 2]
    used = [int(b) for b in tables[tables >= 0]]
    pools = [cache, scales, bounds]
    host = [[torch.zeros_like(x, device="cpu").pin_memory() for x in pair] for pair in pools]
    out = torch.tensor([[b, i] for i, b in enumerate(used)], device="cuda")
    for pair, h in zip(pools, host):
        pkv.swap_blocks(*pair, *h, out, status=status)
    torch.cuda.synchronize()
    for pair in pools:
        for x in pair:
            x.view(torch.uint8).fill_(0x33)
    order = rng.permutation(nb)[:len(used)]
    back = torch.tensor([[i, int(order[i])] for i in range(len(used))], device="cuda")
    for pair, h in zip(pools, host):
        pkv.swap_blocks(*h, *pair, back, status=status)
    moved = tables.copy()
    for i, b in enumerate(used):
        moved[tables == b] = order[i]
    again = build(moved)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    at = torch.from_numpy(order.astype(np.int64)).cuda()
    assert torch.equal(again[at], bounds[0][at]) and torch.equal(again[at] * 2, bounds[1][at])
    q = torch.from_numpy(rng.standard_normal((3, 4, d)).astype(np.float16)).cuda()
    found = []
    for x in (bounds[0], again):
        selected = torch.zeros(3, hkv, 3, dtype=torch.int32, device="cuda")
        number = torch.zeros(3, hkv, dtype=torch.int32, device="cuda")
        pkv.select_blocks(selected, number, q, x, torch.from_numpy(moved).cuda(), ln, bs, status=status)
        found.append((selected, number))
    assert torch.equal(found[0][0], found[1][0]) and torch.equal(found[0][1], found[1][1])
    assert int(status.item()) == 0
