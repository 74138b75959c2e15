"""Key bounds, the choice of blocks and the path they are part of, on the GPU
against the fp64 oracle.  Bounds of an fp16 cache and the choice are exact;
bounds of an 8-bit cache are off by the rounding of the product to fp16."""

import numpy as np
import pytest
import torch

import test_gpu_q8 as G
from oracle import q8 as Q

pytestmark = pytest.mark.gpu
pkv = G.pkv


def pool(seed, kind, hkv, d, bs, lens, fill=1.0):
    """Keys [NB][Hkv][bs][D] (code values), scales, tables with -1 where unused."""
    rng = np.random.default_rng(seed)
    need = [-(-c // bs) for c in lens]
    nb = sum(need) + 2
    order = rng.permutation(nb)
    tables = np.full((len(lens), max(need + [0]) + 1), -1, np.int32)
    at = 0
    for s in range(len(lens)):
        tables[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
    if kind == "fp16":
        return rng, rng.standard_normal((nb, hkv, bs, d)).astype(np.float16).astype(np.float64) * fill, None, tables
    codes = Q.round_codes(rng.standard_normal((nb, hkv, bs, d)) * Q.TOP[kind] / 3, kind)
    return rng, codes, (np.exp(rng.standard_normal((nb, hkv))) / 50).astype(np.float32), tables


@pytest.mark.parametrize("kind", ["fp16", "int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
def test_bounds(pkv, bs, d, kind):
    lens = [1, bs, bs + 1, 3 * bs - 1, 5, 4 * bs + 3, 0, bs - 1]
    new = [1, bs, 1, bs + 2, 3, 4 * bs + 3, 0, 2]
    rng, keys, scale, tables = pool(1, kind, 3, d, bs, lens)
    before = rng.standard_normal((keys.shape[0], 3, 2, d)).astype(np.float16)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    got = torch.from_numpy(before).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = np.array(lens, np.int32)
    args = (G.to_gpu(keys, kind), torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda())
    key_scale = None if scale is None else torch.from_numpy(scale).cuda()
    pkv.block_key_bounds(got, *args, torch.from_numpy(starts).cuda(), int(starts[-1]), key_scale=key_scale,
                         status=status)
    ref = before.astype(np.float64)
    values = keys if scale is None else keys * scale.astype(np.float64)[:, :, None, None]
    Q.key_bounds(ref, values, tables, lens, starts)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = got.double().cpu().numpy()
    if kind == "fp16":
        assert np.array_equal(got, ref)
    else:  # one product in fp32, one rounding to fp16
        assert (np.abs(got - ref) <= np.abs(ref) * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25).all()


def test_bounds_one_token_each_and_out_of_range(pkv):
    """Without query_starts; NaN spreads; bad entries and contexts are reported."""
    lens = np.array([17, 0, 32, 5], np.int32)
    rng, keys, _, tables = pool(2, "fp16", 2, 128, 16, lens)
    keys[tables[2, 1], 1, 3, 7] = np.nan
    got = torch.zeros(keys.shape[0], 2, 2, 128, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache, tab, ln = G.to_gpu(keys, "fp16"), torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda()
    pkv.block_key_bounds(got, cache, tab, ln, status=status)
    ref = np.zeros(got.shape)
    Q.key_bounds(ref, keys, tables, lens, None)
    assert int(status.item()) == 0
    assert np.array_equal(got.double().cpu().numpy(), ref, equal_nan=True)
    assert torch.isnan(got[tables[2, 1], 1, :, 7]).all()
    tab[0, 1] = keys.shape[0]
    ln[3] = 1 << 20
    got.zero_()
    pkv.block_key_bounds(got, cache, tab, ln, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == pkv.PKV_ERR_OUT_OF_RANGE
    assert (got[tables[0, 1]] == 0).all()


def select(pkv, q, bounds, tables, lens, bs, keep, first, last, status=0, **kw):
    n, hkv = len(lens), bounds.shape[1]
    selected = torch.full((n, hkv, keep), -9, dtype=torch.int32, device="cuda")
    number = torch.full((n, hkv), -9, dtype=torch.int32, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.select_blocks(selected, number, torch.from_numpy(q).cuda(), torch.from_numpy(bounds).cuda(),
                      torch.from_numpy(np.asarray(tables, np.int32)).cuda(),
                      torch.from_numpy(np.asarray(lens, np.int32)).cuda(), bs, first_blocks=first, last_blocks=last,
                      status=word, **kw)
    torch.cuda.synchronize()
    assert int(word.item()) == status
    return selected.cpu().numpy(), number.cpu().numpy()


def make(seed, h, hkv, d, bs, lens, quantum=None):
    """Queries and bounds; with a quantum, values so coarse that scores tie."""
    rng = np.random.default_rng(seed)
    need = [-(-c // bs) for c in lens]
    nb = sum(need) + 2
    order = rng.permutation(nb)
    tables = np.full((len(lens), max(need + [0]) + 1), -1, np.int32)
    at = 0
    for s in range(len(lens)):
        tables[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
    q = rng.standard_normal((len(lens), h, d)) * 1.5
    mid, reach = rng.standard_normal((nb, hkv, 1, d)) * 0.7, np.abs(rng.standard_normal((nb, hkv, 2, d)) * 0.4 + 1.5)
    bounds = mid + reach * np.array([1, -1])[:, None]
    if quantum:
        q, bounds = np.round(q / quantum) * quantum, np.round(bounds / quantum) * quantum
    return q.astype(np.float16), bounds.astype(np.float16), tables, np.array(lens, np.int32)


def check(pkv, c, bs, keep, first, last, **kw):
    q, bounds, tables, lens = c
    got = select(pkv, q, bounds, tables, lens, bs, keep, first, last, **kw)
    ref = Q.select(q, bounds.astype(np.float64), tables, lens, bs, keep, first, last)
    assert np.array_equal(got[1], ref[1])
    assert np.array_equal(got[0], ref[0])


@pytest.mark.parametrize("h,hkv", [(1, 1), (4, 4), (4, 2), (7, 1), (8, 1), (9, 1), (16, 1), (12, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_select_head_layouts(pkv, h, hkv, d):
    check(pkv, make(1, h, hkv, d, 16, [1, 900, 0, 160, 177, 2000]), 16, 10, 1, 2)


@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("keep,first,last", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (7, 0, 0), (7, 3, 4), (7, 2, 2), (300, 5, 9)])
def test_select_sizes(pkv, bs, keep, first, last):
    lens = [1, bs, 7 * bs, 7 * bs + 1, 8 * bs, 100 * bs + 3, 299 * bs, 301 * bs - 1, 700 * bs]
    check(pkv, make(2, 2, 1, 64, bs, lens), bs, keep, first, last)


@pytest.mark.parametrize("quantum", [1.0, 0.5, 0.125])
@pytest.mark.parametrize("keep", [1, 20, 150])
def test_select_ties(pkv, quantum, keep):
    """Coarse values: many equal scores, the lowest index wins."""
    check(pkv, make(3, 4, 2, 64, 8, [8 * 400, 8 * 31, 8 * 1200], quantum), 8, keep, 0, 1)


@pytest.mark.parametrize("blocks", [300, 3000, 9000])
def test_select_among_equals(pkv, blocks):
    """All bounds alike but a few: more about the border than are ranked in one
    step, and more blocks than fit in shared memory."""
    q, bounds, tables, lens = make(4, 2, 1, 64, 8, [8 * blocks, 8 * blocks - 3])
    bounds[:] = bounds[0]
    for i in (3, 77, 200):
        bounds[tables[0, i]] = bounds[0] + np.float16(0.25) * np.array([1, -1], np.float16)[:, None]
        bounds[tables[1, i + 5]] = bounds[0] - np.float16(0.25) * np.array([1, -1], np.float16)[:, None]
    check(pkv, (q, bounds, tables, lens), 8, 128, 1, 2)


def test_select_by_the_last_bit(pkv):
    """Blocks whose scores differ by less than fp32 holds."""
    q, bounds, tables, lens = make(5, 1, 1, 64, 8, [8 * 200])
    bounds[:] = bounds[0]
    q[0, 0, :2] = [1000.0, 2.0 ** -14]
    rng = np.random.default_rng(5)
    order = rng.permutation(200)
    for rank, b in enumerate(order):  # the second channel decides, by steps of 2^-24 and less of the score
        bounds[tables[0, b], 0, 0, 1] = np.float16(3.0 + rank / 512)
    check(pkv, (q, bounds, tables, lens), 8, 50, 0, 0)


def test_select_values_that_are_not_finite(pkv):
    q, bounds, tables, lens = make(6, 4, 1, 64, 16, [16 * 90, 16 * 50])
    bounds[tables[0, 17], 0, 0, 5] = np.nan
    bounds[tables[0, 33], 0, 1, 9] = -np.inf
    bounds[tables[0, 71], 0, 0, 0] = np.inf
    check(pkv, (q, bounds, tables, lens), 16, 9, 1, 2)
    check(pkv, (q, bounds, tables, lens), 16, 2, 0, 0)
    q[1, 2, 3] = np.nan
    check(pkv, (q, bounds, tables, lens), 16, 9, 1, 2)
    bounds[...] = np.inf
    check(pkv, (q, bounds, tables, lens), 16, 9, 1, 2)


def test_select_extreme_values(pkv):
    """The largest and the smallest fp16 values, and zeros."""
    for size in (40000.0, 2.0 ** -22, 0.0):
        q, bounds, tables, lens = make(7, 2, 2, 128, 16, [16 * 300])
        q = (np.sign(q) * size).astype(np.float16)
        bounds = (bounds.astype(np.float64) * size / 4).astype(np.float16)
        check(pkv, (q, bounds, tables, lens), 16, 40, 1, 1)


def test_select_out_of_range(pkv):
    q, bounds, tables, lens = make(8, 2, 1, 64, 16, [16 * 30, 16 * 20, 16 * 9])
    bad = tables.copy()
    bad[0, 3], bad[1, 7] = bounds.shape[0], -2
    ref_tables = tables.copy()
    ref_tables[0, 3] = ref_tables[1, 7] = 0
    lens2 = np.array([16 * 30, 16 * 20, -4], np.int32)
    got = select(pkv, q, bounds, bad, lens2, 16, 6, 1, 1, status=pkv.PKV_ERR_OUT_OF_RANGE)
    ref = Q.select(q, bounds.astype(np.float64), ref_tables, np.maximum(lens2, 0), 16, 6, 1, 1)
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])
    with pytest.raises(pkv.PkvError):
        select(pkv, q, bounds, tables, lens, 16, 2, 1, 2)


def test_select_workspace_stream_and_graph(pkv):
    q, bounds, tables, lens = make(9, 4, 2, 128, 16, [16 * 300 + 5, 40])
    ws = pkv.new_select_workspace(2, 2, tables.shape[1])
    ws.fill_(0x7f)
    stream = torch.cuda.Stream()
    for kw in (dict(workspace=ws), dict(stream=stream)):
        stream.wait_stream(torch.cuda.current_stream())
        check(pkv, (q, bounds, tables, lens), 16, 20, 1, 2, **kw)
    t = [torch.from_numpy(x).cuda() for x in (q, bounds, tables, lens)]
    selected = torch.zeros(2, 2, 20, dtype=torch.int32, device="cuda")
    number = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pkv.select_blocks(selected, number, *t, 16, workspace=ws)
    for seed in range(3):
        q = (np.random.default_rng(seed).standard_normal(q.shape) * 2).astype(np.float16)
        t[0].copy_(torch.from_numpy(q))
        graph.replay()
        ref = Q.select(q, bounds.astype(np.float64), tables, lens, 16, 20, 1, 2)
        assert np.array_equal(selected.cpu().numpy(), ref[0]) and np.array_equal(number.cpu().numpy(), ref[1])


@pytest.mark.parametrize("kind", ["fp16", "int8", "e4m3"])
def test_the_path_step_by_step(pkv, kind):
    """Prompts, then tokens one by one, through the block manager: write, bounds,
    choice, decode over the choice; with a fork that copies on write.  Every part
    against the oracle's from the parts before."""
    h, hkv, d, bs, keep = 8, 2, 64, 16, 5
    rng = np.random.default_rng(31)
    nb = 64
    alloc = pkv.BlockAllocator(nb, bs)
    seqs = [alloc.new_seq() for _ in range(3)]
    lens = [150, 33, 16]
    dtype = G.DTYPE[kind]
    kc, vc = (torch.zeros(nb, hkv, bs, d, device="cuda").to(dtype) for _ in range(2))
    scales = [torch.zeros(nb, 4, device="cuda") for _ in range(2)]  # copy_blocks takes multiples of 16 bytes
    bounds = torch.zeros(nb, hkv, 2, d, dtype=torch.float16, device="cuda")
    o_codes = [np.zeros((nb, hkv, bs, d)) for _ in range(2)]
    o_scales = [np.zeros((nb, hkv)) for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for s, n in zip(seqs, lens):
        alloc.append_tokens(s, n)
    new = list(lens)
    for step in range(6):
        if step == 3:
            seqs.append(alloc.fork(seqs[0]))
        if step > 0:
            slots, pairs = alloc.append_batch(seqs)
            if len(pairs):
                p = torch.from_numpy(np.asarray(pairs, np.int64).reshape(-1, 2)).cuda()
                pkv.copy_blocks(kc, vc, p, status=status)
                pkv.copy_blocks(scales[0], scales[1], p, status=status)
                for src, dst in np.asarray(pairs).reshape(-1, 2):
                    for x in o_codes + o_scales:
                        x[dst] = x[src]
            new = [1] * len(seqs)
        tables, ln = alloc.export(seqs, 16)
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        rows = [rng.standard_normal((int(starts[-1]), hkv, d)).astype(np.float16) * np.float16(1 + step / 3) for _ in range(2)]
        q = (rng.standard_normal((len(seqs), h, d)) * 1.5).astype(np.float16)
        g_rows = [torch.from_numpy(x).cuda() for x in rows]
        g_tables, g_lens = torch.from_numpy(tables).cuda(), torch.from_numpy(ln).cuda()
        g_starts = torch.from_numpy(starts).cuda() if step == 0 else None
        g_scales = [x[:, :hkv] for x in scales]
        if kind == "fp16":
            slots = [int(tables[s][p // bs]) * bs + p % bs for s in range(len(seqs)) for p in range(ln[s] - new[s], ln[s])]
            pkv.reshape_and_cache(g_rows[0], g_rows[1], kc, vc, torch.tensor(slots, device="cuda"), status=status)
            for x, codes in zip(rows, o_codes):
                for row, slot in zip(x, slots):
                    codes[slot // bs, :, slot % bs] = row
            values = o_codes
        else:
            pkv.reshape_and_cache_q8(g_rows[0], g_rows[1], kc, vc, g_scales[0], g_scales[1], g_tables, g_lens, g_starts,
                                     status=status)
            for codes, scale, x in zip(o_codes, o_scales, rows):
                Q.write(codes, scale, x, tables, ln, starts, kind)
            values = [c * s[:, :, None, None] for c, s in zip(o_codes, o_scales)]
            for cache, codes in zip((kc, vc), o_codes):
                assert np.array_equal(G.from_gpu(cache), codes)
        pkv.block_key_bounds(bounds, kc, g_tables, g_lens, g_starts, int(starts[-1]) if step == 0 else None,
                             key_scale=None if kind == "fp16" else g_scales[0], status=status)
        selected = torch.zeros(len(seqs), hkv, keep, dtype=torch.int32, device="cuda")
        number = torch.zeros(len(seqs), hkv, dtype=torch.int32, device="cuda")
        pkv.select_blocks(selected, number, torch.from_numpy(q).cuda(), bounds, g_tables, g_lens, bs, status=status)
        out = torch.empty(len(seqs), h, d, dtype=torch.float16, device="cuda")
        g_q = torch.from_numpy(q).cuda()
        if kind == "fp16":
            pkv.paged_attention_decode_selected(out, g_q, kc, vc, g_tables, g_lens, selected, number, 0.125, status=status)
        else:
            pkv.paged_attention_decode_q8(out, g_q, kc, vc, *g_scales, g_tables, g_lens, 0.125, selected=selected,
                                          num_selected=number, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        held = bounds.double().cpu().numpy()
        for s in range(len(seqs)):  # every block's bounds are those of its keys
            for b in range(-(-int(ln[s]) // bs)):
                keys = values[0][tables[s][b], :, :min(bs, int(ln[s]) - b * bs)]
                for k, ref in enumerate((keys.max(axis=1), keys.min(axis=1))):
                    assert (np.abs(held[tables[s][b], :, k] - ref) <= np.abs(ref) * 2.0 ** -10 + 2.0 ** -25).all()
        ref, count = Q.select(q, held, tables, ln, bs, keep, 1, 2)
        assert np.array_equal(selected.cpu().numpy(), ref) and np.array_equal(number.cpu().numpy(), count)
        lists = [[ref[s, k, :count[s, k]].tolist() for k in range(hkv)] for s in range(len(seqs))]
        expect, spread, reach, seen, top = Q.decode(q, values[0], values[1], tables, ln, 0.125, lists)
        got = out.double().cpu().numpy()
        more = G.biased(q, o_scales[0], tables, ln, bs, 0.125) if kind == "int8" else 0.0
        assert (np.abs(got - expect) <= G.bound(expect, spread, reach, seen, top, d, 4, more)).all()


@pytest.mark.parametrize("kind", ["int8", "fp16"])
def test_the_path_past_32_bits(pkv, kind):
    """Write, bounds, choice and decode in blocks whose codes and bounds lie past
    2^32 bytes: the bits of the same blocks in a small pool."""
    h, hkv, d, bs, keep = 8, 8, 128, 8, 9
    rng = np.random.default_rng(32)
    lens, dtype = [150, 33, 8], G.DTYPE[kind]
    tables = np.full((3, 20), -1, np.int32)
    order = rng.permutation(40)
    at = 0
    for s, n in enumerate(lens):
        m = -(-n // bs)
        tables[s, :m] = order[at:at + m]
        at += m
    rows = [torch.from_numpy(rng.standard_normal((sum(lens), hkv, d)).astype(np.float16)).cuda() for _ in range(2)]
    q = torch.from_numpy(rng.standard_normal((3, h, d)).astype(np.float16)).cuda()
    g_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda")

    def path(first):
        nb = first + 40
        kc, vc = (torch.empty(nb, hkv, bs, d, device="cuda", dtype=dtype) for _ in range(2))
        kc[first:], vc[first:] = 0, 0
        ks, vs = (torch.zeros(nb, hkv, device="cuda") for _ in range(2))
        bounds = torch.empty(nb, hkv, 2, d, dtype=torch.float16, device="cuda")
        bounds[first:] = 0
        g_tables = torch.from_numpy(np.where(tables < 0, -1, tables + first).astype(np.int32)).cuda()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        if kind == "fp16":
            slots = [(int(tables[s][p // bs]) + first) * bs + p % bs for s in range(3) for p in range(lens[s])]
            pkv.reshape_and_cache(*rows, kc, vc, torch.tensor(slots, device="cuda"), status=status)
        else:
            pkv.reshape_and_cache_q8(*rows, kc, vc, ks, vs, g_tables, g_lens, starts, status=status)
        pkv.block_key_bounds(bounds, kc, g_tables, g_lens, starts, sum(lens), key_scale=None if kind == "fp16" else ks,
                             status=status)
        selected = torch.zeros(3, hkv, keep, dtype=torch.int32, device="cuda")
        number = torch.zeros(3, hkv, dtype=torch.int32, device="cuda")
        pkv.select_blocks(selected, number, q, bounds, g_tables, g_lens, bs, status=status)
        out = torch.empty_like(q)
        if kind == "fp16":
            pkv.paged_attention_decode_selected(out, q, kc, vc, g_tables, g_lens, selected, number, 0.125, status=status)
        else:
            pkv.paged_attention_decode_q8(out, q, kc, vc, ks, vs, g_tables, g_lens, 0.125, selected=selected,
                                          num_selected=number, status=status)
        assert int(status.item()) == 0
        return [x[first:].clone().view(torch.uint8) for x in (kc, vc, ks, vs, bounds)] + [selected, number, out]

    for near, far in zip(path(0), path((1 << 20) + 24)):
        assert torch.equal(near, far)
