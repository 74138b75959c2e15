"""The 8-bit cache on the GPU against the fp64 oracle: the write's codes and
scales bit for bit, the decode (whole contexts and block lists, fp16 caches
too) within the roundings it makes.

Tolerance of the decode, per output element, with the codes and scales as given:

* the output's rounding to fp16: 2^-11 |out|, 2^-25 below the normal range;
* each weight's rounding to two fp16 terms: 2^-22 of it, together 2^-22 sum_t w_t
  |v_t|; weights are stored times 2^15, where 1 is at most that of the largest score
  with twice the largest value scale, so where the second term is below fp16's
  normal range it is off by at most 2^-25 of 2^15: count * 2^-40 * 2 times the
  largest |v| of any channel (some block's largest element times its scale);
* scores: a product of D terms in fp32 is off by at most D 2^-24 of the terms'
  magnitudes, doubled because tensor cores may cut instead of round; the score's
  factor, the reference's subtraction and the places between, at most 12
  roundings of numbers up to 1.45 of the score's size (log2 units); ex2 and the
  factors of a maximum that rises, 2^-22 each, at most 16 of them: 2^-18.  A
  score off by x moves a weight by e^x, in the numerator and the sum.  The
  products hold an int8 code as code + 128, and 128 times the queries' sum is
  taken off, so their terms' magnitudes count |code| + 256;
* sums in fp32, at most 2^-22 of the magnitudes' sum per step (an instruction
  adds 16 products, each cut at 2^-23 or finer of the largest): a step of 16 rows
  for each of 4 warps, and two dozen joins.
"""

import numpy as np
import pytest
import torch

from oracle import q8 as Q

pytestmark = pytest.mark.gpu

DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "fp16": torch.float16}


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from paged_kv_cache_152_gb300 import build
    build.build()
    import paged_kv_cache_152_gb300 as m
    m.load()
    return m


def bound(ref, spread, reach, count, top, d, warps=4, reach8=0.0):
    """reach8: what int8's 256 steps of the scale add to the terms' magnitudes in the scores."""
    score = (2 * d * (reach + reach8) + 12 * 1.45 * reach) * 2.0 ** -24 + 2.0 ** -18
    sums = (count / 16 / warps + 24) * 2.0 ** -22
    return (2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2.0 ** -22 * spread + (2 * score + sums)[..., None] * spread +
            count[..., None] * 2.0 ** -39 * top.max(axis=-1, keepdims=True))


def biased(q, scale, tables, lens, bs, softmax_scale):
    """reach8 [N][H] of an int8 cache with these key scales."""
    group = q.shape[1] // scale.shape[1]
    reach = np.zeros(q.shape[:2])
    for s in range(len(lens)):
        blocks = tables[s][:-(-int(lens[s]) // bs)]
        if len(blocks):
            largest = np.repeat(scale[blocks].max(axis=0), group)
            reach[s] = softmax_scale * 256 * largest * np.abs(q[s].astype(np.float64)).sum(axis=1)
    return reach


def to_gpu(codes, kind):
    """Code values (fp64) as a cache on the GPU."""
    if kind == "fp16":
        return torch.from_numpy(codes.astype(np.float16)).cuda()
    return torch.from_numpy(codes).float().to(DTYPE[kind]).cuda()


def from_gpu(cache):
    return cache.cpu().to(torch.float32).double().numpy()


class Case:
    """Sequences over shuffled blocks.  Positions behind a context hold NaN (fp16,
    e4m3) or 127 with a scale that would show; unused table entries are -1."""

    def __init__(self, seed, kind, h, hkv, d, bs, lens, columns=1, q_std=1.5, spread=0.5):
        rng = self.rng = np.random.default_rng(seed)
        self.kind, self.d, self.bs, self.scale = kind, d, bs, d ** -0.5
        self.lens = np.array(lens, np.int32)
        need = [-(-int(c) // bs) for c in lens]
        nb = sum(need) + 3
        order = rng.permutation(nb)
        self.tables = np.full((len(lens), max(need + [0]) + columns), -1, np.int32)
        at = 0
        seen = np.zeros((nb, bs), bool)
        for s, c in enumerate(lens):
            self.tables[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
            for t in range(c):
                seen[self.tables[s, t // bs], t % bs] = True
        shape = (nb, hkv, bs, d)
        self.pools, self.scales = [], []
        for which in range(2):
            if kind == "fp16":
                codes = rng.standard_normal(shape).astype(np.float16).astype(np.float64)
                scale = np.ones((nb, hkv))
            else:
                codes = Q.round_codes(rng.standard_normal(shape) * Q.TOP[kind] / 3, kind)
                scale = (np.exp(rng.standard_normal((nb, hkv)) * spread) * 3 / Q.TOP[kind]).astype(np.float32)
                scale = scale.astype(np.float64)
                scale[~seen.any(axis=1)] = 1e30
            codes.transpose(0, 2, 1, 3)[~seen] = 127.0 if kind == "int8" else np.nan
            self.pools.append(codes)
            self.scales.append(scale)
        self.q = (rng.standard_normal((len(lens), h, d)) * q_std).astype(np.float16)
        self.lists = None

    def pick(self, keep, order="ascending"):
        """Block lists: up to `keep` of each context's blocks."""
        n, hkv = len(self.lens), self.pools[0].shape[1]
        self.lists = []
        self.selected = np.full((n, hkv, keep), -7, np.int32)
        self.number = np.zeros((n, hkv), np.int32)
        for s in range(n):
            blocks = -(-int(self.lens[s]) // self.bs)
            self.lists.append([])
            for k in range(hkv):
                count = min(blocks, int(self.rng.integers(0, keep + 1)) if order == "any" else keep)
                chosen = self.rng.permutation(blocks)[:count]
                if order == "ascending":
                    chosen = np.sort(chosen)
                self.lists[s].append([int(b) for b in chosen])
                self.selected[s, k, :count] = chosen
                self.number[s, k] = count
        return self

    def gpu(self):
        self.t = {k: torch.from_numpy(np.ascontiguousarray(getattr(self, k))).cuda() for k in ("q", "tables", "lens")}
        self.t["kc"], self.t["vc"] = (to_gpu(x, self.kind) for x in self.pools)
        self.t["ks"], self.t["vs"] = (torch.from_numpy(x.astype(np.float32)).cuda() for x in self.scales)
        if self.lists is not None:
            self.t["selected"], self.t["number"] = (torch.from_numpy(x).cuda() for x in (self.selected, self.number))
        self.out = torch.full(self.q.shape, -77.0, dtype=torch.float16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self

    def call(self, pkv, out=None, **kw):
        t = self.t
        out = self.out if out is None else out
        kw.setdefault("status", self.status)
        if self.kind == "fp16":
            return pkv.paged_attention_decode_selected(out, t["q"], t["kc"], t["vc"], t["tables"], t["lens"],
                                                       t["selected"], t["number"], self.scale, **kw)
        if self.lists is not None:
            kw.update(selected=t["selected"], num_selected=t["number"])
        return pkv.paged_attention_decode_q8(out, t["q"], t["kc"], t["vc"], t["ks"], t["vs"], t["tables"], t["lens"],
                                             self.scale, **kw)

    def oracle(self):
        k, v = (np.nan_to_num(x) * s[:, :, None, None] for x, s in zip(self.pools, self.scales))
        return Q.decode(self.q, k, v, self.tables, self.lens, self.scale, self.lists)

    def check(self, out, expect=None, status=0, warps=4):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        ref, spread, reach, count, top = expect or self.oracle()
        got = out.float().cpu().numpy().astype(np.float64)
        assert np.isfinite(got).all()
        more = 0.0
        if self.kind == "int8":
            more = biased(self.q, self.scales[0], self.tables, self.lens, self.bs, self.scale)
        over = np.abs(got - ref) / bound(ref, spread, reach, count, top, self.d, warps, more)
        assert over.max() <= 1.0, (over.max(), np.unravel_index(over.argmax(), over.shape))


EIGHT = ["int8", "e4m3"]
ALL = ["int8", "e4m3", "fp16"]


@pytest.mark.parametrize("kind", EIGHT)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
def test_decode_block_sizes(pkv, bs, d, kind):
    c = Case(1, kind, 4, 2, d, bs, [1, 7, 8, 9, 15, 16, 17, 33, 100, 127, 128, 129, 300, 0, 65]).gpu()
    c.check(c.call(pkv))


@pytest.mark.parametrize("kind", EIGHT)
@pytest.mark.parametrize("h,hkv", [(1, 1), (4, 4), (4, 2), (3, 1), (7, 1), (8, 1), (9, 1), (10, 2), (16, 1), (48, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_head_layouts(pkv, h, hkv, d, kind):
    c = Case(2, kind, h, hkv, d, 16, [3, 150, 77, 260, 31]).gpu()
    c.check(c.call(pkv))


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("grid", [1, 2, 3, 7, 40, 152, 500])
def test_grids(pkv, grid, kind):
    """The same result however the work is cut; the same bits twice."""
    c = Case(3, kind, 8, 2, 128, 16, [1, 500, 0, 1800, 40, 129, 700])
    if kind == "fp16":
        c.pick(60)
    c.gpu()
    expect = c.oracle()
    first = c.call(pkv, num_ctas=grid).clone()
    c.check(first, expect)
    again = c.call(pkv, out=torch.zeros_like(first), num_ctas=grid)
    assert torch.equal(first.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("h,hkv", [(3, 3), (4, 2), (9, 3), (8, 2), (10, 2), (24, 2)])
@pytest.mark.parametrize("grid", [1, 3, 11, 0])
def test_many_short_pieces(pkv, grid, h, hkv, kind):
    """Pieces of one to a few steps, some between two long ones, of every number
    of heads that goes between two barriers; cut or not."""
    rng = np.random.default_rng(h)
    lens = [int(x) for x in rng.integers(0, 70, 37)] + [700, 1, 33, 0, 0, 900] + [int(x) for x in rng.integers(0, 200, 20)]
    c = Case(30, kind, h, hkv, 128, 16, lens)
    if kind == "fp16":
        c.pick(50, "any")
    c.gpu()
    expect = c.oracle()
    for _ in range(2):
        c.out.fill_(-77)
        c.check(c.call(pkv, num_ctas=grid), expect)


@pytest.mark.parametrize("kind,d", [("int8", 128), ("e4m3", 64)])
def test_one_long_context(pkv, kind, d):
    c = Case(4, kind, 8, 1, d, 64, [20011, 3]).gpu()
    c.check(c.call(pkv))


@pytest.mark.parametrize("n", [255, 256, 257, 1000, 4096])
def test_many_sequences(pkv, n):
    rng = np.random.default_rng(n)
    c = Case(5, "int8", 2, 1, 64, 8, [int(x) for x in rng.integers(0, 12, n)], columns=3).gpu()
    c.check(c.call(pkv))


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("order", ["ascending", "any"])
@pytest.mark.parametrize("bs,d", [(8, 64), (8, 128), (16, 128), (32, 64), (128, 128)])
def test_block_lists(pkv, kind, order, bs, d):
    c = Case(6, kind, 6, 2, d, bs, [1, 400, bs, 0, bs + 1, 900, 5 * bs]).pick(7, order).gpu()
    c.check(c.call(pkv))
    c.check(c.call(pkv, num_ctas=5))


@pytest.mark.parametrize("kind", ALL)
def test_list_of_every_block_and_more_room(pkv, kind):
    c = Case(7, kind, 4, 4, 128, 16, [100, 333, 16]).pick(40).gpu()
    c.check(c.call(pkv))


def test_a_block_listed_twice_counts_twice(pkv):
    c = Case(8, "int8", 2, 1, 64, 16, [64]).pick(4).gpu()
    c.lists[0][0] = [1, 3, 1]
    c.t["selected"][0, 0, :3] = torch.tensor([1, 3, 1], dtype=torch.int32)
    c.t["number"][0, 0] = 3
    c.check(c.call(pkv))


@pytest.mark.parametrize("kind", ALL)
def test_lists_and_tables_out_of_range(pkv, kind):
    """Listed blocks outside the context are left out, too many are cut off, a bad
    table entry reads block 0; each is reported."""
    c = Case(9, kind, 4, 2, 64, 16, [100, 50]).pick(3).gpu()
    c.lists = [[[0, 2], [5]], [[1], [0, 1, 2]]]
    rows = torch.tensor([[[0, -1, 2], [7, 5, 1 << 30]], [[1, 99, 99], [0, 1, 2]]], dtype=torch.int32)
    c.t["selected"].copy_(rows)
    c.t["number"].copy_(torch.tensor([[3, 3], [1, 9]], dtype=torch.int32))
    c.check(c.call(pkv), status=pkv.PKV_ERR_OUT_OF_RANGE)
    c.status.zero_()
    c.t["number"].copy_(torch.tensor([[-2, 3], [1, 3]], dtype=torch.int32))
    c.lists[0][0] = []
    c.check(c.call(pkv), status=pkv.PKV_ERR_OUT_OF_RANGE)
    c = Case(9, kind, 4, 2, 64, 16, [100, 50]).pick(7).gpu()
    c.t["tables"][0, 3], c.t["tables"][1, 0] = c.pools[0].shape[0], -5
    c.tables[0, 3] = c.tables[1, 0] = 0
    for pool, name in zip(c.pools, ("kc", "vc")):  # block 0 may be unused: fill it
        pool[0] = np.where(np.isnan(pool[0]), 1.0, pool[0])
        c.t[name] = to_gpu(pool, kind)
    for scale, name in zip(c.scales, ("ks", "vs")):
        scale[0] = 0.01 if kind != "fp16" else 1.0
        c.t[name] = torch.from_numpy(scale.astype(np.float32)).cuda()
    c.check(c.call(pkv), status=pkv.PKV_ERR_OUT_OF_RANGE)


def test_contexts_out_of_range(pkv):
    c = Case(10, "int8", 2, 2, 64, 16, [40, 20, 9], columns=0).gpu()
    c.t["lens"].copy_(torch.tensor([1 << 30, -3, 9], dtype=torch.int32))
    pad = c.tables.shape[1] * 16
    for pool, name in zip(c.pools, ("kc", "vc")):
        pool[...] = np.where(pool == 127, 3.0, pool)
        c.t[name] = to_gpu(pool, "int8")
    c.lens = np.array([pad, 0, 9], np.int32)
    c.check(c.call(pkv), status=pkv.PKV_ERR_OUT_OF_RANGE)


@pytest.mark.parametrize("kind", EIGHT)
def test_scales_of_any_size(pkv, kind):
    """Value scales from 2^-33 to 2^9, blocks of zeros, key scales of zero."""
    c = Case(11, kind, 4, 1, 128, 16, [16 * 40])
    c.scales[1] = np.exp2(c.rng.integers(-33, 10, c.scales[1].shape)).astype(np.float64)
    c.scales[1][c.tables[0, 3]] = 0.0
    c.scales[0][c.tables[0, 5]] = 0.0
    c.gpu()
    c.check(c.call(pkv))
    c.scales[1][:] = 0.0
    c.gpu()
    assert (c.call(pkv) == 0).all()


def test_a_large_score_and_many_small_ones(pkv):
    """131072 positions 17.5 below one: together 3.3e-3 of the row."""
    n, bs, d = 131072 + 16, 128, 64
    c = Case(12, "int8", 1, 1, d, bs, [1])
    blocks = -(-n // bs)
    codes = np.zeros((blocks, 1, bs, d))
    codes[0, 0, 5, 0] = 127
    values = np.ones((blocks, 1, bs, d)) * 100
    values[0, 0, 5] = 1
    c.pools, c.scales = [codes, values], [np.full((blocks, 1), 1 / 127), np.full((blocks, 1), 0.01)]
    c.tables = np.arange(blocks, dtype=np.int32)[None]
    c.lens = np.array([n], np.int32)
    c.q = np.zeros((1, 1, d), np.float16)
    c.q[0, 0, 0] = 140.0
    c.gpu()
    c.scales = [s.astype(np.float32).astype(np.float64) for s in c.scales]
    c.check(c.call(pkv))


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("q_std", [600.0, 12000.0])
def test_scores_of_any_size(pkv, kind, q_std):
    """The tolerance grows with the scores; the result stays a weighting."""
    c = Case(13, kind, 4, 2, 128, 16, [300, 77], q_std=q_std)
    c.q = np.clip(c.q, -65504, 65504)
    if q_std > 1000 and kind != "fp16":  # scores of 10^9, and the largest value scales: one position decides
        c.scales[0] *= 65504
        c.scales[1] = np.where(c.scales[1] < 1e20, c.scales[1] * 2.0 ** 12, c.scales[1])
    if kind == "fp16":
        c.pick(20)
    c.gpu()
    c.scales = [x.astype(np.float32).astype(np.float64) for x in c.scales]
    c.check(c.call(pkv))


def test_offsets_past_32_bits(pkv):
    """Blocks whose first byte lies past 2^32."""
    hkv, bs, d = 8, 128, 128
    per = hkv * bs * d
    nb = (1 << 32) // per + 40
    kc = torch.zeros(nb, hkv, bs, d, dtype=torch.int8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = (torch.full((nb, hkv), 0.01, device="cuda") for _ in range(2))
    c = Case(14, "int8", 16, hkv, d, bs, [300, 129])
    small = np.unique(c.tables[c.tables >= 0])
    far = nb - 1 - np.arange(len(small))
    where = dict(zip(small.tolist(), far.tolist()))
    for b, f in where.items():
        kc[f], vc[f] = to_gpu(c.pools[0][b], "int8"), to_gpu(c.pools[1][b], "int8")
        ks[f], vs[f] = (torch.from_numpy(s[b].astype(np.float32)).cuda() for s in c.scales)
    c.gpu()
    expect = c.oracle()
    c.t.update(kc=kc, vc=vc, ks=ks, vs=vs)
    c.t["tables"] = torch.from_numpy(np.vectorize(lambda x: where.get(int(x), -1))(c.tables).astype(np.int32)).cuda()
    c.check(c.call(pkv), expect)


def test_streams_graphs_and_workspaces(pkv):
    """On another stream; captured and replayed on new queries; a workspace of any
    contents; two captured graphs that share one, one after the other."""
    c = Case(15, "e4m3", 8, 2, 128, 16, [700, 33, 1200]).gpu()
    d = Case(16, "int8", 16, 1, 64, 32, [2000, 5]).gpu()
    expect, expect_d = c.oracle(), d.oracle()
    ws = pkv.new_team_workspace(16, 1, 128)
    ws.fill_(0xff)
    c.check(c.call(pkv, workspace=ws), expect)
    d.check(d.call(pkv, workspace=ws), expect_d)
    stream = torch.cuda.Stream()
    c.out.fill_(-77)
    stream.wait_stream(torch.cuda.current_stream())
    c.call(pkv, stream=stream)
    stream.synchronize()
    c.check(c.out, expect)
    graphs = []
    for x in (c, d):
        x.out.fill_(-77)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            x.call(pkv, workspace=ws)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    c.check(c.out, expect)
    d.check(d.out, expect_d)
    c.q = (c.rng.standard_normal(c.q.shape)).astype(np.float16)
    c.t["q"].copy_(torch.from_numpy(c.q))
    graphs[0].replay()
    c.check(c.out)


def test_captured_without_a_workspace(pkv):
    """The captured calls' scratch stays theirs: eager calls and tensors of its
    size, between and beside the replays, on the same stream and on another."""
    c, d = Case(36, "int8", 8, 2, 128, 16, [3000, 40, 2000]).gpu(), Case(37, "fp16", 8, 1, 128, 32, [4000, 77]).pick(60).gpu()
    expect, expect_d = c.oracle(), d.oracle()
    c.call(pkv)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(pkv)
        between = torch.full((pkv.decode_team_workspace_size(8, 2, 128),), 0x7f, dtype=torch.uint8, device="cuda")
        d.call(pkv)
    e = Case(38, "e4m3", 4, 4, 64, 16, [2500, 1, 900]).gpu()
    expect_e = e.oracle()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        c.out.fill_(-77)
        d.out.fill_(-77)
        beside = [torch.full((1 << 18,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(4)]
        e.call(pkv, stream=side)
        graph.replay()
        e.call(pkv, stream=side)
        del beside
    torch.cuda.synchronize()
    c.check(c.out, expect)
    d.check(d.out, expect_d)
    e.check(e.out, expect_e)
    assert bool((between == 0x7f).all())


def test_two_streams_at_once(pkv):
    """Calls that run at the same time, each with a workspace of its own."""
    cases = [Case(31, "int8", 8, 2, 128, 16, [3000, 40, 2000]).gpu(), Case(32, "e4m3", 4, 4, 64, 16, [2500, 1, 900]).gpu(),
             Case(33, "fp16", 8, 1, 128, 32, [4000, 77]).pick(60).gpu()]
    expect = [c.oracle() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(50):
        for c, s in zip(cases, streams):
            c.call(pkv, stream=s)
    for c, e in zip(cases, expect):
        c.check(c.out, e)


def test_the_same_bits_every_time(pkv):
    """500 launches on one workspace, two shapes in turn."""
    a, b = Case(34, "int8", 8, 2, 128, 16, [1500, 3, 0, 800]).gpu(), Case(35, "fp16", 12, 4, 64, 8, [900, 60]).pick(40).gpu()
    ws = pkv.new_team_workspace(8, 2, 128)  # the larger of the two
    first = [x.call(pkv, workspace=ws).clone() for x in (a, b)]
    for x, f in zip((a, b), first):
        x.check(f)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(500):
        for x, f in zip((a, b), first):
            x.out.fill_(-77)
            differ += (x.call(pkv, workspace=ws).view(torch.int16) != f.view(torch.int16)).sum()
    assert int(differ.item()) == 0


def test_shapes_that_do_not_fit(pkv):
    """Each tensor with a dimension of another size."""
    for kind in ALL:
        c = Case(18, kind, 4, 2, 64, 16, [30, 20]).pick(2).gpu()
        for name, t in list(c.t.items()):
            if kind == "fp16" and name in ("ks", "vs"):
                continue
            for dim in range(t.dim()):
                if (name, dim) in (("tables", 1), ("selected", 2)):
                    continue
                c.t[name] = torch.cat([t, t], dim=dim)
                with pytest.raises((ValueError, pkv.PkvError)):
                    c.call(pkv)
                c.t[name] = t
        with pytest.raises(ValueError):
            c.call(pkv, out=torch.cat([c.out, c.out]))
        with pytest.raises(ValueError):
            c.call(pkv, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
        with pytest.raises(pkv.PkvError):
            c.call(pkv, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
        c.check(c.call(pkv))


def test_nothing_to_do(pkv):
    c = Case(17, "int8", 2, 2, 64, 16, [0, 0, 0]).gpu()
    assert (c.call(pkv) == 0).all()
    for name in ("q", "tables", "lens"):
        c.t[name] = c.t[name][:0]
    out = c.out[:0]
    assert c.call(pkv, out=out) is out


# ---------------------------------------------------------------------------
# the write

class Write:
    """A pool with codes and scales in every block, and new rows of sequences that
    end at `lens` with `new` tokens each."""

    def __init__(self, seed, kind, hkv, d, bs, lens, new, before=0, behind=0, size=1.0, starts=True):
        rng = self.rng = np.random.default_rng(seed)
        self.kind, self.bs, self.d, self.hkv = kind, bs, d, hkv
        self.lens = np.array(lens, np.int32)
        need = [-(-c // bs) for c in lens]
        nb = sum(need) + 2
        order = rng.permutation(nb)
        self.tables = np.full((len(lens), max(need + [0]) + 1), -1, np.int32)
        at = 0
        for s in range(len(lens)):
            self.tables[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        top = Q.TOP[kind]
        a = np.abs(rng.standard_normal((2, nb, hkv)) * 2 + 2).astype(np.float16)
        self.scales = [(x.astype(np.float32) / np.float32(top)) for x in a]
        self.codes = [Q.round_codes(rng.uniform(-1, 1, (nb, hkv, bs, d)) * top, kind) for _ in range(2)]
        self.starts = (before + np.concatenate([[0], np.cumsum(new)])).astype(np.int32) if starts else None
        t = int(self.starts[-1]) + behind if starts else len(lens)
        self.rows = [(rng.standard_normal((t, hkv, d)) * size * np.exp(rng.standard_normal((t, 1, 1)))).astype(np.float16)
                     for _ in range(2)]

    def gpu(self):
        self.t = dict(tables=torch.from_numpy(self.tables).cuda(), lens=torch.from_numpy(self.lens).cuda(),
                      starts=None if self.starts is None else torch.from_numpy(self.starts).cuda())
        self.t["kc"], self.t["vc"] = (to_gpu(x, self.kind) for x in self.codes)
        self.t["ks"], self.t["vs"] = (torch.from_numpy(x.copy()).cuda() for x in self.scales)
        self.t["k"], self.t["v"] = (torch.from_numpy(x).cuda() for x in self.rows)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self

    def call(self, pkv, **kw):
        t = self.t
        kw.setdefault("status", self.status)
        pkv.reshape_and_cache_q8(t["k"], t["v"], t["kc"], t["vc"], t["ks"], t["vs"], t["tables"], t["lens"],
                                 t["starts"], **kw)

    def check(self, status=0):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        for codes, scale, rows, cache, gpu_scale in zip(self.codes, self.scales, self.rows,
                                                        (self.t["kc"], self.t["vc"]), (self.t["ks"], self.t["vs"])):
            scale64 = scale.astype(np.float64)
            Q.write(codes, scale64, rows, self.tables, self.lens, self.starts, self.kind)
            assert np.array_equal(from_gpu(cache), codes, equal_nan=True)
            assert np.array_equal(gpu_scale.cpu().numpy(), scale64.astype(np.float32))
            scale[...] = scale64


@pytest.mark.parametrize("kind", EIGHT)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
def test_write_block_sizes(pkv, bs, d, kind):
    lens = [1, bs, bs + 1, 3 * bs - 1, 2 * bs, 5, 4 * bs + 3, bs]
    new = [1, bs, 1, bs + 2, 0, 3, 4 * bs + 3, 1]
    w = Write(20, kind, 3, d, bs, lens, new, before=2, behind=3).gpu()
    w.call(pkv)
    w.check()


@pytest.mark.parametrize("kind", EIGHT)
@pytest.mark.parametrize("hkv", [1, 2, 8, 32])
def test_write_one_token_each(pkv, hkv, kind):
    """Without query_starts, token by token: blocks grow their scales, fill up and
    begin anew; empty sequences have no token."""
    w = Write(21, kind, hkv, 128, 16, [14, 1, 32, 0, 17], None, starts=False).gpu()
    for _ in range(5):
        w.call(pkv)
        w.check()
        w.lens = np.where(w.lens == 0, 0, np.where(w.lens % 16 == 0, w.lens, w.lens + 1)).astype(np.int32)
        w.t["lens"].copy_(torch.from_numpy(w.lens))
        w.rows = [(x * 1.25).astype(np.float16) for x in w.rows]
        w.t["k"].copy_(torch.from_numpy(w.rows[0]))
        w.t["v"].copy_(torch.from_numpy(w.rows[1]))


@pytest.mark.parametrize("kind", EIGHT)
def test_write_of_ties(pkv, kind):
    """Quotients that are exact halves of a code's step, in new rows (x top / a with
    a a power of two times the top) and in the ones rounded again (a0 / a = 1/2)."""
    w = Write(22, kind, 1, 64, 16, [16], [16])
    a = 127.0 if kind == "int8" else 448.0
    x = np.arange(64) + 0.5 if kind == "int8" else (np.arange(64) % 8 + 8.5) * 2.0 ** (np.arange(64) // 8)
    w.rows = [np.tile(x, (16, 1, 1)).astype(np.float16) for _ in range(2)]
    for r in w.rows:
        r[3, 0, 7] = a
        r[1::2] *= -1
    w.gpu()
    w.call(pkv)
    w.check()
    w = Write(23, kind, 1, 64, 16, [9], [1])
    w.scales = [np.full_like(s, np.float32(2) / np.float32(Q.TOP[kind])) for s in w.scales]
    w.rows = [np.full((1, 1, 64), 4.0, np.float16) for _ in range(2)]
    w.gpu()
    w.call(pkv)
    w.check()


@pytest.mark.parametrize("kind", EIGHT)
def test_write_of_unusual_values(pkv, kind):
    """Zeros, infinities, NaN, the smallest and largest fp16 values; scales that
    are zero or no numbers."""
    w = Write(24, kind, 2, 64, 16, [40, 20, 5, 33, 16], [30, 4, 2, 1, 16])
    for r in w.rows:
        r[0:4] = 0
        r[5, 0, 3], r[5, 1, 4] = np.inf, -np.inf
        r[9, 0, 0] = np.nan
        r[30:34] *= 2.0 ** -18
        r[34, 1] = 65504
        r[35, 0], r[35, 1] = 0, np.nan
        r[37:] = 0
    for s in w.scales:
        s[w.tables[1, 1]] = 0
        s[w.tables[2, 0]] = 0
    w.gpu()
    w.call(pkv)
    w.check()


def test_write_from_a_projection(pkv):
    """Rows that are views with strides, and another stream."""
    w = Write(25, "int8", 4, 128, 32, [100, 31], [90, 31]).gpu()
    fused = torch.zeros(121, 3 * 4 * 128, dtype=torch.float16, device="cuda")
    fused[:, 512:1024], fused[:, 1024:] = w.t["k"].flatten(1), w.t["v"].flatten(1)
    w.t["k"], w.t["v"] = fused[:, 512:1024].view(121, 4, 128), fused[:, 1024:].view(121, 4, 128)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    w.call(pkv, stream=stream)
    stream.synchronize()
    w.check()


def test_write_out_of_range(pkv):
    """What is out of range is reported and not written; the rest is."""
    def run(change, lens=(40, 20), new=(30, 20), expect=None):
        w = Write(26, "int8", 2, 64, 16, list(lens), list(new)).gpu()
        held = [x.copy() for x in w.codes + w.scales]
        change(w)
        w.call(pkv)
        torch.cuda.synchronize()
        assert int(w.status.item()) == pkv.PKV_ERR_OUT_OF_RANGE
        return w, held

    def bad_entry(w):
        w.t["tables"][0, 1] = w.codes[0].shape[0]
        w.t["tables"][1, 0] = -1

    w, _ = run(bad_entry)
    keep = [(int(w.tables[0, 1]), None), (int(w.tables[1, 0]), None)]
    before = [(c[p].copy(), s[p].copy()) for c, s in zip(w.codes, w.scales) for p, _ in keep]
    for codes, scale, rows in zip(w.codes, w.scales, w.rows):
        s64 = scale.astype(np.float64)
        Q.write(codes, s64, rows, w.tables, w.lens, w.starts, "int8")
        scale[...] = s64
    i = 0
    for codes, scale in zip(w.codes, w.scales):
        for p, _ in keep:
            codes[p], scale[p] = before[i]
            i += 1
    for cache, codes in zip((w.t["kc"], w.t["vc"]), w.codes):
        assert np.array_equal(from_gpu(cache), codes)

    # more tokens than context: the positions there are
    w = Write(27, "int8", 2, 64, 16, [10], [14]).gpu()
    w.call(pkv)
    w.check(status=pkv.PKV_ERR_OUT_OF_RANGE)
    # a negative context: nothing; one past its table: the positions in it
    w = Write(28, "int8", 2, 64, 16, [10, 30], [4, 30]).gpu()
    w.t["lens"].copy_(torch.tensor([-1, 30], dtype=torch.int32))
    w.lens = np.array([0, 30], np.int32)
    w.starts = np.array([4, 4, 34], np.int32)
    w.call(pkv)
    w.check(status=pkv.PKV_ERR_OUT_OF_RANGE)
    # query_starts that decrease or leave the rows: reported, nothing outside is touched
    for starts in ([0, 40, 34], [0, 4, 99], [-5, 4, 34]):
        w = Write(28, "int8", 2, 64, 16, [10, 30], [4, 30]).gpu()
        w.t["starts"].copy_(torch.tensor(starts, dtype=torch.int32))
        w.call(pkv)
        torch.cuda.synchronize()
        assert int(w.status.item()) == pkv.PKV_ERR_OUT_OF_RANGE


def test_write_in_a_graph(pkv):
    w = Write(29, "e4m3", 2, 128, 16, [50], [1]).gpu()
    w.call(pkv)
    torch.cuda.synchronize()
    w.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.call(pkv)
    for k in range(3):
        w.rows = [(x * 1.5).astype(np.float16) for x in w.rows]
        w.t["k"].copy_(torch.from_numpy(w.rows[0]))
        w.t["v"].copy_(torch.from_numpy(w.rows[1]))
        graph.replay()
        w.check()


@pytest.mark.parametrize("kind", EIGHT)
def test_pools_are_copied_and_swapped(pkv, kind):
    """copy_blocks and swap_blocks, one layer and several, on codes and scales."""
    rng = np.random.default_rng(40)
    nb, hkv, bs, d = 12, 3, 8, 64
    codes = [torch.from_numpy(rng.integers(0, 127, (nb, hkv, bs, d)).astype(np.int8)).view(DTYPE[kind]).cuda()
             for _ in range(4)]
    scales = [torch.from_numpy(rng.standard_normal((nb, 4)).astype(np.float32)).cuda() for _ in range(4)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pairs = torch.tensor([[2, 7], [11, 0], [3, 4]], device="cuda")

    def moved(pools, src=None):
        out = []
        for i, p in enumerate(pools):
            q, s = p.cpu().view(torch.uint8).clone(), (src[i] if src else p).cpu().view(torch.uint8)
            for a, b in pairs.tolist():
                q[b] = s[a]
            out.append(q)
        return out

    def same(pools, expect):
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert all(torch.equal(p.cpu().view(torch.uint8), e) for p, e in zip(pools, expect))

    for group in (codes, scales):
        expect = moved(group[:2])
        pkv.copy_blocks(group[0], group[1], pairs, status=status)
        same(group[:2], expect)
        expect = moved(group)
        pkv.copy_blocks_layers(group[0::2], group[1::2], pairs, status=status)
        same(group, expect)
        host = [torch.empty_like(x, device="cpu").fill_(0).pin_memory() for x in group]
        expect = moved(host, group)
        pkv.swap_blocks(group[0], group[1], host[0], host[1], pairs, status=status)
        pkv.swap_blocks_layers(group[2:3], group[3:4], host[2:3], host[3:4], pairs, status=status)
        same(host, expect)
        expect = moved(group, host)
        pkv.swap_blocks_layers(host[0::2], host[1::2], group[0::2], group[1::2], pairs, status=status)
        same(group, expect)
    with pytest.raises(TypeError):
        pkv.copy_blocks(codes[0], codes[1].view(torch.uint8).half(), pairs)
    with pytest.raises((TypeError, ValueError)):
        pkv.swap_blocks(codes[0], codes[1], scales[0].cpu().pin_memory(), scales[1].cpu().pin_memory(), pairs)
    odd = torch.zeros(nb, 3, device="cuda")
    with pytest.raises(pkv.PkvError):
        pkv.copy_blocks(odd, odd.clone(), pairs)
