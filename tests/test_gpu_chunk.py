"""GPU parity of the chunk attention (through the binding) with the fp64
oracle, at the sizes and masks where it can go wrong.

Tolerance, per output element, from the roundings the call makes:

* the output's rounding to fp16: half a step, 2^-11 |out| (2^-25 below the
  normal range);
* each softmax weight's rounding to fp16: 2^-11 relative, together at most
  2^-11 sum_t w_t |v_t|, and half of fp16's smallest step, 2^-25, where a
  weight is below the normal range.  The stored weights are relative to a
  running maximum that has been at least one visible score, so their sum is
  at least 1: at most count * 2^-25 * max |v|;
* scores in fp32: a product of D terms is off by at most D * 2^-24 of the sum
  of the terms' magnitudes however it is summed, doubled here because tensor
  cores may cut instead of round; the exponent's own arithmetic and ex2 add
  2^-20 for scores below 16 in magnitude (fp32 at 32 has steps of 2^-19); a score off by x
  moves a weight by the factor e^x, in the numerator and the sum;
* the weighted sum and the sum of weights in fp32, at most 256 terms in a
  tile and a few hundred tiles and pieces: 2^-14 of sum_t w_t |v_t|.
"""

import numpy as np
import pytest
import torch

from oracle import chunk as OK

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


def bound(ref, spread, reach, count, top, d):
    score = 2 * d * 2.0 ** -24 * reach + 2.0 ** -20 * np.maximum(1.0, reach / 16)
    return (2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (2.0 ** -11 + 2.0 ** -14) * spread +
            2 * score[..., None] * spread + count[..., None] * 2.0 ** -25 * top)


class Case:
    """Sequences of (new, context) tokens with shuffled blocks.  Every pool
    position that no row sees holds NaN, blocks that no row sees are -1 in the
    tables, and out starts as a sentinel."""

    def __init__(self, seed, h, hkv, d, bs, seqs, causal=True, window=0, before=0, behind=0, q_std=1.5,
                 extra_columns=1):
        rng = np.random.default_rng(seed)
        self.d, self.causal, self.window, self.scale = d, causal, window, d ** -0.5
        new = [n for n, _ in seqs]
        self.lens = np.array([c for _, c in seqs], np.int32)
        self.starts = (before + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)
        rows = int(self.starts[-1]) + behind
        need = [-(-int(c) // bs) for c in self.lens]
        nb = sum(need) + 3
        order = rng.permutation(nb)
        self.tables = np.full((len(seqs), max(need) + extra_columns), -1, np.int32)
        seen = np.zeros((nb, bs), bool)
        at = 0
        for s, (n, c) in enumerate(seqs):
            ids = order[at:at + need[s]]
            at += need[s]
            for i in range(n):
                for t in OK.visible(int(c), n, i, causal, window):
                    seen[ids[t // bs], t % bs] = True
            used = seen[ids].any(axis=1)
            self.tables[s, :need[s]] = np.where(used, ids, -1)
        self.kc = rng.standard_normal((nb, hkv, bs, d)).astype(np.float16)
        self.vc = rng.standard_normal((nb, hkv, bs, d)).astype(np.float16)
        self.kc.transpose(0, 2, 1, 3)[~seen] = np.nan
        self.vc.transpose(0, 2, 1, 3)[~seen] = np.nan
        self.q = (rng.standard_normal((rows, h, d)) * q_std).astype(np.float16)
        self.rows = rows

    def gpu(self):
        self.t = {k: torch.from_numpy(np.ascontiguousarray(getattr(self, k))).cuda()
                  for k in ("q", "kc", "vc", "tables", "lens", "starts")}
        self.out = torch.full(self.q.shape, -77.0, dtype=torch.float16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self

    def call(self, pkv, out=None, **kw):
        t = self.t
        out = self.out if out is None else out
        pkv.paged_attention_chunk(out, t["q"], t["kc"], t["vc"], t["tables"], t["lens"], t["starts"], self.scale,
                                  causal=self.causal, window=self.window, status=self.status, **kw)
        return out

    def oracle(self):
        return OK.paged_chunk_attention(self.q, self.kc, self.vc, self.tables, self.lens, self.starts, self.scale,
                                        self.causal, self.window)

    def check(self, out, expect=None):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        ref, spread, reach, count, top = expect or self.oracle()
        got = out.float().cpu().numpy().astype(np.float64)
        mine = ~np.isnan(ref).all(axis=(1, 2))
        assert (got[~mine] == -77.0).all(), "rows of no sequence were written"
        ref, got = ref[mine], got[mine]
        tol = bound(ref, spread[mine], reach[mine], count[mine], top[mine], self.d)
        assert np.isfinite(got).all()
        over = np.abs(got - ref) / tol
        assert over.max() <= 1.0, (over.max(), np.unravel_index(over.argmax(), over.shape))


LAYOUTS = [(1, 1), (4, 4), (4, 2), (8, 2), (8, 1), (3, 1), (10, 2), (7, 1), (16, 1)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
def test_block_sizes(pkv, bs, d):
    c = Case(1, 4, 2, d, bs, [(1, 1), (1, 130), (5, 5), (37, 200), (129, 129), (2, 127), (64, 301)]).gpu()
    c.check(c.call(pkv))


@pytest.mark.parametrize("h,hkv", LAYOUTS)
@pytest.mark.parametrize("d", [64, 128])
def test_head_layouts(pkv, h, hkv, d):
    c = Case(2, h, hkv, d, 16, [(3, 3), (140, 150), (1, 77), (41, 260)], before=2, behind=3).gpu()
    c.check(c.call(pkv))


@pytest.mark.parametrize("n,length", [(1, 1), (2, 2), (127, 127), (128, 128), (129, 129), (255, 256), (256, 256),
                                      (257, 257), (1, 128), (1, 129), (300, 513), (128, 384), (3, 1000)])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths_around_tile_edges(pkv, n, length, causal):
    c = Case(3, 2, 1, 128, 16, [(n, length)], causal=causal).gpu()
    c.check(c.call(pkv))


@pytest.mark.parametrize("window", [1, 2, 100, 127, 128, 129, 1000])
@pytest.mark.parametrize("d,group", [(64, 1), (128, 1), (128, 4)])
def test_sliding_windows(pkv, window, d, group):
    """Blocks behind every row's window are -1 in the tables."""
    c = Case(4, group, 1, d, 16, [(300, 700), (1, 515), (17, 17), (260, 260)], window=window).gpu()
    c.check(c.call(pkv))


@pytest.mark.parametrize("group,window,d", [(8, 1000, 128), (8, 1024, 64), (5, 900, 128), (2, 1500, 128)])
def test_windows_of_many_steps(pkv, group, window, d):
    """Query tiles whose windows begin in different steps, over more steps than
    are in flight at once."""
    c = Case(27, group, 1, d, 32, [(260, 2300), (150, 1400), (90, 1700)], window=window).gpu()
    c.check(c.call(pkv, num_ctas=3))
    c.check(c.call(pkv))


def test_rows_that_see_nothing(pkv):
    """No context, more new tokens than context, no new tokens."""
    c = Case(5, 4, 2, 128, 16, [(4, 0), (0, 0), (200, 30), (0, 50), (300, 20), (1, 0)], behind=5).gpu()
    c.check(c.call(pkv))
    c = Case(5, 4, 2, 64, 16, [(4, 0), (9, 0)]).gpu()
    c.check(c.call(pkv))
    c = Case(6, 4, 2, 128, 16, [(300, 0), (7, 50)], causal=False).gpu()
    c.check(c.call(pkv))


@pytest.mark.parametrize("lengths", [[(448, 150)], [(1, 1500), (3, 7), (65, 300)]])
def test_cross_attention(pkv, lengths):
    c = Case(7, 6, 6, 64, 16, lengths, causal=False).gpu()
    c.check(c.call(pkv))


@pytest.mark.parametrize("num_ctas", [1, 2, 3, 7, 152, 601])
@pytest.mark.parametrize("window", [0, 90])
def test_any_grid(pkv, num_ctas, window):
    c = Case(8, 8, 2, 128, 16, [(1, 900), (70, 500), (200, 210), (5, 1300), (0, 40), (1, 1)], window=window).gpu()
    expect = c.oracle()
    c.check(c.call(pkv, num_ctas=num_ctas), expect)


def test_many_short_sequences(pkv):
    rng = np.random.default_rng(9)
    seqs = [(int(n), int(n + x)) for n, x in zip(rng.integers(0, 4, 700), rng.integers(0, 40, 700))]
    c = Case(9, 2, 1, 64, 8, seqs).gpu()
    c.check(c.call(pkv))


def test_most_sequences(pkv):
    """4096 sequences, all but the first and last few without tokens."""
    seqs = [(2, 20)] + [(0, 0)] * 2000 + [(1, 300)] + [(0, 5)] * 2093 + [(3, 3)]
    c = Case(10, 2, 2, 128, 16, seqs).gpu()
    c.check(c.call(pkv))


@pytest.mark.parametrize("q_std", [0.0, 30.0, 300.0])
def test_flat_and_peaked_scores(pkv, q_std):
    c = Case(11, 4, 2, 128, 16, [(150, 400), (1, 600)], q_std=q_std).gpu()
    c.check(c.call(pkv))


def test_growing_scores(pkv):
    """Keys that grow along the context: the running maximum rises in every
    tile, by more and by less than a factor a weight can carry."""
    c = Case(12, 2, 1, 128, 16, [(40, 900), (1, 700)])
    for s in range(2):
        for t in range(int(c.lens[s])):
            c.kc[c.tables[s, t // 16], :, t % 16] = 0.0
            c.kc[c.tables[s, t // 16], :, t % 16, :8] = t / 100.0
    c.q[..., :8] = np.abs(c.q[..., :8])
    c.gpu()
    c.check(c.call(pkv))


def test_lowest_keys(pkv):
    """Scores at the bottom of the range fp16 keys reach: -65504 everywhere,
    and everywhere but at one position."""
    c = Case(13, 1, 1, 64, 16, [(130, 300)])
    seen = ~np.isnan(c.kc)
    c.kc[seen] = -65504.0
    c.q[:] = 1.0
    c.kc[c.tables[0, 1], :, 3] = 1.0
    c.gpu()
    c.check(c.call(pkv))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("window,group", [(0, 1), (50, 1), (0, 4), (130, 4)])
def test_hidden_values_reach_no_row(pkv, bad, window, group):
    """A position of the chunk itself holds NaN or infinity, in K and in V: the
    rows that do not see it are as without it, those that see it are not finite."""
    c = Case(14, group, 1, 128, 16, [(300, 340), (40, 90)], window=window).gpu()
    ref, spread, reach, count, top = c.oracle()
    hit = []
    for s, t in ((0, 200), (1, 71)):
        c.t["kc"][c.tables[s, t // 16], :, t % 16] = bad
        c.t["vc"][c.tables[s, t // 16], :, t % 16, 5] = bad
        n, length = int(c.starts[s + 1] - c.starts[s]), int(c.lens[s])
        hit += [int(c.starts[s]) + i for i in range(n) if t in OK.visible(length, n, i, True, window)]
    out = c.call(pkv)
    torch.cuda.synchronize()
    clean = np.setdiff1d(np.arange(c.rows), hit)
    assert len(hit) and len(clean)
    got = out.float().cpu().numpy().astype(np.float64)
    tol = bound(ref, spread, reach, count, top, c.d)
    assert (np.abs(got - ref) <= tol)[clean].all()
    if not np.isinf(bad):
        assert np.isnan(got[hit]).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("window,num_ctas", [(0, 0), (0, 1), (130, 0)])
def test_seen_values_that_are_not_finite(pkv, bad, window, num_ctas):
    """V alone holds NaN or infinity in one element: that element of the rows
    that see it, and nothing else, is so (flat scores: no weight underflows)."""
    c = Case(15, 2, 1, 128, 16, [(300, 340), (1, 700), (40, 90)], window=window, q_std=0.1).gpu()
    expect = c.oracle()
    ref = expect[0].copy()
    for s, t in ((0, 200), (1, 650), (2, 71)):
        c.t["vc"][c.tables[s, t // 16], :, t % 16, 5] = bad
        n, length = int(c.starts[s + 1] - c.starts[s]), int(c.lens[s])
        for i in range(n):
            if t in OK.visible(length, n, i, True, window):
                ref[int(c.starts[s]) + i, :, 5] = bad
    out = c.call(pkv, num_ctas=num_ctas)
    torch.cuda.synchronize()
    got = out.float().cpu().numpy().astype(np.float64)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
    assert (np.abs(got - expect[0]) <= bound(*expect, c.d))[fine].all()


def test_single_tokens_agree_with_the_decode(pkv):
    c = Case(16, 8, 2, 128, 32, [(1, n) for n in (1, 31, 32, 33, 900, 4000, 129)]).gpu()
    out = c.call(pkv)
    c.check(out)
    dec = torch.empty_like(out)
    pkv.paged_attention_decode(dec, c.t["q"], c.t["kc"], c.t["vc"], c.t["tables"], c.t["lens"], c.scale)
    # each is within 2e-3 of the oracle, the decode's documented bound, the chunk's by the check above
    assert (out.float() - dec.float()).abs().max().item() <= 2e-3 + 2e-3


def test_pieces_of_a_prompt_equal_the_whole(pkv):
    """Chunked prefill: the same rows whatever chunks the prompt comes in, each
    within the bound."""
    whole = Case(17, 4, 2, 128, 16, [(700, 700)]).gpu()
    expect = whole.oracle()
    whole.check(whole.call(pkv), expect)
    out = torch.full_like(whole.out, -77.0)
    cuts = [0, 1, 130, 131, 384, 640, 700]
    for a, b in zip(cuts, cuts[1:]):
        pkv.paged_attention_chunk(out[a:b], whole.t["q"][a:b], whole.t["kc"], whole.t["vc"], whole.t["tables"],
                                  torch.tensor([b], dtype=torch.int32, device="cuda"),
                                  torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), whole.scale,
                                  status=whole.status)
    whole.check(out, expect)


def test_same_bits_and_a_dirty_workspace(pkv):
    c = Case(18, 8, 2, 128, 16, [(1, 3000), (70, 500), (200, 210)]).gpu()
    ws = pkv.new_chunk_workspace(c.rows, 8, 2, 128)
    ws.fill_(0xFF)   # NaN in every float
    first = c.call(pkv, workspace=ws).clone()
    c.check(first)
    for fill in (0x00, 0x7F):
        ws.fill_(fill)
        again = c.call(pkv, out=torch.full_like(first, -77.0), workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(first, again)


def test_graphs_and_streams(pkv):
    """Two graphs that share a workspace, replayed in turn with new contents
    in the same buffers, and a call on another stream."""
    a = Case(19, 4, 2, 128, 16, [(1, 2500), (33, 600)]).gpu()
    b = Case(20, 4, 2, 128, 16, [(129, 700), (2, 900)]).gpu()
    ws = pkv.new_chunk_workspace(max(a.rows, b.rows), 4, 2, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.call(pkv, workspace=ws)
        b.call(pkv, workspace=ws)
    side.synchronize()
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(pkv, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    a.check(a.out)
    b.check(b.out)
    # other lengths in the captured buffers
    a.lens[:] = [1234, 77]
    a.t["lens"].copy_(torch.from_numpy(a.lens))
    graphs[0].replay()
    graphs[1].replay()
    a.kc = np.nan_to_num(a.kc)
    a.check(a.out)
    b.check(b.out)
    b.out.fill_(-77.0)
    side.wait_stream(torch.cuda.current_stream())
    b.call(pkv, workspace=ws, stream=side)
    side.synchronize()
    b.check(b.out)


def test_two_calls_at_once(pkv):
    """On two streams, each with its own workspace."""
    cases = [Case(21 + i, 8, 2, 128, 16, [(1, 2000 + i), (100, 400)]).gpu() for i in range(2)]
    expect = [c.oracle() for c in cases]
    ws = [pkv.new_chunk_workspace(c.rows, 8, 2, 128) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, w, s in zip(cases, ws, streams):
            c.call(pkv, workspace=w, stream=s)
    torch.cuda.synchronize()
    for c, e in zip(cases, expect):
        c.check(c.out, e)


def test_own_workspace_stays_with_its_stream(pkv, monkeypatch):
    """The workspace a call allocates is not handed to the current stream's
    work while a call on another stream may still use it."""
    c = Case(28, 8, 2, 128, 16, [(1, 2000), (100, 400)]).gpu()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    taken, empty = [], torch.empty

    def spy(*args, **kw):
        taken.append(empty(*args, **kw))
        return taken[-1]

    monkeypatch.setattr(torch, "empty", spy)
    c.call(pkv, stream=side)
    monkeypatch.undo()
    assert len(taken) == 1
    size, address = taken[0].numel(), taken.pop().data_ptr()
    later = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(x.data_ptr() != address for x in later)
    side.synchronize()
    c.check(c.out)


def test_blocks_far_into_a_large_pool(pkv):
    """Element offsets past 2^32 in each cache (8.6 GB, only the used blocks written)."""
    hkv, bs, d = 8, 16, 128
    nb = (1 << 32) // (hkv * bs * d) + 40
    c = Case(23, 8, hkv, d, bs, [(20, 300), (1, 500)])
    small = c.kc.shape[0]
    shift = nb - small
    c.gpu()
    kc = torch.empty((nb, hkv, bs, d), dtype=torch.float16, device="cuda")
    vc = torch.empty_like(kc)
    kc[:64].fill_(float("nan"))
    vc[:64].fill_(float("nan"))
    kc[shift:], vc[shift:] = c.t["kc"], c.t["vc"]
    c.t["kc"], c.t["vc"] = kc, vc
    c.t["tables"] = torch.where(c.t["tables"] >= 0, c.t["tables"] + shift, c.t["tables"])
    c.check(c.call(pkv))


def _shifted(t, bytes):
    """The same tensor at an address `bytes` past a 256-byte boundary."""
    n = bytes // t.element_size()
    room = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    view = room[n:].view(t.shape)
    view.copy_(t)
    assert view.data_ptr() % 256 == bytes
    return view


@pytest.mark.parametrize("h,hkv,d", [(4, 2, 64), (8, 1, 128)])
def test_addresses_of_the_least_alignment(pkv, h, hkv, d):
    """16 bytes past a boundary: every tensor, for items of one tile and of
    two, whole ones and ones in parts, and rows that see nothing."""
    c = Case(27, h, hkv, d, 16, [(3, 40), (140, 900), (1, 2000), (200, 150), (300, 300)]).gpu()
    expect = c.oracle()
    for k in ("q", "kc", "vc"):
        c.t[k] = _shifted(c.t[k], 16)
    for k in ("tables", "lens", "starts"):
        c.t[k] = _shifted(c.t[k], 4)
    for num_ctas in (0, 3):
        c.check(c.call(pkv, out=_shifted(c.out, 16), num_ctas=num_ctas), expect)


def _refuses(pkv, c, code, rows=None, **changes):
    old = dict(c.t)
    c.t.update(changes)
    c.status.zero_()
    out = c.call(pkv, out=torch.full_like(c.out, -77.0))
    torch.cuda.synchronize()
    assert int(c.status.item()) == code
    c.t = old
    c.status.zero_()
    return out


def test_bad_device_data_is_reported(pkv):
    """Entries outside the pool, contexts outside their table and starts out of
    order set the status word; the sequences not concerned keep their rows and
    the device stays usable."""
    c = Case(24, 4, 2, 128, 16, [(5, 100), (130, 200), (3, 50)], extra_columns=0, behind=2).gpu()
    good = c.call(pkv).clone()
    c.check(good)
    starts = c.starts.tolist()
    for entry in (-1, c.kc.shape[0], 1 << 30):
        tables = c.t["tables"].clone()
        tables[1, 2] = entry
        out = _refuses(pkv, c, pkv.PKV_ERR_OUT_OF_RANGE, tables=tables)
        assert torch.equal(out[:5], good[:5]) and torch.equal(out[135:], good[135:])
    columns = c.tables.shape[1]
    for length in (-1, -(1 << 31), columns * 16 + 1, (1 << 31) - 1):
        lens = c.t["lens"].clone()
        lens[0] = length
        out = _refuses(pkv, c, pkv.PKV_ERR_OUT_OF_RANGE, lens=lens)
        assert torch.equal(out[5:], good[5:])
        if length < 0:
            assert (out[:5] == 0).all()
    for bad in ([starts[0], -3, starts[2], starts[3]], [starts[0], starts[1], starts[2], c.rows + 1],
                [starts[0], starts[2], starts[1], starts[3]], [-1] + starts[1:],
                [(1 << 31) - 1, -(1 << 31), starts[2], starts[3]]):
        out = _refuses(pkv, c, pkv.PKV_ERR_OUT_OF_RANGE,
                       starts=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert (out[starts[3]:] == -77.0).all() or bad[-1] > starts[3]
    c.check(c.call(pkv))


def test_nothing_to_do(pkv):
    c = Case(25, 4, 2, 128, 16, [(5, 100)]).gpu()
    t = c.t
    none = torch.empty(0, 4, 128, dtype=torch.float16, device="cuda")
    pkv.paged_attention_chunk(none, none, t["kc"], t["vc"], t["tables"], t["lens"],
                              torch.zeros(2, dtype=torch.int32, device="cuda"), 0.1)
    pkv.paged_attention_chunk(c.out, t["q"], t["kc"], t["vc"], t["tables"][:0], t["lens"][:0], t["starts"][:1], 0.1)
    torch.cuda.synchronize()
    assert (c.out == -77.0).all()


def test_refusals_on_the_gpu(pkv):
    c = Case(26, 4, 2, 128, 16, [(5, 100)]).gpu()
    for kw, code in ((dict(num_ctas=-1), pkv.PKV_ERR_INVALID_ARG),
                     (dict(workspace=torch.empty(128, dtype=torch.uint8, device="cuda")), pkv.PKV_ERR_INVALID_ARG)):
        with pytest.raises(pkv.PkvError) as e:
            c.call(pkv, **kw)
        assert e.value.status in (code, pkv.PKV_ERR_UNSUPPORTED)
    for causal, window in ((False, 5), (True, -1)):
        c.causal, c.window = causal, window
        with pytest.raises(pkv.PkvError) as e:
            c.call(pkv)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (c.out == -77.0).all() and int(c.status.item()) == 0
