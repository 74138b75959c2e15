"""One layer's serving path (a prompt in chunks, a fork, decode steps) checked
part by part, each at its own rounding, so that one wrong position, token or
block shows.

* queries and cached keys against the norm and rotation in fp64, at the bound of
  test_gpu_rope.py; cached values bit for bit;
* the attention of those very queries, keys and values in fp64 over each
  sequence's tokens in order (no block table): prompt rows at the
  per-element bound of test_gpu_chunk.py, decode rows within 2e-3.

What the tolerances must reject is planted in the fp64 side, on the CPU.
"""

import numpy as np
import pytest
import torch

from oracle import chunk as OK
from test_gpu_chunk import bound

TOTAL, FORK, PROMPT = 300, 170, 265   # tokens, where the second sequence forks, where the decode steps begin
EPS = 1e-6
LAYOUTS = [(8, 2, 128, 16, 128, False), (4, 4, 64, 8, 32, True), (8, 1, 64, 16, 64, False)]


class Inputs:
    def __init__(self, h, hkv, d, rot, seed=0):
        rng = np.random.default_rng(seed + d)
        self.x = {name: rng.standard_normal((2, TOTAL, n, d)).astype(np.float16)
                  for name, n in (("q", h), ("k", hkv), ("v", hkv))}
        for a in self.x.values():
            a[1, :FORK] = a[0, :FORK]
        self.wq = (1 + 0.1 * rng.standard_normal(d)).astype(np.float16)
        self.wk = (1 + 0.1 * rng.standard_normal(d)).astype(np.float16)
        angle = np.arange(512)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)
        self.cs = np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)
        self.scale = d ** -0.5
        self.rng = rng

    def turned(self, name, interleaved, positions=None, norm=True):
        """fp64 (values, sizes) [2][TOTAL][heads][D] of the queries or keys."""
        w = (self.wq if name == "q" else self.wk) if norm else None
        pos = np.arange(TOTAL) if positions is None else positions
        both = [OK.norm_rope(self.x[name][s], w, EPS, pos, self.cs, interleaved) for s in range(2)]
        return np.stack([y for y, _ in both]), np.stack([z for _, z in both])


def turn_tolerance(ref, size):
    return 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2.0 ** -16 * size


def attend(q, k, v, scale, hidden=None):
    """fp64 attention of one sequence from its start, q [L][H][D]; `hidden`
    (row, position) pairs are left out.  -> (out, tolerance) [L][H][D]."""
    length, h, d = q.shape
    group = h // k.shape[1]
    q, k, v = (a.astype(np.float64) for a in (q, k, v))
    out, tol = np.zeros_like(q), np.zeros_like(q)
    mask = np.triu(np.ones((length, length), bool), 1)
    if hidden is not None:
        mask |= hidden
    count = (~mask).sum(axis=1)
    for x in range(h):
        kx, vx = k[:, x // group], v[:, x // group]
        s = scale * q[:, x] @ kx.T
        s[mask] = -np.inf
        w = np.exp(s - s.max(axis=1, keepdims=True))
        w /= w.sum(axis=1, keepdims=True)
        out[:, x] = w @ vx
        spread = w @ np.abs(vx)
        reach = np.where(mask, 0.0, scale * np.abs(q[:, x]) @ np.abs(kx).T).max(axis=1)
        top = np.maximum.accumulate(np.abs(vx), axis=0)
        tol[:, x] = bound(out[:, x], spread, reach, count, top, d)
    tol[PROMPT:] = 2e-3
    return out, tol


def run(pkv, c, bs, interleaved):
    """The serving program; -> (queries, out) [2][TOTAL][H][D] and the keys and
    values that the cache holds for each sequence, [2][TOTAL][Hkv][D]."""
    h, d = c.x["q"].shape[2:]
    hkv = c.x["k"].shape[2]
    dev = {name: torch.from_numpy(a).cuda() for name, a in c.x.items()}
    args = dict(cos_sin=torch.from_numpy(c.cs).cuda(), query_weight=torch.from_numpy(c.wq).cuda(),
                key_weight=torch.from_numpy(c.wk).cuda(), interleaved=interleaved, eps=EPS)
    mb = -(-TOTAL // bs)
    nb = 3 * mb
    kc = torch.full((nb, hkv, bs, d), float("nan"), dtype=torch.float16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    alloc = pkv.BlockAllocator(nb, bs, c.rng.permutation(nb).astype(np.int32))
    out = torch.full((2, TOTAL, h, d), float("nan"), dtype=torch.float16, device="cuda")
    queries = torch.full_like(out, float("nan"))

    def prompt(parts):
        """parts: (sequence id, index, first, count) of one batch of chunks."""
        rows = {name: torch.cat([dev[name][i, a:a + n] for _, i, a, n in parts]) for name in dev}
        slots = []
        for seq, _, _, n in parts:
            got, cows = alloc.append_tokens(seq, n)
            slots += got
            if cows:
                pkv.copy_blocks(kc, vc, torch.tensor(cows, dtype=torch.int64, device="cuda"), status=status)
        pos = torch.cat([torch.arange(a, a + n) for _, _, a, n in parts]).cuda()
        q = torch.empty_like(rows["q"])
        pkv.qk_norm_rope_and_cache(q, rows["q"], rows["k"], rows["v"], kc, vc,
                                   torch.tensor(slots, dtype=torch.int64, device="cuda"), pos, status=status, **args)
        tables, lens = alloc.export([p[0] for p in parts], mb)
        starts = torch.tensor(np.concatenate([[0], np.cumsum([p[3] for p in parts])]), dtype=torch.int32).cuda()
        o = pkv.paged_attention_chunk(torch.empty_like(q), q, kc, vc, torch.from_numpy(tables).cuda(),
                                      torch.from_numpy(lens).cuda(), starts, c.scale, status=status)
        at = 0
        for _, i, a, n in parts:
            out[i, a:a + n], queries[i, a:a + n] = o[at:at + n], q[at:at + n]
            at += n

    first = alloc.new_seq()
    prompt([(first, 0, 0, 133)])
    prompt([(first, 0, 133, FORK - 133)])
    second = alloc.fork(first)
    out[1, :FORK], queries[1, :FORK] = out[0, :FORK], queries[0, :FORK]
    prompt([(first, 0, FORK, 1), (second, 1, FORK, 90)])   # both write behind the shared block
    prompt([(second, 1, FORK + 90, 5), (first, 0, FORK + 1, 94)])
    assert PROMPT == FORK + 95
    for t in range(PROMPT, TOTAL):
        pos = torch.tensor([t, t], device="cuda")
        q, k = torch.empty_like(dev["q"][:, t]), torch.empty_like(dev["k"][:, t])
        pkv.qk_norm_rope(q, k, dev["q"][:, t], dev["k"][:, t], pos, status=status, **args)
        _, cows = alloc.append_batch([first, second])
        assert len(cows) == 0
        tables, lens = alloc.export([first, second], mb)
        out[:, t] = pkv.paged_attention_decode_append(
            torch.empty_like(q), q, k, dev["v"][:, t].contiguous(), kc, vc, torch.from_numpy(tables).cuda(),
            torch.from_numpy(lens).cuda(), c.scale, status=status)
        queries[:, t] = q
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    tables, lens = alloc.export([first, second], mb)
    assert lens.tolist() == [TOTAL, TOTAL]
    at = np.arange(TOTAL)
    kept = [np.stack([a.cpu().numpy()[tables[s][at // bs], :, at % bs] for s in range(2)]) for a in (kc, vc)]
    return queries.cpu().numpy(), out.float().cpu().numpy().astype(np.float64), *kept


@pytest.mark.gpu
@pytest.mark.parametrize("h,hkv,d,bs,rot,interleaved", LAYOUTS)
def test_each_part_at_its_own_rounding(h, hkv, d, bs, rot, interleaved):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    import paged_kv_cache_152_gb300 as pkv
    from paged_kv_cache_152_gb300 import build
    build.build()
    pkv.load()
    c = Inputs(h, hkv, d, rot)
    q, out, k, v = run(pkv, c, bs, interleaved)
    for name, got in (("q", q), ("k", k)):
        ref, size = c.turned(name, interleaved)
        over = np.abs(got.astype(np.float64) - ref) / turn_tolerance(ref, size)
        assert over.max() <= 1.0, (name, over.max())
    assert np.array_equal(v.view(np.uint16), c.x["v"].view(np.uint16))
    for s in range(2):
        ref, tol = attend(q[s], k[s], v[s], c.scale)
        over = np.abs(out[s] - ref) / tol
        assert over.max() <= 1.0, (s, over.max(), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("h,hkv,d,bs,rot,interleaved", LAYOUTS)
def test_the_tolerances_reject_planted_mistakes(h, hkv, d, bs, rot, interleaved):
    c = Inputs(h, hkv, d, rot)
    q, size = c.turned("q", interleaved)
    k, _ = c.turned("k", interleaved)
    at = np.arange(TOTAL)
    # the norm and rotation: each token's row is off by more than its bound
    late = at + (at >= FORK)
    for wrong, rows in ((c.turned("q", interleaved, positions=late)[0], at >= FORK),
                        (c.turned("q", interleaved, norm=False)[0], at >= 0),
                        (c.turned("q", not interleaved)[0], at > 0)):
        over = (np.abs(wrong - q) / turn_tolerance(q, size)).max(axis=(2, 3))
        assert (over[:, rows] > 4.0).all()
    # the attention: every row concerned is off by more than its bound
    q, k = q.astype(np.float16), k.astype(np.float16)
    v = c.x["v"]
    i, j = np.meshgrid(at, at, indexing="ij")
    for s in range(2):
        ref, tol = attend(q[s], k[s], v[s], c.scale)

        def rejected(rows, hidden=None, kk=k[s], vv=v[s], share=1.0):
            bad, _ = attend(q[s], kk, vv, c.scale, hidden)
            over = (np.abs(bad - ref) / tol).max(axis=(1, 2))[rows]
            assert (over > 1.0).mean() >= share, (over > 1.0).mean()

        # a token's own position is missed, one token too few at the start, one block dropped for late rows
        rejected(at >= 1, (i == j) & (i >= 1))
        rejected(at >= 1, (j == 0) & (i >= 1))
        rejected(at >= FORK, (j >= 32) & (j < 32 + bs) & (i >= FORK))
        # the other sequence's token where both wrote behind the shared block (a lost copy-on-write)
        other_k, other_v = k[s].copy(), v[s].copy()
        other_k[FORK], other_v[FORK] = k[1 - s][FORK], v[1 - s][FORK]
        rejected(at >= FORK, kk=other_k, vv=other_v)
        # two blocks exchanged for a row at the end of the prompt's rows and for a decode row: the softmax does
        # not depend on the order, so exchange keys only
        swapped = k[s].copy()
        swapped[[32 + bs + t for t in range(bs)] + [32 + t for t in range(bs)]] = \
            k[s][[32 + t for t in range(bs)] + [32 + bs + t for t in range(bs)]]
        rejected(at >= FORK, kk=swapped)
        # a decode step that reads zeros
        assert (np.abs(ref) / tol)[PROMPT:].max(axis=(1, 2)).min() > 1.0
