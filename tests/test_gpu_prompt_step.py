"""The serving path of one layer, as a program runs it: a prompt comes in
chunks (norm and rotation into the cache, then chunk attention), forks, and is
continued by single tokens (norm and rotation, then the appending decode),
against an fp64 model of the whole layer that never saw the cache."""

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


def dense(q, k, v, scale):
    """fp64 causal attention of one sequence from its start: q [L][H][D]."""
    length, h, d = q.shape
    group = h // k.shape[1]
    out = np.zeros_like(q)
    for x in range(h):
        s = scale * q[:, x] @ k[:, x // group].T
        s[np.triu_indices(length, 1)] = -np.inf
        w = np.exp(s - s.max(axis=1, keepdims=True))
        out[:, x] = w @ v[:, x // group] / w.sum(axis=1, keepdims=True)
    return out


@pytest.mark.parametrize("h,hkv,d,bs,rot,interleaved", [(8, 2, 128, 16, 128, False), (4, 4, 64, 8, 32, True)])
def test_prompt_chunks_fork_and_decode(pkv, h, hkv, d, bs, rot, interleaved):
    rng = np.random.default_rng(d)
    total = 300
    x = {name: rng.standard_normal((2, total, n, d)).astype(np.float16)
         for name, n in (("q", h), ("k", hkv), ("v", hkv))}
    fork_at = 170    # the second sequence forks from the first here (inside a block)
    for name in x:
        x[name][1, :fork_at] = x[name][0, :fork_at]
    wq = (1 + 0.1 * rng.standard_normal(d)).astype(np.float16)
    wk = (1 + 0.1 * rng.standard_normal(d)).astype(np.float16)
    angle = np.arange(512)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)
    cs = np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)
    scale = d ** -0.5
    ref = []
    for s in range(2):
        q, _ = OK.norm_rope(x["q"][s], wq, 1e-6, np.arange(total), cs, interleaved)
        k, _ = OK.norm_rope(x["k"][s], wk, 1e-6, np.arange(total), cs, interleaved)
        ref.append(dense(q, k, x["v"][s].astype(np.float64), scale))

    dev = {name: torch.from_numpy(a).cuda() for name, a in x.items()}
    args = dict(cos_sin=torch.from_numpy(cs).cuda(), query_weight=torch.from_numpy(wq).cuda(),
                key_weight=torch.from_numpy(wk).cuda(), interleaved=interleaved)
    nb, mb = 3 * -(-total // bs), -(-total // bs)
    kc = torch.full((nb, hkv, bs, d), float("nan"), dtype=torch.float16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    alloc = pkv.BlockAllocator(nb, bs, rng.permutation(nb).astype(np.int32))
    out = torch.full((2, total, h, d), float("nan"), dtype=torch.float16, device="cuda")

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
                                      torch.from_numpy(lens).cuda(), starts, scale, status=status)
        at = 0
        for _, i, a, n in parts:
            out[i, a:a + n] = o[at:at + n]
            at += n

    first = alloc.new_seq()
    prompt([(first, 0, 0, 133)])
    prompt([(first, 0, 133, fork_at - 133)])
    second = alloc.fork(first)
    out[1, :fork_at] = out[0, :fork_at]
    prompt([(first, 0, fork_at, 1), (second, 1, fork_at, 90)])   # both write behind the shared block
    prompt([(second, 1, fork_at + 90, 5), (first, 0, fork_at + 1, 94)])
    at = fork_at + 95
    for t in range(at, total):
        pos = torch.tensor([t, t], device="cuda")
        q, k = torch.empty_like(dev["q"][:, t]), torch.empty_like(dev["k"][:, t])
        pkv.qk_norm_rope(q, k, dev["q"][:, t], dev["k"][:, t], pos, status=status, **args)
        _, cows = alloc.append_batch([first, second])
        assert len(cows) == 0
        tables, lens = alloc.export([first, second], mb)
        o = pkv.paged_attention_decode_append(torch.empty_like(q), q, k, dev["v"][:, t].contiguous(), kc, vc,
                                              torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), scale,
                                              status=status)
        out[:, t] = o
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = out.float().cpu().numpy().astype(np.float64)
    # Queries and keys are rounded to fp16 before the scores here and not in
    # the model: 2^-11 relative each.  With normed heads |q|, |k| <= 1.5 sqrt(d)
    # (weights within 1 +- 0.5), so a score is off by at most
    # scale * 2 * 2^-11 * sum |q_i k_i| <= 2^-10 * 2.25 sqrt(d), a weight by
    # twice that relative (numerator and sum), and the output by that times
    # max |v| <= 5.5; the rest is the attention calls' own 2e-3 bound at
    # unit-variance values.
    tol = 2 * 2.0 ** -10 * 2.25 * d ** 0.5 * 5.5 + 2e-3
    assert np.abs(got - np.stack(ref)).max() <= tol
