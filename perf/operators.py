"""The chunk attention and the query/key norm with rotation, as cases to measure.

Two groups of calls stand here.  ``op`` "chunk" is attention of each sequence's
newest tokens over its block-mapped cache (prefill, a chunk of a long prompt,
the verification of drafted tokens, single tokens, a sliding window, and with
``causal`` false the attention over an encoder's cached states).  ``op``
"rotate" is the step before it: an RMS norm of every query and key head and
the position rotation, with the keys and values either written to their cache
slots (``cached``) or returned for a decode call that appends them.

``own`` false: the plain form, elementary torch operations in 32 bits rounded
once to fp16.  ``own`` true: the library's calls.
"""

import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# cases

def _chunk(name, heads, kv_heads, head_dim, block, seqs, ctx, new, singles=0, causal=True, window=0, lens=1):
    """seqs sequences with contexts spread over ctx = (low, high) and new
    tokens over new = (low, high), the first `singles` of them with one; lens
    seeds the spread."""
    return {"name": name, "op": "chunk", "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "block": block,
            "seqs": seqs, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0], "new_hi": new[1],
            "singles": singles, "causal": causal, "window": window, "lens": lens}


def _rotate(name, tokens, heads, kv_heads, head_dim, rot_dim, norm, interleaved, cached, block=16):
    return {"name": name, "op": "rotate", "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rot_dim": rot_dim, "norm": norm, "interleaved": interleaved, "cached": cached,
            "block": block}


def listed():
    return [
        # the smallest serving step: four short chats of a few tokens each (the tiny workload's shape)
        _chunk("tiny-chunk", 8, 8, 64, 16, 4, (5, 100), (2, 9)),
        # checking 5 drafted tokens of each of 64 chats (the 7b workload's batch and contexts)
        _chunk("verify-drafts", 32, 32, 128, 16, 64, (50, 900), (5, 5)),
        # single tokens over long, ragged contexts: few rows, the cache split over the SMs
        _chunk("long-single-tokens", 32, 8, 128, 32, 8, (8000, 32768), (1, 1)),
        # a whole prompt of a 32-head model in one call
        _chunk("prefill", 32, 32, 128, 16, 1, (4096, 4096), (4096, 4096)),
        # a chunk of a long grouped-query prompt
        _chunk("prompt-chunk-gqa", 32, 8, 128, 32, 1, (32768, 32768), (2048, 2048)),
        # a serving batch: 28 single tokens and four prompt chunks together (the gqa workload's contexts)
        _chunk("mixed-batch", 32, 8, 128, 32, 32, (256, 4096), (100, 700), singles=28),
        # a sliding-window layer, group 8, ragged prompts
        _chunk("window-1024", 16, 2, 128, 64, 2, (6000, 9001), (1000, 4001), window=1024),
        # decoder tokens over an encoder's 1500 states each (no causal mask), head_dim 64
        _chunk("cross-1500", 12, 12, 64, 16, 8, (1500, 1500), (63, 448), causal=False),
        # one decode step of 64 chats: norm and rotation for the appending decode
        _rotate("rotate-decode", 64, 32, 32, 128, 128, True, False, False),
        # one token of one chat
        _rotate("rotate-one", 1, 8, 8, 64, 64, True, False, False),
        # a prompt chunk of a grouped-query model, keys and values into the cache
        _rotate("rotate-prefill-cache", 8192, 32, 8, 128, 128, True, False, True, 32),
        # an odd number of tokens, half of each head rotated in adjacent pairs, no norm
        _rotate("rotate-partial-cache", 2047, 16, 16, 64, 32, False, True, True, 16),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.35:
        head_dim = rng.choice([64, 80, 96, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
        heads = kv_heads * rng.choice([1, 1, 2, 4, 7, 8])
        tokens = max(1, min(_spread(rng, 1, 16384), (8192 * 48 * 128) // ((heads + 2 * kv_heads) * head_dim)))
        rot_dim = head_dim if rng.random() < 0.6 else head_dim // 2 // 16 * 16
        c = _rotate("", tokens, heads, kv_heads, head_dim, rot_dim, rng.random() < 0.7, rng.random() < 0.3,
                    rng.random() < 0.6, rng.choice([8, 16, 32, 64, 128]))
    else:
        kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
        heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 4, 6, 8])
        ctx_hi = _spread(rng, 1, 32768)
        ctx_lo = max(1, min(ctx_hi, _spread(rng, max(1, ctx_hi // 16), ctx_hi)))
        new_hi = _spread(rng, 1, ctx_hi)
        new_lo = max(1, min(new_hi, _spread(rng, max(1, new_hi // 8), new_hi)))
        seqs = _spread(rng, 1, 64)
        # the plain form's scores stay under those of the largest listed case
        seqs = max(1, min(seqs, (1 << 31) // (heads * new_hi * ctx_hi), (1 << 19) // ctx_hi))
        if heads * new_hi * ctx_hi > 1 << 31:
            new_hi = max(1, (1 << 31) // (heads * ctx_hi))
            new_lo = min(new_lo, new_hi)
        causal = rng.random() < 0.8
        c = _chunk("", heads, kv_heads, rng.choice([64, 128, 128]), rng.choice([8, 16, 16, 32, 64, 128]), seqs,
                   (ctx_lo, ctx_hi), (new_lo, new_hi), singles=seqs // 2 if rng.random() < 0.3 else 0, causal=causal,
                   window=_spread(rng, 1, ctx_hi) if causal and rng.random() < 0.25 else 0, lens=rng.randrange(1000))
    del c["name"]
    return c


def _lengths(c):
    """Context lengths and new-token counts of a chunk case."""
    r = np.random.default_rng(c["lens"])
    ctx = r.integers(c["ctx_lo"], c["ctx_hi"] + 1, size=c["seqs"])
    new = r.integers(c["new_lo"], c["new_hi"] + 1, size=c["seqs"])
    new[:c["singles"]] = 1
    if c["causal"]:  # new tokens are the context's last; an encoder's states are another sequence's
        new = np.minimum(new, ctx)
    return ctx.astype(np.int64), new.astype(np.int64)


def _visible(c, ctx, new):
    """(query, key) pairs that the mask lets through, and the cache rows read, over all sequences."""
    pairs = rows = 0
    for length, n in zip(ctx.tolist(), new.tolist()):
        if not c["causal"]:
            pairs, rows = pairs + n * length, rows + length
            continue
        pos = np.arange(length - n, length) + 1
        w = c["window"] or length
        pairs += int(np.minimum(pos, w).sum())
        rows += min(length, n - 1 + w)
    return pairs, rows


def work(case):
    c = case
    if c["op"] == "chunk":
        ctx, new = _lengths(c)
        pairs, rows = _visible(c, ctx, new)
        q = int(new.sum()) * c["heads"] * c["head_dim"] * 2
        tables = int(sum(-(-int(x) // c["block"]) for x in ctx)) * 4
        return {"bytes": 2 * q + 2 * rows * c["kv_heads"] * c["head_dim"] * 2 + tables + 8 * c["seqs"],
                "flops": 4 * pairs * c["heads"] * c["head_dim"]}
    t, d = c["tokens"], c["head_dim"]
    heads = c["heads"] + c["kv_heads"] * (2 if c["cached"] else 1)
    return {"bytes": 2 * t * heads * d * 2 + t * c["rot_dim"] * 4 + t * (16 if c["cached"] else 8),
            "flops": t * (c["heads"] + c["kv_heads"]) * (c["rot_dim"] * 3 + (4 * d if c["norm"] else 0))}


# ---------------------------------------------------------------------------
# inputs

def _normal(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).half()


def _pool(blocks, c, g):
    shape = (blocks, c["kv_heads"], c["block"], c["head_dim"])
    return _normal(shape, g), _normal(shape, g)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = np.random.default_rng(seed)
    d = c["head_dim"]
    s = {"case": c}
    if c["op"] == "chunk":
        ctx, new = _lengths(c)
        need = -(-ctx // c["block"])
        blocks = int(math.ceil(1.25 * int(need.sum())))
        order = r.permutation(blocks).astype(np.int32)
        tables = np.full((c["seqs"], int(need.max())), -1, np.int32)
        at = np.concatenate([[0], np.cumsum(need)])
        for i in range(c["seqs"]):
            tables[i, :need[i]] = order[at[i]:at[i + 1]]
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s["key_cache"], s["value_cache"] = _pool(blocks, c, g)
        s["query"] = _normal((int(starts[-1]), c["heads"], d), g, 1.5)
        s["out"] = torch.empty_like(s["query"])
        s["block_tables"] = torch.from_numpy(tables).cuda()
        s["context_lens"] = torch.from_numpy(ctx.astype(np.int32)).cuda()
        s["query_starts"] = torch.from_numpy(starts).cuda()
        s["most_new"] = int(new.max())
        s["scale"] = d ** -0.5
        return s
    t, h, hk, rot = c["tokens"], c["heads"], c["kv_heads"], c["rot_dim"]
    fused = _normal((t, (h + 2 * hk) * d), g, 2.0)  # the output of one projection: rows of queries, keys, values
    s["query"] = fused[:, :h * d].view(t, h, d)
    s["key"] = fused[:, h * d:(h + hk) * d].view(t, hk, d)
    s["value"] = fused[:, (h + hk) * d:].view(t, hk, d)
    reach = 32768
    freq = 10000.0 ** (-torch.arange(0, rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
    angle = torch.arange(reach, device="cuda", dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()
    first = int(r.integers(0, reach - t + 1))
    s["positions"] = torch.arange(first, first + t, device="cuda", dtype=torch.int64)
    s["query_weight"] = s["key_weight"] = None
    if c["norm"]:
        s["query_weight"], s["key_weight"] = 1 + 0.1 * _normal((d,), g), 1 + 0.1 * _normal((d,), g)
    s["query_out"] = torch.empty((t, h, d), device="cuda", dtype=torch.float16)
    if c["cached"]:
        need = -(-t // c["block"])
        blocks = need + need // 4 + 1
        s["key_cache"], s["value_cache"] = _pool(blocks, c, g)
        order = r.permutation(blocks).astype(np.int64)[:need]
        slots = (order[:, None] * c["block"] + np.arange(c["block"])).reshape(-1)[:t]
        s["slot_mapping"] = torch.from_numpy(slots.copy()).cuda()
    else:
        s["key_out"] = torch.empty((t, hk, d), device="cuda", dtype=torch.float16)
    return s


# ---------------------------------------------------------------------------
# the plain form

def _chunk_plain(s):
    c = s["case"]
    hk, d = c["kv_heads"], c["head_dim"]
    group = c["heads"] // hk
    seqs, most = c["seqs"], s["most_new"]
    lens = s["context_lens"].long()
    starts = s["query_starts"].long()
    new = starts[1:] - starts[:-1]
    total = s["query"].shape[0]
    device = s["query"].device
    # each sequence's cache rows in logical order, padded to the longest table
    tables = s["block_tables"].long().clamp(min=0)
    keys = s["key_cache"][tables].permute(0, 2, 1, 3, 4).reshape(seqs, hk, -1, d).float()
    values = s["value_cache"][tables].permute(0, 2, 1, 3, 4).reshape(seqs, hk, -1, d).float()
    rows = (starts[:-1, None] + torch.arange(most, device=device)).clamp(max=total - 1)
    q = s["query"][rows].view(seqs, most, hk, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, hk, most * group, d)
    x = torch.matmul(q.float(), keys.transpose(2, 3)).view(seqs, hk, most, group, -1).mul_(s["scale"])
    t = torch.arange(keys.shape[2], device=device)
    hidden = (t >= lens[:, None])[:, None, :].expand(seqs, most, -1)
    if c["causal"]:
        pos = (lens - new)[:, None] + torch.arange(most, device=device)
        hidden = hidden | (t > pos[..., None])
        if c["window"]:
            hidden = hidden | (t <= pos[..., None] - c["window"])
    x.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    sums = x.sum(dim=-1, keepdim=True)
    o = torch.matmul(x.view(seqs, hk, most * group, -1), values).view(seqs, hk, most, group, d)
    o = (o / sums.clamp(min=1e-30)).permute(0, 2, 1, 3, 4).reshape(seqs, most, hk * group, d)
    token = torch.arange(total, device=device)
    seq = torch.searchsorted(starts, token, right=True) - 1
    s["out"].copy_(o[seq, token - starts[seq]])
    return s["out"]


def _turn(x, weight, s):
    """RMS norm of each head (where there is a weight) and the rotation, in 32 bits."""
    c = s["case"]
    rot = c["rot_dim"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + 1e-6) * weight.float()
    table = s["cos_sin"][s["positions"]]
    cos, sin = table[:, None, :rot // 2], table[:, None, rot // 2:]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _rotate_plain(s):
    c = s["case"]
    s["query_out"].copy_(_turn(s["query"], s["query_weight"], s))
    key = _turn(s["key"], s["key_weight"], s).half()
    if not c["cached"]:
        s["key_out"].copy_(key)
        return s["query_out"], s["key_out"]
    block, offset = s["slot_mapping"] // c["block"], s["slot_mapping"] % c["block"]
    s["key_cache"][block, :, offset] = key
    s["value_cache"][block, :, offset] = s["value"]
    return s["query_out"], s["key_cache"], s["value_cache"]


# ---------------------------------------------------------------------------
# the library's calls

def _run_own(s):
    import paged_kv_cache_152_gb300 as pkv
    c = s["case"]
    if c["op"] == "chunk":
        return pkv.paged_attention_chunk(s["out"], s["query"], s["key_cache"], s["value_cache"], s["block_tables"],
                                         s["context_lens"], s["query_starts"], s["scale"], causal=c["causal"],
                                         window=c["window"])
    if c["cached"]:
        pkv.qk_norm_rope_and_cache(s["query_out"], s["query"], s["key"], s["value"], s["key_cache"],
                                   s["value_cache"], s["slot_mapping"], s["positions"], s["cos_sin"],
                                   query_weight=s["query_weight"], key_weight=s["key_weight"],
                                   interleaved=c["interleaved"])
        return s["query_out"], s["key_cache"], s["value_cache"]
    pkv.qk_norm_rope(s["query_out"], s["key_out"], s["query"], s["key"], s["positions"], s["cos_sin"],
                     query_weight=s["query_weight"], key_weight=s["key_weight"], interleaved=c["interleaved"])
    return s["query_out"], s["key_out"]


def run(state):
    if own:
        return _run_own(state)
    return _chunk_plain(state) if state["case"]["op"] == "chunk" else _rotate_plain(state)


# ---------------------------------------------------------------------------
# the definition in 64 bits

def _chunk_exact(s):
    """One query row block of one sequence and KV head at a time."""
    c = s["case"]
    d, bs = c["head_dim"], c["block"]
    group = c["heads"] // c["kv_heads"]
    ctx, new = _lengths(c)
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for i in range(c["seqs"]):
        length, n = int(ctx[i]), int(new[i])
        used = s["block_tables"][i, :-(-length // bs)].long()
        for k in range(c["kv_heads"]):
            keys = s["key_cache"][used, k].reshape(-1, d)[:length].double()
            values = s["value_cache"][used, k].reshape(-1, d)[:length].double()
            for lo in range(0, n, 1024):
                hi = min(n, lo + 1024)
                heads = slice(k * group, (k + 1) * group)
                q = s["query"][first + lo:first + hi, heads].double()
                z = torch.einsum("ngd,td->ngt", q, keys) * s["scale"]
                if c["causal"]:
                    where = torch.arange(length - n + lo, length - n + hi, device="cuda")[:, None, None]
                    behind = where - torch.arange(length, device="cuda")
                    seen = behind >= 0
                    if c["window"]:
                        seen = seen & (behind < c["window"])
                    z = torch.where(seen, z, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
                out[first + lo:first + hi, heads] = torch.einsum("ngt,td->ngd", torch.softmax(z, dim=-1), values)
        first += n
    return out


def _turn_exact(x, weight, s):
    c = s["case"]
    rot = c["rot_dim"]
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["head_dim"] + 1e-6).sqrt() * weight.double()
    table = s["cos_sin"].double().index_select(0, s["positions"])
    spin = torch.complex(table[:, :rot // 2], table[:, rot // 2:])[:, None]
    if c["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * spin
        x[..., :rot] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * spin
        x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "chunk":
        return _chunk_exact(s)
    query = _turn_exact(s["query"], s["query_weight"], s)
    key = _turn_exact(s["key"], s["key_weight"], s)
    if not case["cached"]:
        return query, key
    caches = []
    for cache, rows in ((s["key_cache"], key), (s["value_cache"], s["value"].double())):
        flat = cache.double().transpose(1, 2).flatten(0, 1)  # [slot][head][element]
        flat[s["slot_mapping"]] = rows
        caches.append(flat.unflatten(0, (cache.shape[0], cache.shape[2])).transpose(1, 2).contiguous())
    return query, caches[0], caches[1]
