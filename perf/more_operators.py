"""The 8-bit paged cache and the block-sparse decode, as cases to measure.

Five calls stand here, by ``op``:

* "write": new tokens into a cache of 8-bit codes with one scale for each block
  and KV head (prompts, or one token of each sequence);
* "decode": single-token attention over such a cache;
* "bounds": the largest and smallest key of each block, channel by channel;
* "select": the blocks whose keys can score highest, for each sequence and KV head;
* "selected": single-token attention over listed blocks of an fp16 cache.

``own`` false: the plain form, elementary torch operations in 32 bits (64 where
a value is rounded to 8 bits or compared with others), rounded once.  ``own``
true: the library's calls.
"""

import math

import numpy as np
import torch

own = False

# the largest code of each 8-bit type
_TOP = {"int8": 127.0, "e4m3": 448.0}
_DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases

def _case(name, op, heads, kv_heads, head_dim, block, seqs, ctx, kind="fp16", new=(1, 1), keep=0, first=1, last=2,
          lens=1):
    """seqs sequences with contexts spread over ctx = (low, high), the last new
    = (low, high) tokens of each being new; kind is the cache's type; keep the
    blocks kept for each sequence and KV head, first and last the ones always
    kept; lens seeds the spread."""
    return {"name": name, "op": op, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "block": block,
            "seqs": seqs, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "kind": kind, "new_lo": new[0], "new_hi": new[1],
            "keep": keep, "first": first, "last": last, "lens": lens}


def listed():
    return [
        # the smallest serving step: four short chats (the tiny workload's shape)
        _case("decode-tiny", "decode", 8, 8, 64, 16, 4, (5, 100), "int8"),
        # a step of 64 chats, one query head per KV head (the 7b workload's batch and contexts)
        _case("decode-chats", "decode", 32, 32, 128, 16, 64, (50, 900), "int8"),
        # a large grouped-query batch (the gqa workload's contexts)
        _case("decode-gqa", "decode", 32, 8, 128, 32, 256, (256, 4096), "e4m3"),
        # few, long, ragged contexts: the cache split over the whole GPU
        _case("decode-long", "decode", 32, 8, 128, 32, 8, (8000, 32768), "int8"),
        # the write of one token of each of 64 sequences, blocks partly filled
        _case("write-step", "write", 32, 8, 128, 16, 64, (1, 64), "int8"),
        # the write of four ragged prompts
        _case("write-prompts", "write", 32, 8, 128, 16, 4, (1000, 4001), "int8", new=(1000, 4001)),
        # one step's upkeep of the bounds: the last block of each of 64 sequences
        _case("bounds-step", "bounds", 32, 8, 128, 32, 64, (256, 4096)),
        # the bounds of two whole prompts
        _case("bounds-prompts", "bounds", 32, 8, 128, 32, 2, (8000, 16384), new=(8000, 16384)),
        # the choice of 64 of up to 1024 blocks for 8 long contexts
        _case("select-long", "select", 32, 8, 128, 32, 8, (8000, 32768), keep=64),
        # ... of 128 blocks of 16 tokens for a batch of 64
        _case("select-batch", "select", 32, 8, 128, 16, 64, (4000, 16384), keep=128, first=4, last=8),
        # attention over 64 blocks of each long context
        _case("selected-long", "selected", 32, 8, 128, 32, 8, (8000, 32768), keep=64),
        # ... and over 128 smaller ones of each of 64
        _case("selected-batch", "selected", 32, 8, 128, 16, 64, (4000, 16384), keep=128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "write", "bounds", "select", "selected"])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 4, 6, 8, 16])
    head_dim = rng.choice([64, 128, 128])
    block = rng.choice([8, 16, 16, 32, 64, 128])
    sparse = op in ("select", "selected")
    ctx_hi = _spread(rng, 64 if sparse else 1, 32768)
    ctx_lo = max(1, min(ctx_hi, _spread(rng, max(1, ctx_hi // 16), ctx_hi)))
    # cache elements of the longest context, times the sequences: at most those of 8 contexts of 32768 and 8 KV heads
    row = kv_heads * head_dim
    most = (8 * 32768 * 8 * 128) if op in ("decode", "selected") else (1 << 23)
    if op == "select":
        most = 8 * 32768 * 8 * 128 * block // 32
    while ctx_hi * row > most:
        ctx_hi, ctx_lo = ctx_hi // 2, max(1, ctx_lo // 2)
    seqs = max(1, min(_spread(rng, 1, 256), most // (ctx_hi * row)))
    new = (1, 1)
    if op in ("write", "bounds") and rng.random() < 0.6:
        new_hi = _spread(rng, 1, ctx_hi)
        new = (max(1, new_hi // 3), new_hi)
    blocks = -(-ctx_hi // block)
    keep = _spread(rng, 1, max(1, min(blocks, 4096 // block * 4))) if sparse else 0
    first = rng.randrange(0, 1 + min(4, keep))
    last = rng.randrange(0, 1 + min(8, keep - first))
    kind = "fp16"
    if op in ("decode", "write"):
        kind = rng.choice(["int8", "e4m3"])
    elif op == "selected":
        kind = rng.choice(["fp16", "fp16", "int8", "e4m3"])
    c = _case("", op, heads, kv_heads, head_dim, block, seqs, (ctx_lo, ctx_hi), kind, new, keep, first, last,
              rng.randrange(1000))
    del c["name"]
    return c


def _lengths(c):
    """Context lengths and new-token counts."""
    r = np.random.default_rng(c["lens"])
    ctx = r.integers(c["ctx_lo"], c["ctx_hi"] + 1, size=c["seqs"])
    new = np.minimum(r.integers(c["new_lo"], c["new_hi"] + 1, size=c["seqs"]), ctx)
    return ctx.astype(np.int64), new.astype(np.int64)


def work(case):
    c = case
    ctx, new = _lengths(c)
    h, hk, d, bs = c["heads"], c["kv_heads"], c["head_dim"], c["block"]
    blocks = -(-ctx // bs)
    touched = blocks - (ctx - new) // bs  # blocks that hold new tokens
    size = 2 if c["kind"] == "fp16" else 1
    scales = 0 if size == 2 else 8
    lists = int(blocks.sum()) * 4 + 4 * c["seqs"]
    if c["op"] == "write":
        t = int(new.sum())
        return {"bytes": t * hk * d * 6 + int(touched.sum()) * (hk * scales + 4) + 8 * c["seqs"], "flops": 4 * t * hk * d}
    if c["op"] == "bounds":
        rows = int((ctx - (ctx - new) // bs * bs).sum())
        return {"bytes": rows * hk * d * 2 + int(touched.sum()) * (hk * d * 4 + 4) + 8 * c["seqs"],
                "flops": 2 * rows * hk * d}
    kept = np.minimum(blocks, c["keep"])
    if c["op"] == "select":
        n = int(blocks.sum())
        return {"bytes": n * hk * d * 4 + c["seqs"] * h * d * 2 + lists + (int(kept.sum()) + c["seqs"]) * hk * 4,
                "flops": 4 * n * h * d}
    if c["op"] == "selected":  # the last block is among those kept
        rows = np.where(kept < blocks, kept * bs - (blocks * bs - ctx), ctx)
        lists += int(kept.sum()) * hk * 4
        blocks = kept
    else:
        rows = ctx
    rows = int(rows.sum())
    return {"bytes": 2 * rows * hk * d * size + 2 * c["seqs"] * h * d * 2 + int(blocks.sum()) * hk * scales + lists,
            "flops": 4 * rows * h * d}


# ---------------------------------------------------------------------------
# inputs

def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _codes(x, kind):
    """The pool x (fp32 [NB][Hkv][bs][D]) in fp16, or as 8-bit codes and scales."""
    if kind == "fp16":
        return x.half(), None
    top = _TOP[kind]
    a = x.abs().amax(dim=(2, 3)).half().float()
    codes = x.mul_((top / a)[..., None, None]).clamp_(-top, top)
    return (codes.round_() if kind == "int8" else codes).to(_DTYPE[kind]), a / top


def _pools(blocks, c, g):
    """Key and value pools: keys with some channels larger than the rest, values whose size changes from block to block."""
    shape = (blocks, c["kv_heads"], c["block"], c["head_dim"])
    channel = 1 + 3 * (torch.rand((c["kv_heads"], 1, c["head_dim"]), generator=g, device="cuda") < 0.05)
    keys, key_scale = _codes(_normal(shape, g, 0.8).mul_(channel), c["kind"])
    values, value_scale = _codes(_normal(shape, g).mul_(_normal((blocks, 1, 1, 1), g, 0.4).exp_()), c["kind"])
    return keys, values, key_scale, value_scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = np.random.default_rng(seed)
    h, hk, d, bs, n = c["heads"], c["kv_heads"], c["head_dim"], c["block"], c["seqs"]
    ctx, new = _lengths(c)
    need = -(-ctx // bs)
    blocks = int(math.ceil(1.25 * int(need.sum())))
    order = r.permutation(blocks).astype(np.int32)
    tables = np.full((n, int(need.max())), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    for i in range(n):
        tables[i, :need[i]] = order[at[i]:at[i + 1]]
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s = {"case": c, "block_tables": torch.from_numpy(tables).cuda(),
         "context_lens": torch.from_numpy(ctx.astype(np.int32)).cuda(),
         "query_starts": torch.from_numpy(starts).cuda(), "tokens": int(starts[-1]), "scale": d ** -0.5}
    if c["op"] in ("decode", "selected"):
        s["key_cache"], s["value_cache"], s["key_scale"], s["value_scale"] = _pools(blocks, c, g)
    if c["op"] == "write":
        # what the cache holds of the tokens before, and new rows of one projection's output
        s["key_cache"], s["value_cache"], s["key_scale"], s["value_scale"] = _pools(blocks, c, g)
        rows = _normal((s["tokens"], 2 * hk * d), g, 1.2).half()
        s["key"], s["value"] = rows[:, :hk * d].view(-1, hk, d), rows[:, hk * d:].view(-1, hk, d)
        s["key_values"] = torch.empty(s["key_cache"].shape, device="cuda", dtype=torch.float16)
        s["value_values"] = torch.empty_like(s["key_values"])
        return s
    if c["op"] == "bounds":
        s["key_cache"] = _normal((blocks, hk, bs, d), g).half()
        s["key_bounds"] = torch.zeros((blocks, hk, 2, d), device="cuda", dtype=torch.float16)
        return s
    s["query"] = _normal((n, h, d), g, 1.5).half()
    if c["op"] == "select":
        middle = _normal((blocks, hk, 1, d), g, 0.7)
        reach = _normal((blocks, hk, 2, d), g, 0.4).add_(1.5).abs_()
        reach[:, :, 1].neg_()
        s["key_bounds"] = reach.add_(middle).half()
        s["selected"] = torch.full((n, hk, c["keep"]), -1, device="cuda", dtype=torch.int32)
        s["num_selected"] = torch.zeros((n, hk), device="cuda", dtype=torch.int32)
        return s
    s["out"] = torch.empty_like(s["query"])
    if c["op"] == "selected":
        # any choice of blocks, the last one among them
        count = torch.from_numpy(need).cuda()
        index = torch.arange(tables.shape[1], device="cuda")
        x = torch.rand((n, hk, tables.shape[1]), generator=g, device="cuda")
        x = torch.where(index == count[:, None, None] - 1, 2.0, x)
        x = torch.where(index >= count[:, None, None], -1.0, x)
        best = x.topk(min(c["keep"], tables.shape[1]), dim=2)
        kept = torch.where(best.values < 0, 1 << 30, best.indices).sort(dim=2).values
        s["selected"] = torch.full((n, hk, c["keep"]), -1, device="cuda", dtype=torch.int32)
        s["selected"][..., :kept.shape[2]] = torch.where(kept == 1 << 30, -1, kept).int()
        s["num_selected"] = (s["selected"] >= 0).sum(dim=2).int()
    return s


# ---------------------------------------------------------------------------
# the plain form

def _softmax_sum(s, keys, values, hidden):
    """Attention of each sequence's query over keys and values (fp32 [N][Hkv][rows][D]) where `hidden` [N][1 or Hkv][rows] is false."""
    c = s["case"]
    q = s["query"].float().view(c["seqs"], c["kv_heads"], -1, c["head_dim"])
    x = torch.matmul(q, keys.transpose(2, 3)).mul_(s["scale"])
    x.masked_fill_(hidden[:, :, None, :], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    o = torch.matmul(x, values) / x.sum(dim=-1, keepdim=True).clamp(min=1e-30)
    s["out"].copy_(o.view(s["out"].shape))
    return s["out"]


def _decode_plain(s):
    c = s["case"]
    tables = s["block_tables"].long().clamp(min=0)
    rows = []
    for cache, scale in ((s["key_cache"], s["key_scale"]), (s["value_cache"], s["value_scale"])):
        x = cache[tables].float() * scale[tables][..., None, None]
        rows.append(x.transpose(1, 2).reshape(c["seqs"], c["kv_heads"], -1, c["head_dim"]))
    t = torch.arange(rows[0].shape[2], device="cuda")
    return _softmax_sum(s, rows[0], rows[1], (t >= s["context_lens"][:, None])[:, None])


def _selected_plain(s):
    c = s["case"]
    kept = s["selected"].long()
    seq = torch.arange(c["seqs"], device="cuda")[:, None, None]
    head = torch.arange(c["kv_heads"], device="cuda")[None, :, None]
    phys = s["block_tables"][seq, kept.clamp(min=0)].long().clamp(min=0)
    rows = []
    for cache, scale in ((s["key_cache"], s["key_scale"]), (s["value_cache"], s["value_scale"])):
        x = cache[phys, head].float()
        if scale is not None:
            x = x * scale[phys, head][..., None, None]
        rows.append(x.flatten(2, 3))
    t = (kept[..., None] * c["block"] + torch.arange(c["block"], device="cuda")).flatten(2)
    return _softmax_sum(s, rows[0], rows[1], (t < 0) | (t >= s["context_lens"][:, None, None]))


def _values(s):
    """What the caches' codes stand for, and the scales."""
    for codes, scale, values in ((s["key_cache"], s["key_scale"], s["key_values"]),
                                 (s["value_cache"], s["value_scale"], s["value_values"])):
        torch.mul(codes if codes.dtype == torch.int8 else codes.half(), scale[..., None, None], out=values)
    return s["key_values"], s["value_values"], s["key_scale"], s["value_scale"]


def _places(s):
    """Physical block and offset of each new token."""
    c = s["case"]
    starts = s["query_starts"].long()
    token = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(starts, token, right=True) - 1
    pos = s["context_lens"].long()[seq] - starts[seq + 1] + token
    return s["block_tables"].long()[seq, pos // c["block"]], pos % c["block"]


def _write_one(s, x, codes, scale, phys, offset):
    c = s["case"]
    top, bs = _TOP[c["kind"]], c["block"]
    int8 = c["kind"] == "int8"
    x = x.float()
    a_new = torch.zeros_like(scale).index_reduce_(0, phys, x.abs().amax(dim=2), "amax")
    first = torch.full((scale.shape[0],), bs, device="cuda").scatter_reduce_(0, phys, offset, "amin")
    a_old = (scale * top).half().float()
    a = torch.maximum(torch.where(first[:, None] == 0, 0.0, a_old), a_new)
    # earlier rows of a block whose largest magnitude has grown
    grown = ((first > 0) & (first < bs))[:, None] & (a > a_old)
    row = torch.arange(bs, device="cuda")
    again = grown[:, :, None, None] & (row < first[:, None])[:, None, :, None]
    old = codes.float()
    turned = old.double() * a_old.double()[..., None, None] / a.double().clamp(min=1e-30)[..., None, None]
    old = torch.where(again, turned.round().float() if int8 else turned.float(), old)
    codes.copy_(old.to(codes.dtype))
    y = x.double() * top / a[phys].double().clamp(min=1e-30)[..., None]
    codes[phys, :, offset] = (y.round().float() if int8 else y.float()).to(codes.dtype)
    scale.copy_(torch.where((first < bs)[:, None], a / top, scale))


def _write_plain(s):
    phys, offset = _places(s)
    _write_one(s, s["key"], s["key_cache"], s["key_scale"], phys, offset)
    _write_one(s, s["value"], s["value_cache"], s["value_scale"], phys, offset)
    return _values(s)


def _bounds_plain(s):
    c = s["case"]
    seq = torch.arange(c["seqs"], device="cuda")
    index = torch.arange(s["block_tables"].shape[1], device="cuda")
    lens = s["context_lens"].long()
    new = (s["query_starts"][1:] - s["query_starts"][:-1]).long()
    touched = (index >= ((lens - new) // c["block"])[:, None]) & (index * c["block"] < lens[:, None])
    seq, index = touched.nonzero(as_tuple=True)
    phys = s["block_tables"].long()[seq, index]
    keys = s["key_cache"][phys].float()
    t = index[:, None] * c["block"] + torch.arange(c["block"], device="cuda")
    hidden = (t >= lens[seq][:, None])[:, None, :, None]
    hi = keys.masked_fill(hidden, -math.inf).amax(dim=2)
    lo = keys.masked_fill(hidden, math.inf).amin(dim=2)
    s["key_bounds"][phys] = torch.stack([hi, lo], dim=2).half()
    return s["key_bounds"]


def _select_plain(s):
    c = s["case"]
    keep = c["keep"]
    tables = s["block_tables"].long().clamp(min=0)
    bounds = s["key_bounds"][tables].double().permute(0, 2, 4, 3, 1)  # [N][Hkv][D][hi, lo][blocks]
    q = s["query"].double().view(c["seqs"], c["kv_heads"], -1, c["head_dim"])
    score = torch.matmul(q.clamp(min=0), bounds[:, :, :, 0]) + torch.matmul(q.clamp(max=0), bounds[:, :, :, 1])
    score = score.amax(dim=2)
    count = (s["context_lens"].long() + c["block"] - 1) // c["block"]
    count = count[:, None, None]
    index = torch.arange(tables.shape[1], device="cuda")
    score = torch.where((index < c["first"]) | (index >= count - c["last"]), math.inf, score)
    score = torch.where(index < count, score, -math.inf)
    order = score.sort(dim=2, descending=True, stable=True).indices[..., :keep]
    kept = torch.where(order < count, order, 1 << 30).sort(dim=2).values
    s["selected"].fill_(-1)
    s["selected"][..., :kept.shape[2]] = torch.where(kept == 1 << 30, -1, kept).int()
    s["num_selected"].copy_(count[..., 0].clamp(max=keep).expand(-1, c["kv_heads"]))
    return s["selected"], s["num_selected"]


# ---------------------------------------------------------------------------
# the library's calls

def _run_own(s):
    import paged_kv_cache_152_gb300 as pkv
    c = s["case"]
    if c["op"] == "decode":
        return pkv.paged_attention_decode_q8(s["out"], s["query"], s["key_cache"], s["value_cache"], s["key_scale"],
                                             s["value_scale"], s["block_tables"], s["context_lens"], s["scale"])
    if c["op"] == "selected":
        if c["kind"] == "fp16":
            return pkv.paged_attention_decode_selected(s["out"], s["query"], s["key_cache"], s["value_cache"],
                                                       s["block_tables"], s["context_lens"], s["selected"],
                                                       s["num_selected"], s["scale"])
        return pkv.paged_attention_decode_q8(s["out"], s["query"], s["key_cache"], s["value_cache"], s["key_scale"],
                                             s["value_scale"], s["block_tables"], s["context_lens"], s["scale"],
                                             selected=s["selected"], num_selected=s["num_selected"])
    if c["op"] == "write":
        pkv.reshape_and_cache_q8(s["key"], s["value"], s["key_cache"], s["value_cache"], s["key_scale"],
                                 s["value_scale"], s["block_tables"], s["context_lens"], s["query_starts"])
        return _values(s)
    if c["op"] == "bounds":
        return pkv.block_key_bounds(s["key_bounds"], s["key_cache"], s["block_tables"], s["context_lens"],
                                    s["query_starts"], s["tokens"])
    return pkv.select_blocks(s["selected"], s["num_selected"], s["query"], s["key_bounds"], s["block_tables"],
                             s["context_lens"], c["block"], first_blocks=c["first"], last_blocks=c["last"])


def run(state):
    if own:
        return _run_own(state)
    return {"decode": _decode_plain, "selected": _selected_plain, "write": _write_plain, "bounds": _bounds_plain,
            "select": _select_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definition in 64 bits

def _decode_exact(s, ctx):
    """One sequence and KV head at a time."""
    c = s["case"]
    bs, d = c["block"], c["head_dim"]
    group = c["heads"] // c["kv_heads"]
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device="cuda")
    offsets = torch.arange(bs, device="cuda")
    for i in range(c["seqs"]):
        blocks = torch.arange(-(-int(ctx[i]) // bs), device="cuda")
        for k in range(c["kv_heads"]):
            use = blocks
            if c["op"] == "selected":
                use = s["selected"][i, k, :int(s["num_selected"][i, k])].long()
            phys = s["block_tables"][i, use].long()
            seen = (use[:, None] * bs + offsets < int(ctx[i])).reshape(-1)
            keys, values = s["key_cache"][phys, k].double(), s["value_cache"][phys, k].double()
            if s["key_scale"] is not None:
                keys = keys * s["key_scale"][phys, k].double().view(-1, 1, 1)
                values = values * s["value_scale"][phys, k].double().view(-1, 1, 1)
            heads = slice(k * group, (k + 1) * group)
            z = s["query"][i, heads].double() @ keys.reshape(-1, d)[seen].T * s["scale"]
            out[i, heads] = torch.softmax(z, dim=-1) @ values.reshape(-1, d)[seen]
    return out


def _to_codes(y, kind):
    if kind == "int8":
        return torch.round(y)
    # e4m3: four significant bits down to 2^-6, steps of 2^-9 below
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _write_exact(s, ctx, new):
    """One sequence's block at a time, all KV heads together."""
    c = s["case"]
    bs, top = c["block"], _TOP[c["kind"]]
    starts = np.concatenate([[0], np.cumsum(new)])
    tables = s["block_tables"].cpu().numpy()
    found = []
    for x, cache, scale in ((s["key"], s["key_cache"], s["key_scale"]), (s["value"], s["value_cache"], s["value_scale"])):
        values = cache.to(torch.float32).double()
        codes = values.clone()
        scales = scale.double()
        for i in range(c["seqs"]):
            begin, end = int(ctx[i] - new[i]), int(ctx[i])
            for b in range(begin // bs, (end - 1) // bs + 1):
                lo, hi = max(begin, b * bs), min(end, (b + 1) * bs)
                rows = x[int(starts[i]) + lo - begin:int(starts[i]) + hi - begin].double().transpose(0, 1)
                p, r = int(tables[i, b]), lo - b * bs
                size = rows.abs().amax(dim=(1, 2))
                if r > 0:
                    before = (scale[p] * top).half().double()
                    size = torch.maximum(size, before)
                    scaled = _to_codes(codes[p, :, :r] * (before / size)[:, None, None], c["kind"])
                    grew = (size > before)[:, None, None]
                    codes[p, :, :r] = torch.where(grew, scaled, codes[p, :, :r])
                codes[p, :, r:r + hi - lo] = _to_codes(top * rows / size[:, None, None], c["kind"])
                scales[p] = size / top
        found.append((codes * scales[..., None, None], scales))
    return found[0][0], found[1][0], found[0][1], found[1][1]


def _bounds_exact(s, ctx, new):
    c = s["case"]
    bs = c["block"]
    tables = s["block_tables"].cpu().numpy()
    bounds = s["key_bounds"].double()
    for i in range(c["seqs"]):
        for b in range(int(ctx[i] - new[i]) // bs, (int(ctx[i]) - 1) // bs + 1):
            keys = s["key_cache"][int(tables[i, b]), :, :min(bs, int(ctx[i]) - b * bs)].double()
            bounds[int(tables[i, b])] = torch.stack([keys.max(dim=1).values, keys.min(dim=1).values], dim=1)
    return bounds


def _select_exact(s, ctx):
    c = s["case"]
    group, keep = c["heads"] // c["kv_heads"], c["keep"]
    selected = torch.full((c["seqs"], c["kv_heads"], keep), -1, dtype=torch.int64)
    number = torch.zeros((c["seqs"], c["kv_heads"]), dtype=torch.int64)
    for i in range(c["seqs"]):
        n = -(-int(ctx[i]) // c["block"])
        forced = [b for b in range(n) if b < c["first"] or b >= n - c["last"]]
        bounds = s["key_bounds"][s["block_tables"][i, :n].long()].double()
        for k in range(c["kv_heads"]):
            best = None
            for q in s["query"][i, k * group:(k + 1) * group].double():
                x = torch.maximum(q * bounds[:, k, 0], q * bounds[:, k, 1]).sum(dim=1)
                best = x if best is None else torch.maximum(best, x)
            ranked = sorted(range(n), key=lambda b, v=best.tolist(): (-v[b], b))
            chosen = set(forced)
            for b in ranked:
                if len(chosen) >= min(keep, n):
                    break
                chosen.add(b)
            row = sorted(chosen)
            selected[i, k, :len(row)] = torch.tensor(row)
            number[i, k] = len(row)
    return selected.int().cuda(), number.int().cuda()


def exact(case, seed):
    s = prepare(case, seed)
    ctx, new = _lengths(case)
    if case["op"] == "write":
        return _write_exact(s, ctx, new)
    if case["op"] == "bounds":
        return _bounds_exact(s, ctx, new)
    if case["op"] == "select":
        return _select_exact(s, ctx)
    return _decode_exact(s, ctx)
