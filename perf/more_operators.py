"""The operators that fill the paged caches, and those that read a prefix once for all who share it, as
cases that can be timed and compared.

- ``latent``: new tokens' latent vectors, normalised, their rotary part turned by the token's position, into
  the slots of a paged cache; the queries' rotary parts turned in the same call;
- ``index``: new tokens' indexer keys, normalised, turned and rounded (to 8 bits with a scale a key) into
  their cache; the indexer's queries likewise, with the scales that they got in the heads' weights;
- ``shared``: absorbed latent attention of rows in groups, the first tokens of a group's rows being the same
  cached ones, read once for all of them;
- ``behind``: expanded latent attention of a ragged batch of prompts behind keys that several of them share,
  which are there once.

``own`` false: plain torch operations in 32 bits. ``own`` true: the library's kernels.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
ROPE = 64
MOST8 = 448.0  # e4m3's largest number
LEAST = 2.0 ** -100  # a key whose largest element is below it is scaled as if that were this


def listed():
    return [
        # one decode step of 128 requests, the heads of one of several cards; latency is all of it
        dict(name="latent_decode", op="latent", requests=128, new=1, length=8192, heads=16, latent=512, page=64, pairs="near", norm=True, type="bf16"),
        # uneven prompts of odd lengths in half precision, the smaller latent vectors, halves turned
        dict(name="latent_ragged", op="latent", requests=5, new=777, length=3000, heads=24, latent=256, page=16, pairs="halves", norm=False, type="fp16"),
        # a prefill step of 16384 tokens with all 128 heads on this card: memory bound
        dict(name="latent_prefill", op="latent", requests=4, new=4096, length=16384, heads=128, latent=512, page=64, pairs="near", norm=True, type="bf16"),
        # the indexer's part of that decode step: 64 heads, 8-bit keys and queries
        dict(name="index_decode_fp8", op="index", requests=128, new=1, length=8192, heads=64, dim=128, page=64, pairs="halves", norm=True, type="bf16", to="fp8"),
        # prompts of odd lengths, keys kept as they come (16 bits)
        dict(name="index_ragged_fp16", op="index", requests=7, new=1001, length=5001, heads=32, dim=64, page=16, pairs="near", norm=True, type="fp16", to="fp16"),
        # the indexer's part of the prefill step
        dict(name="index_prefill_fp8", op="index", requests=4, new=4096, length=16384, heads=64, dim=128, page=64, pairs="halves", norm=True, type="bf16", to="fp8"),
        # 33 requests with three drafted tokens beside the last one: a request's four rows share all they read
        dict(name="shared_drafts", op="shared", groups=33, rows=4, shared=5001, own=0, even=False, heads=16, latent=512, page=64, type="fp16"),
        # 64 requests behind one system prompt of 16384 tokens, up to 1000 tokens of their own each, 16 heads
        dict(name="shared_decode", op="shared", groups=1, rows=64, shared=16384, own=1000, even=False, heads=16, latent=512, page=64, type="bf16"),
        # several prompts, each shared by an uneven number of requests
        dict(name="shared_groups", op="shared", groups=9, rows=13, shared=8192, own=700, even=False, heads=40, latent=512, page=16, type="bf16"),
        # samples of one long context, all 128 heads on this card: matrix-unit bound
        dict(name="shared_long", op="shared", groups=2, rows=16, shared=32768, own=257, even=False, heads=128, latent=512, page=64, type="bf16"),
        # short uneven prompts behind a shared one of odd length
        dict(name="behind_ragged", op="behind", groups=2, requests=4, rows=777, shared=2001, even=False, heads=16, type="fp16"),
        # 16 prompts of 512 tokens behind 16384 tokens that all of them share
        dict(name="behind_prefill", op="behind", groups=1, requests=16, rows=512, shared=16384, even=True, heads=16, type="bf16"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["latent", "index", "shared", "shared", "behind"])
    if op in ("latent", "index"):
        kind = rng.choice(["bf16", "fp16"])
        heads = rng.choice([1, 5, 8, 16, 24, 32, 64, 128] if op == "latent" else [8, 16, 32, 48, 64])
        tokens = _log_int(rng, 1, min(16384, (1 << 20) // heads))
        new = rng.choice([1, _log_int(rng, 1, tokens)])
        c = dict(op=op, requests=min(1024, max(1, tokens // new)), new=new, length=new + _log_int(rng, 1, 131072 - new), heads=heads, page=rng.choice([1, 16, 32, 64, 128]),
                 pairs=rng.choice(["near", "halves"]), norm=rng.random() < 0.7, type=kind)
        return dict(c, latent=rng.choice([256, 512])) if op == "latent" else dict(c, dim=rng.choice([64, 128]), to=rng.choice(["fp8", kind]))
    if op == "shared":
        heads, latent = rng.choice([1, 8, 16, 16, 24, 32, 64, 128]), rng.choice([256, 512, 512])
        shared = _log_int(rng, 64, 65536)
        rows = rng.choice([1, 2, 4, _log_int(rng, 1, max(1, min(128, (1 << 25) // (shared * heads))))])
        groups = _log_int(rng, 1, max(1, min(64, (1 << 26) // (shared * heads * rows), (1 << 19) // shared)))
        # drafted rows share all they read; requests behind a prompt have tokens of their own
        tokens = 0 if rows <= 8 and rng.random() < 0.4 else _log_int(rng, 1, max(1, min(4096, (1 << 18) // (groups * rows))))
        return dict(op=op, groups=groups, rows=rows, shared=shared, own=tokens, even=rng.random() < 0.3, heads=heads, latent=latent, page=rng.choice([1, 16, 64]), type=rng.choice(["bf16", "fp16"]))
    groups, requests, rows = rng.randint(1, 3), rng.randint(1, 8), _log_int(rng, 1, 1000)
    shared = _log_int(rng, 1, max(1, min(16384, (1 << 26) // (groups * requests * rows))))
    return dict(op=op, groups=groups, requests=requests, rows=rows, shared=shared, even=rng.random() < 0.3, heads=rng.choice([1, 3, 8, 16]), type=rng.choice(["bf16", "fp16"]))


# ---------------------------------------------------------------------------------------------------------
# Inputs


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)


def _normal(g, kind, *shape):
    return torch.empty(shape, device=DEVICE, dtype=kind).normal_(generator=g)


def _spread(c, what, count, low, high, even):
    """`count` lengths of a case: all `high`, or uniform over [low, high] with one of them `high`. They go by
    the case alone, so that the outputs' shapes are the same for every seed."""
    if even or low >= high:
        return [high] * count
    r = random.Random("%s of %s" % (what, sorted((k, v) for k, v in c.items() if k != "name")))
    return [high] + [r.randint(low, high) for _ in range(count - 1)]


def _dealt(lengths, g):
    """The lengths as the seed deals them out."""
    return torch.tensor(lengths, dtype=torch.int64, device=DEVICE)[torch.randperm(len(lengths), generator=g, device=DEVICE)]


def _new(c):
    return _spread(c, "new", c["requests"], 1, c["new"], c["new"] == 1)


def _group_rows(c):
    return _spread(c, "rows", c["groups"], 1, c["rows"], c["even"] or c["own"] == 0)


def _shared(c):
    """Tokens that each group shares; whole pages where its rows go on with pages of their own."""
    lens = _spread(c, "shared", c["groups"], c["shared"] // 2 + 1, c["shared"], c["even"])
    return lens if c["own"] == 0 else [max(0, n // c["page"] * c["page"]) for n in lens]


def _own(c):
    return [0] * sum(_group_rows(c)) if c["own"] == 0 else _spread(c, "own", sum(_group_rows(c)), 1, c["own"], c["even"])


def _behind(c):
    """(new tokens of each request, shared tokens of each group)."""
    return (_spread(c, "rows", c["groups"] * c["requests"], 1, c["rows"], c["even"]),
            _spread(c, "shared", c["groups"], c["shared"] // 2 + 1, c["shared"], c["even"]))


def _i32(v):
    return v.to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    return dict(case, **{"latent": _prepare_latent, "index": _prepare_index, "shared": _prepare_shared, "behind": _prepare_behind}[case["op"]](case, g))


def _prepare_tokens(c, g):
    """A step's new tokens: slots and windows as the page maps give them (empty rows behind), the angles' table."""
    n, page = c["requests"], c["page"]
    new = _dealt(_new(c), g)
    first = torch.randint(0, c["length"] - c["new"] + 1, (n,), generator=g, device=DEVICE)
    total = sum(_new(c))
    tokens = -(-total // 8) * 8
    request = torch.repeat_interleave(torch.arange(n, device=DEVICE), new, output_size=total)
    position = first[request] + torch.arange(total, device=DEVICE) - (new.cumsum(0) - new)[request]
    width = -(-c["new"] // page) + 1
    # page 0 is nobody's
    table = torch.randperm(n * width, generator=g, device=DEVICE).view(n, width) + 1
    slots = table[request, position // page - first[request] // page] * page + position % page
    empty = torch.zeros(tokens - total, dtype=torch.int64, device=DEVICE)
    angle = torch.arange(c["length"], dtype=torch.float64, device=DEVICE)[:, None] * 10000.0 ** (-torch.arange(ROPE // 2, dtype=torch.float64, device=DEVICE) / (ROPE // 2))
    return dict(slots=_i32(torch.cat([slots, empty - 1])), row_lens=_i32(torch.cat([position + 1, empty])), tokens=tokens, pages=n * width + 1,
                cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float())


def _prepare_latent(c, g):
    s, kind, dim = _prepare_tokens(c, g), TYPES[c["type"]], c["latent"] + ROPE
    # what a projection leaves: tokens of different sizes
    s["latent_in"] = (_rand(g, s["tokens"], dim) * (0.5 + torch.rand(s["tokens"], 1, generator=g, device=DEVICE))).to(kind)
    s["weight"] = 1.0 + 0.1 * _rand(g, c["latent"]) if c["norm"] else None
    s["cache"] = _normal(g, kind, s["pages"], c["page"], dim)
    q = _normal(g, kind, s["tokens"], c["heads"], 128 + ROPE)
    s["q_rope"] = q[..., 128:]
    # prompts: their vectors go on to the keys' and values' projections; decode: the queries' part beside the absorbed one
    s["out"] = torch.zeros_like(s["latent_in"]) if c["new"] > 1 else None
    s["q_out"] = None if c["new"] > 1 else torch.zeros(s["tokens"], c["heads"], dim, device=DEVICE, dtype=kind)[..., c["latent"]:]
    return s


def _prepare_index(c, g):
    s, kind = _prepare_tokens(c, g), TYPES[c["type"]]
    s["keys"] = (_rand(g, s["tokens"], c["dim"]) * (0.5 + torch.rand(s["tokens"], 1, generator=g, device=DEVICE))).to(kind)
    s["weight"] = 1.0 + 0.1 * _rand(g, c["dim"]) if c["norm"] else None
    s["bias"] = 0.1 * _rand(g, c["dim"]) if c["norm"] else None
    s["index_keys"] = _normal(g, kind, s["pages"], c["page"], c["dim"]).to(TYPES[c["to"]])
    s["scales"] = torch.rand(s["pages"], c["page"], generator=g, device=DEVICE) if c["to"] == "fp8" else None
    s["q"] = _normal(g, kind, s["tokens"], c["heads"], c["dim"])
    s["weights"] = _rand(g, s["tokens"], c["heads"]) * (c["heads"] * c["dim"]) ** -0.5 if c["to"] == "fp8" else None
    return s


def _prepare_shared(c, g):
    heads, page, kind, dim = c["heads"], c["page"], TYPES[c["type"]], c["latent"] + ROPE
    group_rows, shared = _dealt(_group_rows(c), g), _dealt(_shared(c), g)
    rows = sum(_group_rows(c))
    group = torch.repeat_interleave(torch.arange(c["groups"], device=DEVICE), group_rows, output_size=rows)
    starts = torch.cat([group_rows.new_zeros(1), group_rows.cumsum(0)])
    nth = torch.arange(rows, device=DEVICE) - starts[group]
    s = dict(group_starts=_i32(starts), shared_lens=_i32(shared), group=group, nth=nth, most=c["rows"], scale=192 ** -0.5 * 0.5)
    whole = -(-c["shared"] // page)
    if c["own"] == 0:
        # a request's drafted rows: each sees one token more than the one before it
        lens = (shared[group] - group_rows[group] + 1 + nth).clamp(min=0)
        width, pages = whole, c["groups"] * whole
        table = torch.randperm(pages, generator=g, device=DEVICE).view(c["groups"], width)
        s["table_rows"] = _i32(group)
    else:
        lens = shared[group] + _dealt(_own(c), g)
        more = -(-c["own"] // page)
        width, pages = whole + more, c["groups"] * whole + rows * more
        pool = torch.randperm(pages, generator=g, device=DEVICE)
        column = torch.arange(width, device=DEVICE)
        held = (shared // page)[group][:, None]
        own_at = c["groups"] * whole + torch.arange(rows, device=DEVICE)[:, None] * more + (column - held).clamp(0, more - 1)
        table = pool[torch.where(column < held, group[:, None] * whole + column.clamp(max=whole - 1), own_at)]
        s["table_rows"] = None
    s["cache"] = _normal(g, kind, pages, page, dim)
    return dict(s, q=_rand(g, rows, heads, dim).to(kind), seq_lens=_i32(lens), table=_i32(table))


def _prepare_behind(c, g):
    heads, kind = c["heads"], TYPES[c["type"]]
    rows, shared = (_dealt(v, g) for v in _behind(c))
    requests = c["groups"] * c["requests"]
    # the shared tokens' keys come first, then each request's own
    ends = shared.cumsum(0)
    group = torch.arange(requests, device=DEVICE) // c["requests"]
    q_starts = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
    k_starts = q_starts + sum(_behind(c)[1])
    tq = sum(_behind(c)[0])
    tk = tq + sum(_behind(c)[1])
    kv = _normal(g, kind, tk, heads, 256)
    return dict(q=_normal(g, kind, tq, heads, 192), k=kv[..., :128], v=kv[..., 128:], k_rope=_normal(g, kind, tk, 64), q_starts=_i32(q_starts), k_starts=_i32(k_starts),
                shared_starts=_i32((ends - shared)[group]), shared_lens=_i32(shared[group]), max_q=max(_behind(c)[0]), max_shared=max(_behind(c)[1]), scale=192 ** -0.5)


# ---------------------------------------------------------------------------------------------------------
# One pass


def run(s):
    if own:
        return _run_own(s)
    return {"latent": _plain_latent, "index": _plain_index, "shared": _plain_shared, "behind": _plain_behind}[s["op"]](s)


def _run_own(s):
    import row_top_selection_amd as dt

    near = s.get("pairs") == "near"
    if s["op"] == "latent":
        q = dt.append_latent(s["latent_in"], s["cache"], s["slots"], s["row_lens"], s["cos_sin"], weight=s["weight"], q_rope=s["q_rope"], q_out=s["q_out"], out=s["out"], interleaved=near)
        return dict(cache=s["cache"], q=q, out=s["out"])
    if s["op"] == "index":
        q, weights = dt.append_index(s["keys"], s["index_keys"], s["slots"], s["row_lens"], s["cos_sin"], key_scales=s["scales"], weight=s["weight"], bias=s["bias"],
                                     q=s["q"], weights=s["weights"], interleaved=near)
        return dict(index_keys=s["index_keys"], scales=s["scales"], q=q, weights=weights)
    if s["op"] == "shared":
        out, lse = dt.attend_shared(s["q"], s["cache"], s["seq_lens"], s["table"], s["group_starts"], s["shared_lens"], s["latent"], s["scale"], table_rows=s["table_rows"],
                                    max_shared_len=s["shared"], max_own_len=s["own"])
        return dict(out=out, lse=lse)
    out, lse = dt.attend_expanded_shared(s["q"], s["k"], s["v"], s["k_rope"], s["q_starts"], s["k_starts"], s["shared_starts"], s["shared_lens"], s["scale"],
                                         max_keys=s["max_shared"] + s["max_q"])
    return dict(out=out, lse=lse)


def _turned(x, s):
    """x [tokens, ..., 64] turned by its token's angles; tokens without a position as they are."""
    position = s["row_lens"].long() - 1
    at = s["cos_sin"][position.clamp(0, s["cos_sin"].shape[0] - 1)]
    at = at.view(at.shape[0], *[1] * (x.dim() - 2), ROPE)
    there = ((position >= 0) & (position < s["cos_sin"].shape[0])).view(-1, *[1] * (x.dim() - 1))
    cos, sin = torch.where(there, at[..., :ROPE // 2], 1.0), torch.where(there, at[..., ROPE // 2:], 0.0)
    if s["pairs"] == "near":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _put(cache, slots, values):
    """values into their slots; a token without one writes back what slot 0, which is nobody's, holds."""
    at = slots.clamp(min=0).long()
    there = (slots >= 0).view(-1, *[1] * (values.dim() - 1))
    bits = (lambda t: t.view(torch.uint8)) if cache.dtype == TYPES["fp8"] else (lambda t: t)
    bits(cache).index_copy_(0, at, torch.where(there, bits(values), bits(cache)[at]))


def _plain_latent(s):
    x, latent = s["latent_in"].float(), s["latent"]
    body = x[:, :latent]
    if s["weight"] is not None:
        body = body * torch.rsqrt(body.square().mean(-1, keepdim=True) + 1e-6) * s["weight"]
    x = torch.cat([body, _turned(x[:, latent:], s)], -1).to(s["cache"].dtype)
    _put(s["cache"].view(-1, latent + ROPE), s["slots"], x)
    if s["out"] is not None:
        s["out"].copy_(x)
    q = _turned(s["q_rope"].float(), s).to(s["q_rope"].dtype)
    return dict(cache=s["cache"], q=q if s["q_out"] is None else s["q_out"].copy_(q), out=s["out"])


def _eight(x):
    """x as 8-bit numbers and the factor of each of its last dimension's vectors."""
    scale = x.abs().amax(-1, keepdim=True).clamp(min=LEAST) / MOST8
    return (x / scale).clamp(-MOST8, MOST8).to(TYPES["fp8"]), scale.squeeze(-1)


def _plain_index(s):
    x, dim = s["keys"].float(), s["dim"]
    if s["weight"] is not None:
        x = x - x.mean(-1, keepdim=True)
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["weight"] + s["bias"]
    x = torch.cat([_turned(x[:, :ROPE], s), x[:, ROPE:]], -1)
    q = s["q"].float()
    q = torch.cat([_turned(q[..., :ROPE], s), q[..., ROPE:]], -1)
    if s["scales"] is None:
        _put(s["index_keys"].view(-1, dim), s["slots"], x.to(s["index_keys"].dtype))
        return dict(index_keys=s["index_keys"], scales=None, q=q.to(s["q"].dtype), weights=None)
    x, scale = _eight(x)
    _put(s["index_keys"].view(-1, dim), s["slots"], x)
    _put(s["scales"].view(-1), s["slots"], scale)
    q, scale = _eight(q)
    return dict(index_keys=s["index_keys"], scales=s["scales"], q=q, weights=s["weights"] * scale)


def _softmax(scores, seen):
    """Weights and log-sum-exp over the last axis; rows that see nothing have zeros and -inf."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    weights = torch.exp(scores - top)
    total = weights.sum(-1, keepdim=True)
    return weights / total.clamp(min=1e-38), (top + torch.log(total)).squeeze(-1)


def _plain_shared(s):
    q, cache, page, latent = s["q"].float() * s["scale"], s["cache"].view(-1, s["cache"].shape[-1]), s["page"], s["latent"]
    rows, heads, dim = q.shape
    groups, group, nth, most = s["groups"], s["group"], s["nth"], s["most"]
    table, lens, device = s["table"].long(), s["seq_lens"].long(), q.device
    table_rows = torch.arange(rows, device=device) if s["table_rows"] is None else s["table_rows"].long()
    shared = s["shared_lens"].long()
    # a group's shared vectors once, against all of its rows' heads
    j = torch.arange(s["shared"], device=device)
    first = table_rows[s["group_starts"][:-1].long()]
    vectors = cache[table[first][:, j // page] * page + j % page].float()  # [groups, shared, dim]
    packed = q.new_zeros(groups, most, heads, dim)
    packed[group, nth] = q
    dots = torch.matmul(packed.view(groups, most * heads, dim), vectors.transpose(1, 2)).view(groups, most, heads, -1)
    seen = j < torch.minimum(shared[group], lens)[:, None]
    scores = dots[group, nth]
    if s["own"]:
        i = torch.arange(s["own"], device=device)
        at = (shared[group][:, None] + i).clamp(max=table.shape[1] * page - 1)
        mine = cache[table[table_rows].gather(1, at // page) * page + at % page].float()  # [rows, own, dim]
        scores = torch.cat([scores, torch.matmul(q, mine.transpose(1, 2))], -1)
        seen = torch.cat([seen, shared[group][:, None] + i < lens[:, None]], -1)
    weights, lse = _softmax(scores, seen[:, None])
    packed = weights.new_zeros(groups, most, heads, s["shared"])
    packed[group, nth] = weights[..., :s["shared"]]
    out = torch.matmul(packed.view(groups, most * heads, -1), vectors[..., :latent]).view(groups, most, heads, latent)[group, nth]
    if s["own"]:
        out = out + torch.matmul(weights[..., s["shared"]:], mine[..., :latent])
    return dict(out=out.to(s["q"].dtype), lse=lse)


def _plain_behind(s):
    q_starts, k_starts = s["q_starts"].long(), s["k_starts"].long()
    lens, behind = q_starts.diff(), s["shared_lens"].long()
    row = torch.arange(s["max_q"], device=q_starts.device)
    column = torch.arange(s["max_shared"] + s["max_q"], device=q_starts.device)
    q_at = (q_starts[:-1, None] + row).clamp(max=s["q"].shape[0] - 1)
    k_at = torch.where(column < behind[:, None], s["shared_starts"].long()[:, None] + column, k_starts[:-1, None] + column - behind[:, None]).clamp(max=s["k"].shape[0] - 1)
    q = s["q"][q_at].float().transpose(1, 2)  # [requests, heads, rows, 192]
    k = s["k"][k_at].float().transpose(1, 2)
    rope = s["k_rope"][k_at].float()[:, None]
    v = s["v"][k_at].float().transpose(1, 2)
    scores = torch.matmul(q[..., :128], k.transpose(2, 3)) + torch.matmul(q[..., 128:], rope.transpose(2, 3))
    seen = column <= row[:, None] + behind[:, None, None]
    weights, lse = _softmax(scores * s["scale"], seen[:, None])
    out = torch.matmul(weights, v).transpose(1, 2)
    real = row < lens[:, None]
    return dict(out=out[real].to(s["q"].dtype), lse=lse.transpose(1, 2)[real])


# ---------------------------------------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    c = case
    if c["op"] in ("latent", "index"):
        tokens, heads = sum(_new(c)), c["heads"]
        words = 4 * tokens * (2 + ROPE)  # slot, window, angles
        if c["op"] == "latent":
            dim = c["latent"] + ROPE
            moved = 2 * tokens * (dim * (3 if c["new"] > 1 else 2) + 2 * heads * ROPE)
            return {"bytes": words + moved + (4 * c["latent"] if c["norm"] else 0), "flops": tokens * (4 * c["latent"] + 3 * ROPE * (1 + heads))}
        dim, size = c["dim"], 1 if c["to"] == "fp8" else 2
        scales = tokens * (4 + 8 * heads) if size == 1 else 0
        return {"bytes": words + scales + tokens * (1 + heads) * dim * (2 + size) + (8 * dim if c["norm"] else 0), "flops": tokens * (1 + heads) * 6 * dim}
    if c["op"] == "shared":
        heads, dim = c["heads"], c["latent"] + ROPE
        rows = sum(_group_rows(c))
        if c["own"] == 0:
            # row i of a group's m sees m - 1 - i tokens fewer than the last
            pairs = sum(max(0, n - i) for n in _shared(c) for i in range(c["rows"]))
        else:
            # lengths are dealt out by the seed: rows of a group times its tokens, in the mean
            pairs = rows * sum(_shared(c)) / c["groups"] + sum(_own(c))
        tokens = sum(_shared(c)) + sum(_own(c))
        return {"bytes": 2 * (tokens * dim + rows * heads * (dim + c["latent"])) + 4 * (rows * heads + tokens / c["page"]), "flops": pairs * heads * 2 * (dim + c["latent"])}
    rows, shared = _behind(c)
    heads, keys = c["heads"], sum(rows) + sum(shared)
    pairs = sum(rows) * sum(shared) / c["groups"] + sum(n * (n + 1) // 2 for n in rows)
    return {"bytes": 2 * (heads * (sum(rows) * (192 + 128) + keys * 256) + keys * 64) + 4 * sum(rows) * heads, "flops": pairs * heads * 2 * (192 + 128)}


# ---------------------------------------------------------------------------------------------------------
# The operators' definitions, in 64 bits; numbers kept in fewer bits are given as they are before their rounding


def exact(case, seed):
    s = prepare(case, seed)
    return {"latent": _exact_latent, "index": _exact_index, "shared": _exact_shared, "behind": _exact_behind}[case["op"]](s)


def _exact_turned(x, s):
    """The pairs as complex numbers, multiplied by those of the angles (as the table has them)."""
    table = torch.complex(s["cos_sin"][:, :ROPE // 2].double(), s["cos_sin"][:, ROPE // 2:].double())
    turn = torch.ones(x.shape[0], ROPE // 2, dtype=torch.complex128, device=x.device)
    real = s["row_lens"] > 0
    turn[real] = table[s["row_lens"][real].long() - 1]
    out = torch.empty_like(x)
    for i in range(ROPE // 2):
        a, b = (2 * i, 2 * i + 1) if s["pairs"] == "near" else (i, i + ROPE // 2)
        z = torch.complex(x[..., a], x[..., b]) * turn[:, i].view(-1, *[1] * (x.dim() - 2))
        out[..., a], out[..., b] = z.real, z.imag
    return out


def _exact_latent(s):
    x, latent = s["latent_in"].double(), s["latent"]
    if s["weight"] is not None:
        x[:, :latent] /= (x[:, :latent].pow(2).sum(1, keepdim=True) / latent + 1e-6).sqrt()
        x[:, :latent] *= s["weight"].double()
    x[:, latent:] = _exact_turned(x[:, latent:], s)
    cache = s["cache"].double()
    real = s["slots"] >= 0
    slot = s["slots"][real].long()
    cache[slot // s["page"], slot % s["page"]] = x[real]
    return dict(cache=cache, q=_exact_turned(s["q_rope"].double(), s), out=None if s["out"] is None else x)


def _exact_index(s):
    x, q = s["keys"].double(), s["q"].double()
    if s["weight"] is not None:
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        x = (x - mean) / (var + 1e-6).sqrt() * s["weight"].double() + s["bias"].double()
    x[:, :ROPE] = _exact_turned(x[:, :ROPE], s)
    q[..., :ROPE] = _exact_turned(q[..., :ROPE], s)
    keys, real = s["index_keys"].double(), s["slots"] >= 0
    slot = s["slots"][real].long()
    at = (slot // s["page"], slot % s["page"])
    if s["scales"] is None:
        keys[at] = x[real]
        return dict(index_keys=keys, scales=None, q=q, weights=None)
    scales = s["scales"].double()
    scales[at] = x[real].abs().max(1).values / MOST8
    keys[at] = x[real] / scales[at][:, None]
    by = q.abs().max(2).values / MOST8
    return dict(index_keys=keys, scales=scales, q=q / by[..., None], weights=s["weights"].double() * by)


def _exact_shared(s):
    page, latent = s["page"], s["latent"]
    q, cache = s["q"].double(), s["cache"].view(-1, s["cache"].shape[-1])
    starts, shared, lens = s["group_starts"].tolist(), s["shared_lens"].tolist(), s["seq_lens"].tolist()
    outs, sums = [], []
    for g in range(s["groups"]):
        for r in range(starts[g], starts[g + 1]):
            line = s["table"][r if s["table_rows"] is None else int(s["table_rows"][r])].long()
            j = torch.arange(lens[r], device=q.device)
            x = cache[line[j // page] * page + j % page].double()
            logits = (q[r] @ x.T) * s["scale"]
            sums.append(torch.logsumexp(logits, -1))
            outs.append(torch.softmax(logits, -1) @ x[:, :latent])
    return dict(out=torch.stack(outs), lse=torch.stack(sums))


def _exact_behind(s):
    q_at, k_at = s["q_starts"].tolist(), s["k_starts"].tolist()
    out = torch.zeros(s["q"].shape[0], s["heads"], 128, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["q"].shape[0], s["heads"], dtype=torch.float64, device=s["q"].device)
    for r in range(len(q_at) - 1):
        a, b, n = q_at[r], q_at[r + 1], q_at[r + 1] - q_at[r]
        first, before = int(s["shared_starts"][r]), int(s["shared_lens"][r])
        where = torch.cat([torch.arange(first, first + before, device=out.device), torch.arange(k_at[r], k_at[r + 1], device=out.device)])
        hidden = torch.arange(before + n, device=out.device) > torch.arange(n, device=out.device)[:, None] + before
        rope = s["k_rope"][where].double()
        for h in range(s["heads"]):
            logits = (s["q"][a:b, h].double() @ torch.cat([s["k"][where, h].double(), rope], dim=1).T) * s["scale"]
            logits[hidden] = -math.inf
            lse[a:b, h] = torch.logsumexp(logits, -1)
            out[a:b, h] = torch.softmax(logits, -1) @ s["v"][where, h].double()
    return dict(out=out, lse=lse)
