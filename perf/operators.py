"""The serving operators around the top-k, as cases that can be timed and compared.

Four operators, in the order a serving step uses them:

- ``maps``: from request lengths, the pages a step takes, the cache slot of each new token, and the
  top-k's row arguments (table row and window length of each token);
- ``scores``: the indexer's scores that the top-k selects from, sum over heads of weight * relu(q . k), over a
  paged key cache or over flattened keys;
- ``attend``: latent attention in its absorbed form (all heads read one shared latent vector a token), over
  the selected cache slots or over a request's whole window;
- ``expand``: latent attention in its expanded form (keys and values of each head, one rotary key shared by
  the heads), causal, over ragged batches.

``own`` false: plain torch operations in 32 bits. ``own`` true: the library's kernels.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}


def listed():
    return [
        # one decode step of 128 requests (the paged decode workload's batch): latency is all of it
        dict(name="maps_decode", op="maps", requests=128, new=1, length=8192, page=64),
        # a large prefill step of uneven requests: about half a million tokens get their slots
        dict(name="maps_prefill", op="maps", requests=256, new=4096, length=32768, page=64),
        # the smallest indexer call: 4 short requests of up to 3000 tokens, 64 indexer heads, 8-bit keys
        dict(name="scores_small_fp8", op="scores", form="paged", requests=4, rows=1, length=3000, even=False, heads=64, dim=128, page=64, type="fp8"),
        # paged decode, 128 rows of 8192: every key is read once, memory bound
        dict(name="scores_decode_bf16", op="scores", form="paged", requests=128, rows=1, length=8192, even=True, heads=64, dim=128, page=64, type="bf16"),
        # prefill extend: 4 requests of 1024 query rows over 16384 flattened keys each, matrix-unit bound
        dict(name="scores_extend_fp8", op="scores", form="ragged", requests=4, rows=1024, length=16384, even=True, heads=64, dim=128, page=1, type="fp8"),
        # one token for each of 4 short requests, heads of one of several cards: latency
        dict(name="attend_selected_small", op="attend", form="slots", requests=4, rows=1, length=3000, k=512, heads=16, latent=512, rope=64, page=64, type="bf16"),
        # paged decode behind the top-k: 128 rows, 2048 selected slots each, all 128 heads on this card
        dict(name="attend_selected_decode", op="attend", form="slots", requests=128, rows=1, length=8192, k=2048, heads=128, latent=512, rope=64, page=64, type="bf16"),
        # prefill rows behind the top-k: each of 4 x 256 rows has its own selection out of 16384 tokens
        dict(name="attend_selected_extend", op="attend", form="slots", requests=4, rows=256, length=16384, k=2048, heads=64, latent=512, rope=64, page=64, type="bf16"),
        # a long context read whole: 8 rows of 131072 tokens, 16 heads; few rows, so the long axis is split
        dict(name="attend_paged_long", op="attend", form="paged", requests=8, rows=1, length=131072, k=0, heads=16, latent=512, rope=64, page=64, type="bf16"),
        # two tokens a request (a drafted token beside the last one) over uneven windows in half precision
        dict(name="attend_paged_two_rows", op="attend", form="paged", requests=33, rows=2, length=5001, k=0, heads=40, latent=512, rope=64, page=16, type="fp16"),
        # a ragged prefill of uneven, odd lengths from nothing
        dict(name="expand_ragged", op="expand", requests=5, rows=777, past=0, even=False, heads=16, type="fp16"),
        # prefill extend: 4 requests of 1024 new tokens behind 15360 earlier ones
        dict(name="expand_extend", op="expand", requests=4, rows=1024, past=15360, even=True, heads=16, type="bf16"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["maps", "scores", "scores", "attend", "attend", "attend", "expand"])
    if op == "maps":
        requests = _log_int(rng, 1, 1024)
        length = _log_int(rng, 1, 65536)
        new = min(length, rng.choice([1, 2, _log_int(rng, 1, 4096)]), max(1, (1 << 20) // requests))
        return dict(op=op, requests=requests, new=new, length=length, page=rng.choice([1, 16, 32, 64, 128]) if requests * length < 1 << 24 else 64)
    if op == "scores":
        heads, dim, kind = rng.choice([8, 16, 32, 48, 64]), rng.choice([64, 128]), rng.choice(["bf16", "fp16", "fp8"])
        if rng.random() < 0.6:
            rows = rng.choice([1, 1, 2, 4])
            length = _log_int(rng, 1, 131072)
            requests = _log_int(rng, 1, max(1, min(256, (1 << 20) // (length * rows))))
            return dict(op=op, form="paged", requests=requests, rows=rows, length=max(rows, length), even=rng.random() < 0.3, heads=heads, dim=dim, page=rng.choice([1, 16, 64, 128]), type=kind)
        requests, length = rng.randint(1, 4), _log_int(rng, 64, 16384)
        return dict(op=op, form="ragged", requests=requests, rows=min(length, _log_int(rng, 1, 1024)), length=length, even=rng.random() < 0.3, heads=heads, dim=dim, page=1, type=kind)
    if op == "attend":
        heads, kind, latent = rng.choice([1, 8, 16, 24, 32, 64, 128]), rng.choice(["bf16", "fp16"]), rng.choice([256, 512, 512])
        page = rng.choice([1, 16, 64])
        if rng.random() < 0.6:
            k = _log_int(rng, 1, 2048)
            rows = _log_int(rng, 1, min(1024, (1 << 21) // k))
            requests = rng.choice([1, 2, 4]) if rows >= 4 else 1
            return dict(op=op, form="slots", requests=requests, rows=max(1, rows // requests), length=max(rows, _log_int(rng, 1, 16384)), k=k, heads=heads, latent=latent, rope=64, page=page, type=kind)
        rows, length = rng.choice([1, 1, 2, 3]), _log_int(rng, 4, 131072)
        return dict(op=op, form="paged", requests=_log_int(rng, 1, max(1, min(128, (1 << 19) // length))), rows=rows, length=length, k=0, heads=heads, latent=latent, rope=64, page=page, type=kind)
    requests, rows = rng.randint(1, 6), _log_int(rng, 1, 1500)
    past = rng.choice([0, 0, _log_int(rng, 1, 12000)])
    heads = rng.choice([1, 3, 8, 16])
    return dict(op=op, requests=requests, rows=rows, past=min(past, max(0, (1 << 26) // (rows * requests) - rows)), even=rng.random() < 0.3, heads=heads, type=rng.choice(["bf16", "fp16"]))


# ---------------------------------------------------------------------------------------------------------
# Inputs


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)


def _spread(c, what, low, high, even):
    """A case's lengths, one a request: all `high`, or uniform over [low, high] with one of them `high`.
    They go by the case alone, so that its sums (and with them the outputs' shapes) are the same for every seed."""
    if even or low >= high:
        return [high] * c["requests"]
    r = random.Random("%s of %s" % (what, sorted((k, v) for k, v in c.items() if k != "name")))
    return [high] + [r.randint(low, high) for _ in range(c["requests"] - 1)]


def _dealt(lengths, g):
    """The lengths as the seed deals them to the requests."""
    return torch.tensor(lengths, dtype=torch.int64, device=DEVICE)[torch.randperm(len(lengths), generator=g, device=DEVICE)]


def _new(c):
    return _spread(c, "new", 1, c["new"], c["new"] == 1)


def _seen(c):
    """Tokens that a request's last row sees, where the case has one `length`."""
    if c["op"] == "scores":
        return _spread(c, "length", min(c["rows"], c["length"]), c["length"], c["even"])
    return _spread(c, "length", 1, c["length"], c["form"] == "slots" or c["length"] > 65536)


def _expand_lengths(c):
    """(new, earlier) tokens of each request."""
    return list(zip(_spread(c, "rows", 1, c["rows"], c["even"]), _spread(c, "past", 0, c["past"], c["even"])))


def _tables(g, requests, width):
    """Page tables of requests that share one pool: [requests, width], no page twice."""
    return torch.randperm(requests * width, generator=g, device=DEVICE).view(requests, width).to(torch.int32)


def _i32(v):
    return v.to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    return dict(case, **{"maps": _prepare_maps, "scores": _prepare_scores, "attend": _prepare_attend, "expand": _prepare_expand}[case["op"]](case, g))


def _prepare_maps(c, g):
    n, page = c["requests"], c["page"]
    new = _dealt(_new(c), g)
    lens = new + torch.randint(0, c["length"] - c["new"] + 1, (n,), generator=g, device=DEVICE)
    width = -(-c["length"] // page)
    pool = torch.randperm(2 * n * width, generator=g, device=DEVICE).to(torch.int32)
    table = pool[: n * width].view(n, width).clone()
    held = (lens - new + page - 1) // page
    table[torch.arange(width, device=DEVICE) >= held[:, None]] = -1
    # a program launches for the step's token count, rounded up to the size that its graph was captured for
    tokens = -(-sum(_new(c)) // 64) * 64
    return dict(seq_lens=_i32(lens), new_lens=None if c["new"] == 1 else _i32(new), table=table, free=pool[n * width:].clone(), tokens=tokens)


def _prepare_scores(c, g):
    n, m, heads, dim, page, kind = c["requests"], c["rows"], c["heads"], c["dim"], c["page"], TYPES[c["type"]]
    total = n * m
    lens = _dealt(_seen(c), g)
    # the last of a request's rows sees all of its tokens, the one before one fewer
    row_lens = (lens[:, None] - (m - 1) + torch.arange(m, device=DEVICE)).clamp(min=0).view(-1)
    s = dict(q=_rand(g, total, heads, dim).to(kind), weights=_rand(g, total, heads) * (heads * dim) ** -0.5, seq_lens=_i32(row_lens), scales=None)
    if c["form"] == "paged":
        width = -(-c["length"] // page)
        s["table"] = _tables(g, n, width)
        s["table_rows"] = None if m == 1 else _i32(torch.arange(total, device=DEVICE) // m)
        s["keys"] = _rand(g, n * width, page, dim).to(kind)
        columns = -(-c["length"] // 4) * 4
    else:
        ends = lens.cumsum(0)
        s["request_starts"] = ends - lens
        s["starts"] = _i32(s["request_starts"].repeat_interleave(m))
        s["keys"] = _rand(g, int(ends[-1]), dim).to(kind)
        columns = -(-int(ends[-1]) // 4) * 4
    if c["type"] == "fp8":
        s["scales"] = torch.rand(s["keys"].shape[:-1], generator=g, device=DEVICE) + 0.5
    # the score buffer of a serving program: what lies outside the windows is left as it is
    s["out"] = torch.full((total, columns), -math.inf, device=DEVICE)
    return s


def _prepare_attend(c, g):
    n, m, heads, page, kind = c["requests"], c["rows"], c["heads"], c["page"], TYPES[c["type"]]
    dim, total = c["latent"] + c["rope"], n * m
    width = -(-c["length"] // page)
    table = _tables(g, n, width)
    # a latent vector is normalised to unit variance; its rotary part is of the same order
    cache = torch.empty(n * width, page, dim, device=DEVICE, dtype=kind).normal_(generator=g)
    s = dict(q=_rand(g, total, heads, dim).to(kind), cache=cache, scale=192 ** -0.5 * 0.5)
    lens = _dealt(_seen(c), g)
    row_lens = (lens[:, None] - (m - 1) + torch.arange(m, device=DEVICE)).clamp(min=0).view(-1)
    table_rows = torch.arange(total, device=DEVICE) // m
    if c["form"] == "paged":
        return dict(s, table=table, seq_lens=_i32(row_lens), table_rows=None if m == 1 else _i32(table_rows), max_len=c["length"])
    # what the top-k leaves: distinct positions in no order, then -1 where a row has fewer than k
    k = c["k"]
    slots = torch.full((total, k), -1, dtype=torch.int32, device=DEVICE)
    take = min(k, c["length"])
    for at in range(0, total, 512):
        rows = slice(at, min(total, at + 512))
        key = torch.rand(table_rows[rows].numel(), c["length"], generator=g, device=DEVICE)
        key[torch.arange(c["length"], device=DEVICE) >= row_lens[rows, None]] = -1.0
        value, position = key.topk(take, dim=1)
        page_of = table[table_rows[rows]].long().gather(1, position // page)
        slots[rows, :take] = torch.where(value >= 0, page_of * page + position % page, -1).to(torch.int32)
    return dict(s, slots=slots)


def _prepare_expand(c, g):
    n, heads, kind = c["requests"], c["heads"], TYPES[c["type"]]
    lens = torch.tensor(_expand_lengths(c), device=DEVICE)[torch.randperm(n, generator=g, device=DEVICE)]
    q_lens, k_lens = lens[:, 0], lens.sum(1)
    q_starts = torch.cat([q_lens.new_zeros(1), q_lens.cumsum(0)])
    k_starts = torch.cat([k_lens.new_zeros(1), k_lens.cumsum(0)])
    tq, tk = int(q_starts[-1]), int(k_starts[-1])
    # keys and values come out of one projection, side by side
    kv = _rand(g, tk, heads, 256).to(kind)
    return dict(q=_rand(g, tq, heads, 192).to(kind), k=kv[..., :128], v=kv[..., 128:], k_rope=_rand(g, tk, 64).to(kind),
                q_starts=_i32(q_starts), k_starts=_i32(k_starts), max_q=int(q_lens.max()), max_k=int(k_lens.max()), scale=192 ** -0.5)


# ---------------------------------------------------------------------------------------------------------
# One pass


def run(s):
    if own:
        return _run_own(s)
    return {"maps": _plain_maps, "scores": _plain_scores, "attend": _plain_attend, "expand": _plain_expand}[s["op"]](s)


def _run_own(s):
    import row_top_selection_amd as dt

    if s["op"] == "maps":
        m = dt.page_maps(s["seq_lens"], s["table"], s["page"], s["free"], s["tokens"], new_lens=s["new_lens"])
        return dict(table=s["table"], slots=m.slots, table_rows=m.table_rows, row_lens=m.row_lens, token_starts=m.token_starts, counts=m.counts)
    if s["op"] == "scores":
        if s["form"] == "paged":
            return dt.scores_paged(s["q"], s["weights"], s["keys"], s["seq_lens"], s["table"], key_scales=s["scales"], table_rows=s["table_rows"], out=s["out"])
        return dt.scores_ragged(s["q"], s["weights"], s["keys"], s["seq_lens"], s["starts"], key_scales=s["scales"], out=s["out"])
    if s["op"] == "attend":
        if s["form"] == "paged":
            out, lse = dt.attend_paged(s["q"], s["cache"], s["seq_lens"], s["table"], s["latent"], s["scale"], table_rows=s["table_rows"], max_seq_len=s["max_len"])
        else:
            out, lse = dt.attend_selected(s["q"], s["cache"], s["slots"], s["latent"], s["scale"])
        return dict(out=out, lse=lse)
    out, lse = dt.attend_expanded(s["q"], s["k"], s["v"], s["k_rope"], s["q_starts"], s["k_starts"], s["max_q"], s["scale"])
    return dict(out=out, lse=lse)


def _plain_maps(s):
    page, table, free, tokens = s["page"], s["table"], s["free"], s["tokens"]
    requests, width = table.shape
    lens = s["seq_lens"].clamp(min=0)
    new = torch.ones_like(lens) if s["new_lens"] is None else s["new_lens"]
    new = new.clamp(min=0).minimum(lens)
    held, need = (lens - new + page - 1) // page, (lens + page - 1) // page
    starts = torch.cat([new.new_zeros(1), new.cumsum(0, dtype=torch.int32)])
    taken = (need - held).cumsum(0, dtype=torch.int32)
    first = taken - (need - held)
    # the free list's pages go to the requests in their order
    column = torch.arange(width, dtype=torch.int32, device=table.device)
    source = first[:, None] + column - held[:, None]
    fresh = (column >= held[:, None]) & (column < need[:, None])
    page_or_none = torch.where(source < free.numel(), free[source.clamp(0, free.numel() - 1).long()], -1)
    table = torch.where(fresh, page_or_none, table)
    # each token: its request, its position, its slot
    token = torch.arange(tokens, dtype=torch.int32, device=table.device)
    request = torch.searchsorted(starts[1:].contiguous(), token, right=True)
    real = request < requests
    request = request.clamp(max=requests - 1)
    position = (lens - new)[request] + token - starts[request]
    entry = table[request, (position // page).clamp(0, width - 1).long()]
    slots = torch.where(real & (entry >= 0), entry * page + position % page, -1)
    return dict(table=table, slots=slots.to(torch.int32), table_rows=torch.where(real, request, 0).to(torch.int32),
                row_lens=torch.where(real, position + 1, 0).to(torch.int32), token_starts=starts, counts=torch.stack([starts[-1], taken[-1]]))


def _plain_scores(s):
    n, m, heads, dim, page = s["requests"], s["rows"], s["heads"], s["dim"], s["page"]
    q, lens, out = s["q"].float(), s["seq_lens"].long(), s["out"]
    position = torch.arange(s["length"], device=out.device)
    if s["form"] == "paged":
        at = (s["table"].long()[:, position // page] * page + position % page)
    else:
        at = (s["request_starts"][:, None] + position).clamp(max=s["keys"].shape[0] - 1)
    keys = s["keys"].view(-1, dim)[at].float()  # [requests, length, dim]
    dots = torch.matmul(q.view(n, m * heads, dim), keys.transpose(1, 2)).relu_()
    got = torch.matmul(s["weights"].view(n, m, 1, heads), dots.view(n, m, heads, -1)).view(n * m, -1)
    if s["scales"] is not None:
        got = (got.view(n, m, -1) * s["scales"].view(-1)[at][:, None]).view(n * m, -1)
    column = torch.arange(out.shape[1], device=out.device)
    start = s["starts"].long()[:, None] if s["form"] == "ragged" else 0
    inside = (column >= start) & (column < start + lens[:, None])
    return torch.where(inside, got.gather(1, (column - start).expand(n * m, -1).clamp(0, s["length"] - 1)), out)


def _softmax(scores, seen):
    """Weights and log-sum-exp over the last axis; rows that see nothing have zeros and -inf."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    weights = torch.exp(scores - top)
    total = weights.sum(-1, keepdim=True)
    return weights / total.clamp(min=1e-38), (top + torch.log(total)).squeeze(-1)


def _plain_attend(s):
    q, cache, latent, page = s["q"].float(), s["cache"], s["latent"], s["page"]
    if s["form"] == "paged":
        position = torch.arange(s["max_len"], device=q.device)
        rows = torch.arange(q.shape[0], device=q.device) if s["table_rows"] is None else s["table_rows"].long()
        at = s["table"].long()[rows][:, position // page] * page + position % page
        seen = position < s["seq_lens"][:, None]
    else:
        at, seen = s["slots"].long().clamp(min=0), s["slots"] >= 0
    vectors = cache.view(-1, cache.shape[-1])[at].float()  # [rows, tokens, latent + rope]
    weights, lse = _softmax(torch.matmul(q, vectors.transpose(1, 2)) * s["scale"], seen[:, None])
    return dict(out=torch.matmul(weights, vectors[..., :latent]).to(s["q"].dtype), lse=lse)


def _plain_expand(s):
    q_starts, k_starts = s["q_starts"].long(), s["k_starts"].long()
    q_lens, k_lens = q_starts.diff(), k_starts.diff()
    row = torch.arange(s["max_q"], device=q_starts.device)
    column = torch.arange(s["max_k"], device=q_starts.device)
    q_at = (q_starts[:-1, None] + row).clamp(max=s["q"].shape[0] - 1)
    k_at = (k_starts[:-1, None] + column).clamp(max=s["k"].shape[0] - 1)
    q = s["q"][q_at].float().transpose(1, 2)  # [requests, heads, rows, 192]
    k = s["k"][k_at].float().transpose(1, 2)
    rope = s["k_rope"][k_at].float()[:, None]
    v = s["v"][k_at].float().transpose(1, 2)
    scores = torch.matmul(q[..., :128], k.transpose(2, 3)) + torch.matmul(q[..., 128:], rope.transpose(2, 3))
    seen = (column < k_lens[:, None, None]) & (column <= row[:, None] + (k_lens - q_lens)[:, None, None])
    weights, lse = _softmax(scores * s["scale"], seen[:, None])
    out = torch.matmul(weights, v).transpose(1, 2)
    real = row < q_lens[:, None]
    return dict(out=out[real].to(s["q"].dtype), lse=lse.transpose(1, 2)[real])


# ---------------------------------------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    c = case
    size = 1 if c.get("type") == "fp8" else 2
    if c["op"] == "maps":
        tokens, pages = sum(_new(c)), sum(n / c["page"] for n in _new(c))
        entries = sum(-(-n // c["page"]) for n in _new(c))
        # lengths and first tokens; a table entry for each page that a new token lies in; the free list's pages out
        # of it and into the table; three numbers a token
        return {"bytes": 4 * (3 * c["requests"] + entries + 2 * pages + 3 * tokens), "flops": 0}
    if c["op"] == "scores":
        m, heads, dim = c["rows"], c["heads"], c["dim"]
        pairs = sum(max(0, n - i) for n in _seen(c) for i in range(m))
        keys = sum(_seen(c)) * (dim * size + (4 if size == 1 else 0))
        return {"bytes": keys + c["requests"] * m * heads * (dim * size + 4) + 4 * pairs, "flops": pairs * heads * (2 * dim + 2)}
    if c["op"] == "attend":
        rows, heads, dim = c["requests"] * c["rows"], c["heads"], c["latent"] + c["rope"]
        if c["form"] == "slots":
            take = min(c["k"], c["length"])
            pairs, index = rows * take, rows * c["k"]
            # each distinct vector once: rows of a request share its tokens
            tokens = c["requests"] * c["length"] * (1 - (1 - take / c["length"]) ** c["rows"])
        else:
            pairs, tokens = sum(max(0, n - i) for n in _seen(c) for i in range(c["rows"])), sum(_seen(c))
            index = tokens / c["page"]
        return {"bytes": 2 * (tokens * dim + rows * heads * (dim + c["latent"])) + 4 * (rows * heads + index), "flops": pairs * heads * 2 * (dim + c["latent"])}
    lens, heads = _expand_lengths(c), c["heads"]
    rows, keys = sum(n for n, _ in lens), sum(n + past for n, past in lens)
    pairs = sum(n * past + n * (n + 1) // 2 for n, past in lens)
    return {"bytes": 2 * (heads * (rows * (192 + 128) + keys * 256) + keys * 64) + 4 * rows * heads, "flops": pairs * heads * 2 * (192 + 128)}


# ---------------------------------------------------------------------------------------------------------
# The operators' definitions, in 64 bits, a request or a row at a time


def exact(case, seed):
    if case["op"] == "maps":
        return None  # whole numbers
    s = prepare(case, seed)
    return {"scores": _exact_scores, "attend": _exact_attend, "expand": _exact_expand}[case["op"]](s)


def _exact_scores(s):
    m, page, dim = s["rows"], s["page"], s["dim"]
    out = s["out"].double()
    lens = s["seq_lens"].tolist()
    q, w = s["q"].double(), s["weights"].double()
    for r in range(s["requests"]):
        longest = max(lens[r * m:(r + 1) * m])
        j = torch.arange(longest, device=out.device)
        begin = 0
        if s["form"] == "paged":
            where = s["table"][r].long()[j // page] * page + j % page
        else:
            begin = int(s["request_starts"][r])
            where = begin + j
        keys = s["keys"].view(-1, dim)[where].double()
        factor = s["scales"].view(-1)[where].double() if s["scales"] is not None else torch.ones(longest, dtype=torch.float64, device=out.device)
        for first in range(r * m, (r + 1) * m, 64):
            rows = slice(first, min((r + 1) * m, first + 64))
            value = torch.zeros(len(lens[rows]), longest, dtype=torch.float64, device=out.device)
            for h in range(s["heads"]):
                value += w[rows, h, None] * (q[rows, h] @ keys.T).clamp(min=0)
            value *= factor
            for i, length in enumerate(lens[rows]):
                out[first + i, begin:begin + length] = value[i, :length]
    return out


def _exact_attend(s):
    page, latent = s["page"], s["latent"]
    q, cache = s["q"].double(), s["cache"].view(-1, s["cache"].shape[-1])
    outs, sums = [], []
    lens = s["seq_lens"].tolist() if s["form"] == "paged" else None
    for r in range(q.shape[0]):
        if lens is None:
            where = s["slots"][r]
            where = where[where >= 0].long()
        else:
            j = torch.arange(max(0, lens[r]), device=q.device)
            where = s["table"][r // s["rows"]].long()[j // page] * page + j % page
        x = cache[where].double()
        logits = (q[r] @ x.T) * s["scale"]
        if where.numel():
            sums.append(torch.logsumexp(logits, -1))
            outs.append(torch.softmax(logits, -1) @ x[:, :latent])
        else:
            sums.append(torch.full((q.shape[1],), -math.inf, dtype=torch.float64, device=q.device))
            outs.append(q.new_zeros(q.shape[1], latent))
    return dict(out=torch.stack(outs), lse=torch.stack(sums))


def _exact_expand(s):
    q_at, k_at = s["q_starts"].tolist(), s["k_starts"].tolist()
    out = torch.zeros(s["q"].shape[0], s["heads"], 128, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["q"].shape[0], s["heads"], dtype=torch.float64, device=s["q"].device)
    for r in range(s["requests"]):
        a, b, c, d = q_at[r], q_at[r + 1], k_at[r], k_at[r + 1]
        rope = s["k_rope"][c:d].double()
        hidden = torch.arange(d - c, device=out.device) > torch.arange(b - a, device=out.device)[:, None] + (d - c) - (b - a)
        for h in range(s["heads"]):
            key = torch.cat([s["k"][c:d, h].double(), rope], dim=1)
            logits = (s["q"][a:b, h].double() @ key.T) * s["scale"]
            logits[hidden] = -math.inf
            lse[a:b, h] = torch.logsumexp(logits, -1)
            out[a:b, h] = torch.softmax(logits, -1) @ s["v"][c:d, h].double()
    return dict(out=out, lse=lse)
