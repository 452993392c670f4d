"""Cache writes on the GPU against their definition in 64 bits
(tests/append_plain.py)."""
import numpy as np
import pytest
import torch

from tests import append_plain as plain

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
BITS = {1: torch.uint8, 2: torch.int16, 4: torch.int32}


def i32(v):
    return torch.as_tensor(np.asarray(v, dtype=np.int32)).to(DEV)


def bits(t):
    return t.contiguous().view(BITS[t.element_size()])


def rand(g, kind, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(TYPES[kind])


def step(rng, tokens, pages, page, positions):
    """Slots and windows, some of them of tokens that are not cached: (slots, row_lens, cached)."""
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    lens = rng.integers(1, positions + 1, tokens)
    for t in range(2, tokens, 7):
        kind = (t // 7) % 5
        if kind == 0:
            slots[t] = -1
        elif kind == 1:
            slots[t] = pages * page + t  # a page that the cache does not have
        elif kind == 2:
            lens[t] = 0
        elif kind == 3:
            lens[t] = positions + 1 + t
        else:
            slots[t], lens[t] = 2 ** 31 - 1, -5
    cached = (slots >= 0) & (slots < pages * page) & (lens > 0) & (lens <= positions)
    return slots, lens, cached


def untouched(before, after, slots):
    """Everything but the slots is byte for byte as it was."""
    before, after = bits(before).flatten(0, 1).clone(), bits(after).flatten(0, 1)
    at = torch.as_tensor(slots, device=DEV)
    before[at] = after[at]
    assert torch.equal(before, after)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("latent,tokens,heads,page,norm,near", [
    (512, 1, 1, 64, True, True),
    (512, 3, 16, 1, True, False),
    (256, 1, 5, 16, True, True),
    (256, 9, 128, 64, False, False),
    (512, 130, 7, 16, False, True),
    (256, 77, 0, 128, True, False),
    (512, 61, 33, 32, True, True),
])
def test_latent(kind, latent, tokens, heads, page, norm, near):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(latent + tokens)
    rng = np.random.default_rng(tokens + heads)
    positions, pages = 300, -(-tokens // page) + 3
    slots, lens, cached = step(rng, tokens, pages, page, positions)
    x = rand(g, kind, tokens, latent + 64) * torch.rand(tokens, 1, generator=g, device=DEV).to(TYPES[kind])
    weight = 1 + 0.2 * torch.randn(latent, generator=g, device=DEV) if norm else None
    cos_sin = plain.angles(positions).to(DEV)
    q = rand(g, kind, tokens, heads, 192)[..., 128:] if heads else None
    cache = rand(g, kind, pages, page, latent + 64)
    before, out = cache.clone(), torch.zeros_like(x)
    got = dt.append_latent(x, cache, i32(slots), i32(lens), cos_sin, weight=weight, eps=1e-5, q_rope=q, out=out, interleaved=near)
    torch.cuda.synchronize()
    want, off = plain.latent(x, weight, 1e-5, lens, cos_sin, near, latent)
    plain.close(out, want, off, "out")
    assert norm or torch.equal(out[:, :latent], x[:, :latent])
    real = slots[cached]
    assert torch.equal(bits(cache.view(-1, latent + 64)[torch.as_tensor(real, device=DEV)]), bits(out[torch.as_tensor(cached, device=DEV)]))
    untouched(before, cache, real)
    if heads:
        want, size = plain.turn(q.double().cpu(), q.double().cpu().abs(), lens, cos_sin, near)
        plain.close(got, want, size * 2.0 ** -22, "q")
    else:
        assert got is None


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("to", ["same", "fp8"])
@pytest.mark.parametrize("dim,tokens,heads,page,norm,near", [
    (128, 1, 64, 64, True, False),
    (64, 1, 1, 1, True, True),
    (128, 5, 3, 16, False, True),
    (64, 33, 8, 64, True, False),
    (128, 130, 0, 32, True, True),
    (128, 70, 10, 64, False, False),
    (64, 50, 128, 16, False, True),
])
def test_index(kind, to, dim, tokens, heads, page, norm, near):
    import row_top_selection_amd as dt

    eight = to == "fp8"
    to = "fp8" if eight else kind
    g = torch.Generator(DEV).manual_seed(dim + tokens)
    rng = np.random.default_rng(tokens + heads)
    positions, pages = 200, -(-tokens // page) + 3
    slots, lens, cached = step(rng, tokens, pages, page, positions)
    x = rand(g, kind, tokens, dim) + torch.randn(tokens, 1, generator=g, device=DEV).to(TYPES[kind])
    weight = 1 + 0.2 * torch.randn(dim, generator=g, device=DEV) if norm else None
    bias = 0.2 * torch.randn(dim, generator=g, device=DEV) if norm else None
    cos_sin = plain.angles(positions).to(DEV)
    q = rand(g, kind, tokens, heads, dim) if heads else None
    if heads > 2:
        q[0, 1] = 0.0  # a head of nothing
    weights = torch.randn(tokens, heads, generator=g, device=DEV) if eight and heads else None
    keys = rand(g, kind, pages, page, dim).to(TYPES[to])
    scales = torch.rand(pages, page, generator=g, device=DEV) if eight else None
    before, scales_before = keys.clone(), None if scales is None else scales.clone()
    got = dt.append_index(x, keys, i32(slots), i32(lens), cos_sin, key_scales=scales, weight=weight, bias=bias, eps=1e-5, q=q, weights=weights, interleaved=near)
    torch.cuda.synchronize()
    real, pick = slots[cached], torch.as_tensor(cached)
    want, off = plain.index(x, weight, bias, 1e-5, lens, cos_sin, near)
    stored = keys.view(-1, dim)[torch.as_tensor(real, device=DEV)]
    if eight:
        plain.close8(stored, scales.view(-1)[torch.as_tensor(real, device=DEV)], want[pick], off[pick], "keys")
        untouched(scales_before[..., None], scales[..., None], real)
    else:
        plain.close(stored, want[pick], off[pick], "keys")
    untouched(before, keys, real)
    if not heads:
        assert got is None
        return
    q_out, weights_out = got
    assert q_out.dtype == TYPES[to] and q_out.shape == q.shape
    want, off = plain.index(q, None, None, 0.0, lens, cos_sin, near)
    if eight:
        scale = (weights_out.double() / weights.double()).cpu()
        # the product's rounding
        plain.close8(q_out, scale, want, off + want.abs().amax(-1, keepdim=True) * 2.0 ** -23, "q")
        if heads > 2:
            assert (q_out[0, 1].float() == 0).all()
    else:
        assert weights_out is None
        plain.close(q_out, want, off, "q")


def test_strided_inputs_and_outputs_in_place():
    """Parts of wider tensors, caches with room between their pages, results over the inputs."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(5)
    tokens, heads, page, positions = 37, 6, 16, 100
    rng = np.random.default_rng(5)
    slots, lens, cached = step(rng, tokens, 5, page, positions)
    cos_sin = torch.zeros(positions, 72, device=DEV)
    cos_sin[:, :64] = plain.angles(positions).to(DEV)
    at = (i32(slots), i32(lens), cos_sin[:, :64])
    with pytest.raises(dt.DsatopkError) as e:  # rows 1400 bytes apart
        dt.append_latent(rand(g, "bf16", tokens, 700)[:, 24:600], torch.zeros(5, page, 576, device=DEV).bfloat16(), *at)
    assert e.value.status == 2
    wide = rand(g, "bf16", tokens, 704)
    x = wide[:, 24:600]
    weight = 1 + 0.1 * torch.randn(512, generator=g, device=DEV)
    q = rand(g, "bf16", tokens, heads, 192)
    cache, room = torch.zeros(5, page, 576, device=DEV).bfloat16(), torch.zeros(7, page + 1, 640, device=DEV).bfloat16()
    first = dt.append_latent(x.contiguous(), cache, *at, weight=weight, q_rope=q[..., 128:].contiguous(), interleaved=True)
    absorbed = torch.full((tokens, heads, 576), 3.0, device=DEV).bfloat16()
    got = dt.append_latent(x, room[1:6, :page, 64:], *at, weight=weight, q_rope=q[..., 128:], q_out=absorbed[..., 512:], interleaved=True)
    assert got.data_ptr() == absorbed[..., 512:].data_ptr()
    assert torch.equal(absorbed[..., 512:], first) and (absorbed[..., :512] == 3).all()
    assert torch.equal(room[1:6, :page, 64:], cache)
    room[1:6, :page, 64:] = 0
    assert (room == 0).all()
    # in place
    other = torch.zeros_like(cache)
    kept, kept_q = wide.clone(), q.clone()
    dt.append_latent(x, other, *at, weight=weight, out=x, q_rope=q[..., 128:], q_out=q[..., 128:], interleaved=True)
    assert torch.equal(other, cache) and torch.equal(q[..., 128:], first) and torch.equal(q[..., :128], kept_q[..., :128])
    assert torch.equal(wide[:, :24], kept[:, :24]) and torch.equal(wide[:, 600:], kept[:, 600:])
    pick = torch.as_tensor(cached, device=DEV)
    assert torch.equal(x[pick], cache.view(-1, 576)[torch.as_tensor(slots[cached], device=DEV)])

    # the indexer's
    keys, iq = rand(g, "fp16", tokens, 200)[:, 8:136], rand(g, "fp16", tokens, heads, 136)[..., :128]
    a, b = torch.zeros(5, page, 128, device=DEV).half(), torch.zeros(5, page + 2, 160, device=DEV).half()
    one, _ = dt.append_index(keys.contiguous(), a, *at, q=iq.contiguous())
    two, _ = dt.append_index(keys, b[:, :page, :128], *at, q=iq, q_out=iq)
    assert two.data_ptr() == iq.data_ptr() and torch.equal(one, iq) and torch.equal(a, b[:, :page, :128])
    iq, weights = rand(g, "fp16", tokens, heads, 128), torch.randn(tokens, heads + 3, generator=g, device=DEV)
    a, b = (torch.zeros(5, page, 128, device=DEV).to(TYPES["fp8"]) for _ in range(2))
    sa, sb = torch.zeros(5, page, device=DEV), torch.zeros(5, 2 * page, device=DEV)
    one, w1 = dt.append_index(keys, a, *at, key_scales=sa, q=iq, weights=weights[:, 2:2 + heads].contiguous())
    two, w2 = dt.append_index(keys, b, *at, key_scales=sb[:, :page], q=iq, weights=weights[:, 2:2 + heads], weights_out=weights[:, 2:2 + heads],
                              q_out=torch.zeros(tokens, heads + 1, 256, device=DEV).to(TYPES["fp8"])[:, 1:, 64:192])
    assert torch.equal(bits(one), bits(two)) and torch.equal(w1, w2) and torch.equal(w1, weights[:, 2:2 + heads])
    assert torch.equal(bits(a), bits(b)) and torch.equal(sa, sb[:, :page]) and (sb[:, page:] == 0).all()


def test_slots_past_32_bits_of_bytes():
    """Caches and queries whose ends lie more than 2^32 bytes from their starts."""
    import row_top_selection_amd as dt

    pages = 60000
    cache = torch.zeros(pages, 64, 576, device=DEV, dtype=torch.bfloat16)  # 4.4 GB
    x = torch.randn(2, 576, device=DEV).bfloat16()
    dt.append_latent(x, cache, i32([5, pages * 64 - 3]), i32([1, 1]), plain.angles(4).to(DEV))
    assert torch.equal(cache.view(-1, 576)[[5, -3]], x) and (cache.view(-1, 576)[[4, 6, -4, -2]] == 0).all()
    del cache
    keys = torch.zeros(1 << 19, 64, 128, device=DEV, dtype=torch.float8_e4m3fn)  # 4.3 GB
    scales = torch.zeros(1 << 19, 64, device=DEV)
    dt.append_index(x[:, :128], keys, i32([7, (1 << 25) - 2]), i32([1, 1]), plain.angles(4).to(DEV), key_scales=scales)
    plain.close8(keys.view(-1, 128)[[7, -2]], scales.view(-1)[[7, -2]], x[:, :128].double().cpu(), torch.zeros(2, 128))
    assert int((scales != 0).sum()) == 2
    del keys, scales
    q = torch.zeros(5, 2, (1 << 28) + 64, device=DEV, dtype=torch.bfloat16)  # heads 2^29 bytes apart: 5.4 GB
    q[..., -64:] = torch.randn(5, 2, 64, device=DEV).bfloat16()
    got = dt.append_latent(torch.zeros(5, 576, device=DEV).bfloat16(), torch.zeros(1, 64, 576, device=DEV).bfloat16(), i32([-1] * 5), i32([1] * 5),
                           plain.angles(4).to(DEV), q_rope=q[..., -64:])
    assert torch.equal(got, q[..., -64:])  # position 0 turns by nothing


def test_captured_and_replayed():
    """One graph of both calls; each replay is the eager result of what the inputs hold then."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(9)
    tokens, heads = 21, 5
    cos_sin = plain.angles(64).to(DEV)
    x, q = rand(g, "bf16", tokens, 576), rand(g, "bf16", tokens, heads, 64)
    keys, iq, w = rand(g, "bf16", tokens, 128), rand(g, "bf16", tokens, heads, 128), torch.rand(tokens, heads, generator=g, device=DEV)
    slots, lens = i32(np.arange(tokens)), i32(np.arange(tokens) + 1)

    def caches():
        return (torch.zeros(4, 16, 576, device=DEV).bfloat16(), torch.zeros(4, 16, 128, device=DEV).to(TYPES["fp8"]), torch.zeros(4, 16, device=DEV))

    def call(to):
        got = dt.append_latent(x, to[0], slots, lens, cos_sin, q_rope=q)
        return (got, *dt.append_index(keys, to[1], slots, lens, cos_sin, key_scales=to[2], q=iq, weights=w))

    mine = caches()
    call(caches())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(mine)
    for n in range(4):
        for t in (x, q, keys, iq):
            t.copy_(rand(g, "bf16", *t.shape))
        slots.copy_(torch.randperm(64, generator=g, device=DEV)[:tokens].int())
        lens.copy_(torch.randint(0, 70, (tokens,), generator=g, device=DEV).int())
        for t in mine:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        theirs = caches()
        want = call(theirs)
        torch.cuda.synchronize()
        for a, b in zip((*out, *mine), (*want, *theirs)):
            assert torch.equal(bits(a), bits(b)), n


def test_another_stream():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(2)
    x, cos_sin = rand(g, "bf16", 50, 576), plain.angles(64).to(DEV)
    at = (i32(np.arange(50)), i32(np.arange(50) + 1), cos_sin)
    a, b = (torch.zeros(1, 64, 576, device=DEV).bfloat16() for _ in range(2))
    q = rand(g, "bf16", 50, 3, 64)
    want = dt.append_latent(x, a, *at, q_rope=q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dt.append_latent(x, b, *at, q_rope=q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b) and torch.equal(got, want)


def test_no_tokens_is_no_error():
    import row_top_selection_amd as dt

    cos_sin, none = plain.angles(4).to(DEV), i32([])
    cache = torch.ones(1, 16, 576, device=DEV).bfloat16()
    x = torch.zeros(0, 576, device=DEV).bfloat16()
    assert dt.append_latent(x, cache, none, none, cos_sin) is None
    assert dt.append_latent(x, cache, none, none, cos_sin, q_rope=torch.zeros(0, 3, 64, device=DEV).bfloat16()).shape == (0, 3, 64)
    keys = torch.ones(1, 16, 128, device=DEV).to(TYPES["fp8"])
    q, w = dt.append_index(x[:, :128], keys, none, none, cos_sin, key_scales=torch.ones(1, 16, device=DEV), q=torch.zeros(0, 3, 128, device=DEV).bfloat16(),
                           weights=torch.zeros(0, 3, device=DEV))
    assert q.shape == (0, 3, 128) and w.shape == (0, 3)
    # no heads, no pages, no positions
    x = torch.ones(2, 576, device=DEV).bfloat16()
    got = dt.append_latent(x, cache[:0], i32([0, 1]), i32([1, 2]), cos_sin[:0], q_rope=torch.zeros(2, 0, 64, device=DEV).bfloat16())
    assert got.shape == (2, 0, 64) and (cache == 1).all()


def test_scores_of_appended_keys():
    """The 8-bit keys, scales, queries and weights are what scores_paged takes."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(4)
    tokens, heads, dim = 90, 16, 128
    cos_sin = plain.angles(tokens).to(DEV)
    lens, table = i32(np.arange(tokens) + 1), i32([[3, 0, 5, 1, 4, 2]])
    maps = dt.page_maps(i32([tokens]), table, 16, i32([3, 0, 5, 1, 4, 2]), tokens, new_lens=i32([tokens]))
    assert torch.equal(maps.row_lens, lens)
    x, q, w = rand(g, "bf16", tokens, dim), rand(g, "bf16", tokens, heads, dim), torch.randn(tokens, heads, generator=g, device=DEV)
    keys, scales = torch.zeros(6, 16, dim, device=DEV).to(TYPES["fp8"]), torch.zeros(6, 16, device=DEV)
    q8, w8 = dt.append_index(x, keys, maps.slots, maps.row_lens, cos_sin, key_scales=scales, q=q, weights=w)
    got = dt.scores_paged(q8, w8, keys, maps.row_lens, table, key_scales=scales, table_rows=maps.table_rows).double().cpu()
    want_k, _ = plain.index(x, None, None, 0.0, lens.tolist(), cos_sin, False)
    want_q, _ = plain.index(q, None, None, 0.0, lens.tolist(), cos_sin, False)
    for t in range(0, tokens, 13):
        dots = want_q[t] @ want_k[:t + 1].T
        want = (w[t].double().cpu()[:, None] * dots.clamp(min=0)).sum(0)
        # both factors of every product are off by 2^-4 of themselves, or half of the smallest step of their scale
        qa, ka = want_q[t].abs(), want_k[:t + 1].abs()
        qa, ka = (v * 2.0 ** -4 + v.amax(-1, keepdim=True) / 448 * 2.0 ** -10 for v in (qa, ka))
        size = (w[t].double().cpu().abs()[:, None] * ((want_q[t].abs() + qa) @ (want_k[:t + 1].abs() + ka).T - want_q[t].abs() @ want_k[:t + 1].abs().T)).sum(0)
        assert ((got[t, :t + 1] - want).abs() <= size * 1.001).all()
