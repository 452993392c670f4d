"""Latent attention on the GPU against its definition in 64 bits
(tests/serve_plain.py)."""
import math

import numpy as np
import pytest
import torch

from tests import serve_plain

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def i32(v):
    return torch.as_tensor(np.asarray(v, dtype=np.int32)).to(DEV)


def close(out, lse, want, logit_size, dim):
    """`want` = (out, lse, size) in 64 bits.

    A logit is a sum of `dim` exact products in fp32, off by at most dim *
    2^-24 of the products' sizes, times the scale (two more roundings) and
    taken in base 2 (one more): `off`, beside exp2's and log2's own 2^-20.
    That shifts a weight and the weights' sum by a factor e^off each. A
    weight is rounded to the type, and so is the output: half a step each.
    Sums over tokens in fp32 are covered by 2^-16 of the values' sizes."""
    want_out, want_lse, size = want
    off = (dim + 4) * 2.0 ** -24 * logit_size + 2.0 ** -20
    half = torch.finfo(out.dtype).eps / 2
    got, got_lse = out.cpu().double(), lse.cpu().double()
    assert torch.isfinite(got).all()
    bound = size * (math.expm1(2 * off) + half * (1 + half) + 2.0 ** -16) + want_out.abs() * half
    # below the type's normal range a step no longer shrinks
    bound = bound + torch.finfo(out.dtype).smallest_normal * half
    assert ((got - want_out).abs() <= bound).all(), ((got - want_out).abs() / bound).max()
    seen = torch.isfinite(want_lse)
    assert torch.equal(torch.isfinite(got_lse), seen) and (got_lse[~seen] == -math.inf).all()
    assert (got[~seen] == 0).all()
    assert ((got_lse - want_lse)[seen].abs() <= off + 2.0 ** -20 * (1 + want_lse[seen].abs())).all()


def logit_size(q, vectors, scale):
    if not vectors.numel() or not q.numel():
        return 0.0
    return float((q.float().abs().flatten(0, 1).max(0).values * vectors.float().abs().max(0).values).sum() * scale)


def make(g, rows, heads, latent, pages, page, kind):
    q = torch.randn(rows, heads, latent + 64, generator=g, device=DEV).to(TYPES[kind])
    cache = torch.randn(pages, page, latent + 64, generator=g, device=DEV).to(TYPES[kind])
    return q, cache


SCALE = 192 ** -0.5


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,latent,page,k,valid", [
    (16, 512, 64, 128, [128, 0, 1, 63, 64, 65, 127]),
    (1, 512, 1, 70, [70, 69, 2]),
    (8, 256, 16, 2048, [2048, 1000, 15]),
    (24, 512, 64, 200, [200, 31, 33, 0]),
    (32, 256, 128, 96, [96, 95]),
    (40, 512, 16, 300, [300, 17, 16]),
    (64, 512, 64, 513, [513, 512]),
    (128, 512, 64, 64, [64, 1, 40]),
    (100, 256, 64, 333, [333, 200]),
    (200, 512, 4, 90, [90, 3]),
])
def test_selected(kind, heads, latent, page, k, valid):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads * k)
    rng = np.random.default_rng(heads + k)
    rows, pages = len(valid), -(-2500 // page)
    q, cache = make(g, rows, heads, latent, pages, page, kind)
    slots = np.full((rows, k), -1)
    for b, n in enumerate(valid):
        slots[b, :n] = rng.permutation(pages * page)[:n]
    out, lse = dt.attend_selected(q, cache, i32(slots), latent, SCALE)
    torch.cuda.synchronize()
    vectors = cache.view(-1, latent + 64)
    want = serve_plain.attend(q, vectors, latent, SCALE, [slots[b, :n] for b, n in enumerate(valid)])
    close(out, lse, want, logit_size(q, vectors, SCALE), latent + 64)


@pytest.mark.parametrize("rows", [1, 3, 100, 300])
def test_selected_row_counts_and_scattered_holes(rows):
    """Batches that split, that fill the card once and more than once; -1
    and slots past the cache anywhere in a row; slots named twice."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(rows)
    rng = np.random.default_rng(rows)
    q, cache = make(g, rows, 16, 512, 20, 64, "bf16")
    slots = rng.integers(-400, 20 * 64 + 400, (rows, 150))
    slots[0, :140] = -1
    slots[0, 0] = 2 ** 31 - 1
    out, lse = dt.attend_selected(q, cache, i32(slots), 512, SCALE)
    torch.cuda.synchronize()
    picked = [s[(s >= 0) & (s < 20 * 64)] for s in slots]
    want = serve_plain.attend(q, cache.view(-1, 576), 512, SCALE, picked)
    close(out, lse, want, logit_size(q, cache.view(-1, 576), SCALE), 576)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,latent,page,per,lens", [
    (16, 512, 64, 1, [0, 1, 64, 65, 1000, -4]),
    (128, 512, 16, 1, [700, 33]),
    (16, 256, 1, 2, [130, 3]),
    (40, 512, 16, 3, [5, 500]),
    (20, 512, 128, 1, [4000]),
    (64, 256, 64, 1, [4001, 100, 2]),
])
def test_paged(kind, heads, latent, page, per, lens):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads + page)
    n, width = len(lens), -(-max(lens) // page) + 2
    rows = n * per
    q, cache = make(g, rows, heads, latent, n * width, page, kind)
    table = torch.randperm(n * width, generator=g, device=DEV).view(n, width).to(torch.int32)
    row_lens = [x - (per - 1) + i for x in lens for i in range(per)]
    table_rows = None if per == 1 else i32(np.arange(rows) // per)
    out, lse = dt.attend_paged(q, cache, i32(row_lens), table, latent, SCALE, table_rows=table_rows)
    torch.cuda.synchronize()
    picked = []
    for b, x in enumerate(row_lens):
        j = np.arange(max(0, x))
        picked.append(table[b // per].cpu().numpy()[j // page] * page + j % page)
    vectors = cache.view(-1, latent + 64)
    want = serve_plain.attend(q, vectors, latent, SCALE, picked)
    close(out, lse, want, logit_size(q, vectors, SCALE), latent + 64)
    # a bound that is too small, or exact, changes how rows are split and nothing else
    for bound in (0, 70, max(lens)):
        out, lse = dt.attend_paged(q, cache, i32(row_lens), table, latent, SCALE,
                                   table_rows=table_rows, max_seq_len=bound)
        close(out, lse, want, logit_size(q, vectors, SCALE), latent + 64)


@pytest.mark.parametrize("heads,latent,lens", [(16, 256, [20000, 3, 9000]), (70, 512, [12000, 0]),
                                               (33, 256, [9999])])
def test_paged_long_rows_in_many_parts(heads, latent, lens):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads)
    page, pages = 64, 40
    width = -(-max(lens) // page)
    q, cache = make(g, len(lens), heads, latent, pages, page, "bf16")
    table = torch.randint(0, pages, (len(lens), width), generator=g, device=DEV).to(torch.int32)
    out, lse = dt.attend_paged(q, cache, i32(lens), table, latent, SCALE)
    torch.cuda.synchronize()
    picked = []
    for b, n in enumerate(lens):
        j = np.arange(n)
        picked.append(table[b].cpu().numpy()[j // page] * page + j % page)
    vectors = cache.view(-1, latent + 64)
    want = serve_plain.attend(q, vectors, latent, SCALE, picked)
    close(out, lse, want, logit_size(q, vectors, SCALE), latent + 64)


def test_paged_pages_that_are_not_there():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(1)
    q, cache = make(g, 3, 16, 512, 6, 16, "bf16")
    table = i32([[2, -1, 9, 3], [-1, -1, -1, -1], [1 << 30, 0, 5, -7]])
    out, lse = dt.attend_paged(q, cache, i32([60, 64, 99]), table, 512, SCALE)
    torch.cuda.synchronize()
    rows = [[2, -1, -1, 3], [-1] * 4, [-1, 0, 5, -1]]
    picked = [[t[j // 16] * 16 + j % 16 for j in range(n) if t[j // 16] >= 0]
              for t, n in zip(rows, (60, 64, 64))]
    want = serve_plain.attend(q, cache.view(-1, 576), 512, SCALE, picked)
    close(out, lse, want, logit_size(q, cache.view(-1, 576), SCALE), 576)


def test_tokens_that_no_row_reads_may_hold_anything():
    """NaN and infinities in unselected slots, behind a row's end inside its
    last page, and in the padding between strided tokens."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(2)
    q, cache = make(g, 2, 16, 512, 8, 64, "bf16")
    wide = torch.full((8, 80, 640), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :64, :576] = cache
    view = wide[:, :64, :576]
    slots = i32([[0, 5, 200, -1, 70], [9, 9, 1, 511, 510]])
    used = torch.zeros(512, dtype=torch.bool, device=DEV)
    used[slots.flatten()[slots.flatten() >= 0].long()] = True
    view[~used.view(8, 64)] = float("inf")
    a = dt.attend_selected(q, cache, slots, 512, SCALE)
    b = dt.attend_selected(q, view, slots, 512, SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(a[0]).all()
    lens = i32([100, 33])
    table = i32([[3, 6], [1, 0]])
    view.copy_(cache)
    view[6, 36:] = float("nan")
    view[1, 33:] = -float("inf")
    view[0] = float("nan")
    a = dt.attend_paged(q, cache, lens, table, 512, SCALE)
    b = dt.attend_paged(q, view, lens, table, 512, SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(b[0]).all()


def test_strided_queries_and_out_arguments():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(3)
    q, cache = make(g, 4, 16, 512, 8, 64, "fp16")
    wide = torch.full((4, 20, 704), float("nan"), dtype=torch.float16, device=DEV)
    wide[:, 2:18, 64:640] = q
    slots = i32(np.random.default_rng(3).permutation(512)[:400].reshape(4, 100))
    a = dt.attend_selected(q, cache, slots, 512, SCALE)
    out = torch.empty(4, 16, 512, dtype=torch.float16, device=DEV)
    lse = torch.empty(4, 16, device=DEV)
    work = torch.full((dt.attend_bytes(4, 16, 512, 100) + 64,), 255, dtype=torch.uint8, device=DEV)
    big = torch.full((4, 140), 3, dtype=torch.int32, device=DEV)
    big[:, :100] = slots
    b = dt.attend_selected(wide[:, 2:18, 64:640], cache, big[:, :100], 512, SCALE, out=out, lse=lse,
                           workspace=work)
    assert b[0] is out and b[1] is lse
    assert torch.equal(a[0], out) and torch.equal(a[1], lse)
    assert (work[-64:] == 255).all()


def test_logits_of_every_size():
    """A maximum that keeps growing along the row, one that comes first, equal
    logits, and logits far from 0: the softmax's reference follows."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(4)
    n = 700
    cache = torch.randn(1, 1024, 576, generator=g, device=DEV)
    cache[0, :, 0] = torch.arange(1024, device=DEV) * 0.5
    cache = cache.to(torch.bfloat16)
    q = torch.zeros(5, 16, 576, device=DEV)
    q[0, :, 0] = 1.0     # growing by 0.5 a token
    q[1, :, 0] = -1.0    # falling
    q[2] = 0.0           # equal
    q[3, :, 1] = 200.0   # spread of hundreds
    q[4, :, 0] = -16.0   # down to -6000 and below
    q = q.to(torch.bfloat16)
    slots = i32(np.tile(np.arange(n), (5, 1)))
    out, lse = dt.attend_selected(q, cache, slots, 512, 1.0)
    torch.cuda.synchronize()
    want = serve_plain.attend(q, cache[0], 512, 1.0, [np.arange(n)] * 5)
    # sizes by row: one row's large logits do not excuse another's
    for b in range(5):
        size = float((q[b].float().abs() @ cache[0, :n].float().abs().T).max())
        close(out[b:b + 1], lse[b:b + 1], tuple(w[b:b + 1] for w in want), size, 576)


def test_same_inputs_same_bits_and_graph_replays():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(5)
    rng = np.random.default_rng(5)
    q, cache = make(g, 3, 16, 512, 40, 64, "bf16")
    slots = i32(rng.integers(0, 2560, (3, 512)))
    first = dt.attend_selected(q, cache, slots, 512, SCALE)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = dt.attend_selected(q, cache, slots, 512, SCALE)
    side.synchronize()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    work = torch.empty(dt.attend_bytes(3, 16, 512, 512), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dt.attend_selected(q, cache, slots, 512, SCALE, out=out, lse=lse, workspace=work)
    for _ in range(4):
        slots.copy_(i32(rng.integers(-1, 2560, (3, 512))))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = dt.attend_selected(q, cache, slots, 512, SCALE)
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])


def test_cache_past_32_bit_offsets():
    """A cache of 4.6 GB: slots and pages past 2^32 bytes."""
    import row_top_selection_amd as dt

    pages, page = 62500, 64
    cache = torch.zeros(pages, page, 576, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(DEV).manual_seed(6)
    q = torch.randn(2, 16, 576, generator=g, device=DEV).to(torch.bfloat16)
    at = np.array([pages * page - 1, 0, 4_000_000 - 77, 1_900_000, 3_800_000])
    cache.view(-1, 576)[torch.as_tensor(at, device=DEV)] = torch.randn(5, 576, generator=g, device=DEV).to(torch.bfloat16)
    out, lse = dt.attend_selected(q, cache, i32(np.stack([at, at])), 512, SCALE)
    few = cache.view(-1, 576)[torch.as_tensor(at, device=DEV)]
    want = serve_plain.attend(q, few, 512, SCALE, [np.arange(5)] * 2)
    close(out, lse, want, logit_size(q, few, SCALE), 576)
    table = i32([[pages - 1, 59000], [0, pages - 2]])
    out, lse = dt.attend_paged(q, cache, i32([128, 100]), table, 512, SCALE)
    rows = cache[table.long()].reshape(2, 128, 576)
    want = serve_plain.attend(q, rows.reshape(-1, 576), 512, SCALE, [np.arange(128), 128 + np.arange(100)])
    close(out, lse, want, logit_size(q, rows, SCALE), 576)


def test_empty_calls():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(7)
    q, cache = make(g, 2, 16, 512, 4, 64, "bf16")
    out, lse = dt.attend_selected(q, cache, torch.empty(2, 0, dtype=torch.int32, device=DEV), 512, SCALE)
    assert (out == 0).all() and (lse == -math.inf).all()
    out, lse = dt.attend_selected(q[:0], cache, torch.empty(0, 9, dtype=torch.int32, device=DEV), 512, SCALE)
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
    out, lse = dt.attend_selected(q, cache[:0], i32([[0, 1, -1], [5, 5, 5]]), 512, SCALE)
    assert (out == 0).all() and (lse == -math.inf).all()


# -------------------------------------------------------------------------
# expanded form


def check_expanded(q_lens, k_lens, heads, kind, causal=True, joined=True, extra=0):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(sum(q_lens) + heads)
    q_starts = np.concatenate([[0], np.cumsum(q_lens)])
    k_starts = np.concatenate([[0], np.cumsum(k_lens)])
    tq, tk = int(q_starts[-1]) + extra, int(k_starts[-1])
    t = TYPES[kind]
    q = torch.randn(tq, heads, 192, generator=g, device=DEV).to(t)
    if joined:
        kv = torch.randn(tk, heads, 256, generator=g, device=DEV).to(t)
        k, v = kv[..., :128], kv[..., 128:]
    else:
        k = torch.randn(tk, heads, 128, generator=g, device=DEV).to(t)
        v = torch.randn(tk, heads, 128, generator=g, device=DEV).to(t)
    rope = torch.randn(tk, 64, generator=g, device=DEV).to(t)
    out = torch.full((tq, heads, 128), 7.0, dtype=t, device=DEV)
    lse = torch.full((tq, heads), 7.0, device=DEV)
    dt.attend_expanded(q, k, v, rope, i32(q_starts), i32(k_starts), max(q_lens), SCALE,
                       causal=causal, out=out, lse=lse)
    torch.cuda.synchronize()
    want = serve_plain.expand(q, k, v, rope, q_starts.tolist(), k_starts.tolist(), SCALE, causal)
    n = int(q_starts[-1])
    size = 0.0
    if tk:
        size = float((q.float().abs().flatten(0, 1).max(0).values * torch.cat(
            [k.float().abs().flatten(0, 1).max(0).values, rope.float().abs().max(0).values])).sum() * SCALE)
    close(out[:n], lse[:n], tuple(w[:n] for w in want), size, 192)
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("q_lens,k_lens,heads", [
    ([1], [1], 1),
    ([1, 1, 1], [1, 64, 65], 3),
    ([128, 129, 31], [128, 129, 31], 2),
    ([5, 0, 70], [200, 9, 70], 1),
    ([33, 1], [513, 700], 5),
    ([300], [300], 1),
])
def test_expanded(kind, q_lens, k_lens, heads):
    check_expanded(q_lens, k_lens, heads, kind)


@pytest.mark.parametrize("q_lens,k_lens,heads,kind", [
    ([2, 130, 1], [3000, 2050, 1], 1, "bf16"),   # parts of many sizes, and empty ones
    ([40, 0, 7], [5000, 10, 600], 2, "fp16"),
    ([1], [20000], 1, "bf16"),
])
def test_expanded_split_over_keys(q_lens, k_lens, heads, kind):
    import row_top_selection_amd as dt

    assert dt.expanded_bytes(len(q_lens), heads, sum(q_lens) + 3, sum(k_lens), max(q_lens)) > 0
    check_expanded(q_lens, k_lens, heads, kind, extra=3)


def test_expanded_wide_workgroups():
    """Enough rows for eight waves a workgroup: odd lengths, a prompt shorter
    than the longest by more than a workgroup's rows, keys that end inside a
    tile and inside its halves."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(12)
    q_lens, k_lens, heads = [515, 300, 1, 600, 512], [517, 333, 65, 631, 512], 64
    qs, ks = np.concatenate([[0], np.cumsum(q_lens)]), np.concatenate([[0], np.cumsum(k_lens)])
    q, k, v, rope = (torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16) for s in (
        (qs[-1], heads, 192), (ks[-1], heads, 128), (ks[-1], heads, 128), (ks[-1], 64)))
    out, lse = dt.attend_expanded(q, k, v, rope, i32(qs), i32(ks), 600, SCALE)
    torch.cuda.synchronize()
    # heads apart: each as a batch of its own, by the narrow kernel
    for h in (0, 17, 63):
        one = [t[:, h:h + 1] for t in (q, k, v)]
        a = dt.attend_expanded(*one, rope, i32(qs), i32(ks), 600, SCALE)
        size = float((one[0].float().abs().flatten(0, 1).max(0).values * torch.cat(
            [one[1].float().abs().flatten(0, 1).max(0).values, rope.float().abs().max(0).values])).sum() * SCALE)
        rows = [0, 1, 255, 256, 514, 515, 814, 815, 816, 1415, 1416, 1927]
        want_out = torch.zeros(len(rows), 1, 128, dtype=torch.float64)
        want_lse, want_size = torch.zeros(len(rows), 1, dtype=torch.float64), torch.zeros_like(want_out)
        for n, i in enumerate(rows):
            r = int(np.searchsorted(qs, i, side="right")) - 1
            end = int(ks[r]) + i - int(qs[r]) + 1 + k_lens[r] - q_lens[r]
            kv = slice(int(ks[r]), end)
            o, l, s = serve_plain.expand(one[0][i:i + 1], one[1][kv], one[2][kv], rope[kv], [0, 1],
                                         [0, end - int(ks[r])], SCALE, False)
            want_out[n], want_lse[n], want_size[n] = o[0], l[0], s[0]
        for got in (a, (out[:, h:h + 1], lse[:, h:h + 1])):
            close(got[0][rows], got[1][rows], (want_out, want_lse, want_size), size, 192)


@pytest.mark.parametrize("causal", [True, False])
def test_expanded_queries_without_keys(causal):
    """Requests with fewer keys than queries (the first queries see none),
    with no keys at all, and rows behind the last request."""
    check_expanded([10, 40, 3, 140], [4, 0, 3, 70], 2, "bf16", causal=causal, joined=False, extra=5)


def test_expanded_without_any_key():
    check_expanded([3], [0], 2, "bf16")


def test_expanded_without_causality():
    check_expanded([40, 130], [100, 65], 2, "fp16", causal=False)


def test_expanded_hidden_keys_may_hold_anything():
    """Keys (not values) that causality hides, and everything of other
    requests and behind the last one."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(8)
    q, k, v, rope = (torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
                     for s in ((90, 2, 192), (300, 2, 128), (300, 2, 128), (300, 64)))
    starts = i32([0, 90]), i32([60, 150])
    a = dt.attend_expanded(q, k, v, rope, *starts, 90, SCALE)
    for t in (k, v, rope):
        t[:60] = float("nan")
        t[150:] = float("inf")
    b = dt.attend_expanded(q, k, v, rope, *starts, 90, SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(b[0]).all()
    # query 0 of 90 sees key 0 alone: keys 1 .. 89 hidden from it hold infinities
    k[61:150] = float("inf")
    c = dt.attend_expanded(q, k, v, rope, *starts, 90, SCALE)
    assert torch.equal(c[0][0], a[0][0]) and torch.equal(c[1][0], a[1][0])


def test_expanded_logits_of_every_size():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(9)
    n = 400
    k = torch.randn(n, 1, 128, generator=g, device=DEV)
    k[:, 0, 0] = torch.arange(n, device=DEV) * 0.5
    k, rope = k.to(torch.bfloat16), torch.zeros(n, 64, dtype=torch.bfloat16, device=DEV)
    v = torch.randn(n, 1, 128, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.zeros(4, 1, 192, device=DEV)
    q[0, 0, 0], q[1, 0, 0], q[3, 0, 1] = 1.0, -1.0, 200.0
    q = q.to(torch.bfloat16)
    out, lse = dt.attend_expanded(q, k, v, rope, i32([0, 4]), i32([0, n]), 4, 1.0, causal=False)
    torch.cuda.synchronize()
    want = serve_plain.expand(q, k, v, rope, [0, 4], [0, n], 1.0, False)
    for b in range(4):
        size = float((q[b, 0, :128].float().abs() @ k[:, 0].float().abs().T).max())
        close(out[b:b + 1], lse[b:b + 1], tuple(w[b:b + 1] for w in want), size, 192)


def test_expanded_is_absorbed():
    """The two forms agree where values are the latent vectors themselves:
    one head of 128 + 64 dimensions, keys and values the same vectors."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(10)
    x = torch.randn(500, 1, 128, generator=g, device=DEV).to(torch.bfloat16)
    rope = torch.randn(500, 64, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(1, 1, 192, generator=g, device=DEV).to(torch.bfloat16)
    a = dt.attend_expanded(q, x, x, rope, i32([0, 1]), i32([0, 500]), 1, SCALE)
    wide_q = torch.zeros(1, 1, 320, dtype=torch.bfloat16, device=DEV)
    wide_q[..., :128], wide_q[..., 256:] = q[..., :128], q[..., 128:]
    cache = torch.zeros(1, 512, 320, dtype=torch.bfloat16, device=DEV)
    cache[0, :500, :128], cache[0, :500, 256:] = x[:, 0], rope
    b = dt.attend_paged(wide_q, cache, i32([500]), i32([[0]]), 256, SCALE)
    # both round weights (2^-8 of the values' weighted sizes) and outputs
    size = serve_plain.expand(q, x, x, rope, [0, 1], [0, 500], SCALE)[2][0, 0]
    diff = (a[0][0, 0].cpu().double() - b[0][0, 0, :128].cpu().double()).abs()
    assert (diff <= 4 * 2.0 ** -8 * size).all()
    assert abs(float(a[1][0, 0] - b[1][0, 0])) < 1e-5 * abs(float(a[1][0, 0]))


def test_expanded_graph_replays_follow_the_lengths():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(11)
    rng = np.random.default_rng(11)
    q, k, v, rope = (torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
                     for s in ((200, 4, 192), (900, 4, 128), (900, 4, 128), (900, 64)))
    qs, ks = i32([0, 100, 200]), i32([0, 500, 900])
    out, lse = dt.attend_expanded(q, k, v, rope, qs, ks, 200, SCALE)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dt.attend_expanded(q, k, v, rope, qs, ks, 200, SCALE, out=out, lse=lse)
    for _ in range(4):
        qs.copy_(i32([0, rng.integers(0, 201), 200]))
        ks.copy_(i32([0, rng.integers(0, 901), 900]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = dt.attend_expanded(q, k, v, rope, qs, ks, 200, SCALE)
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])


@pytest.mark.parametrize("heads,k,pages", [(64, 300, 9), (128, 2048, 100), (32, 257, 1000), (17, 640, 3)])
def test_selected_many_rows(heads, k, pages):
    """Batches of prompt rows: more rows than the card has CUs, of every
    length, with holes and repeated slots."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads)
    rng = np.random.default_rng(heads)
    rows = 513
    q, cache = make(g, rows, heads, 512, pages, 64, "bf16")
    slots = rng.integers(0, pages * 64, (rows, k))
    slots[rng.random((rows, k)) < 0.1] = -1
    slots[np.arange(k) >= rng.integers(0, k + 1, rows)[:, None]] = -1
    slots[0], slots[1], slots[2, 0] = -1, 7, pages * 64
    out, lse = dt.attend_selected(q, cache, i32(slots), 512, SCALE)
    again = dt.attend_selected(q, cache, i32(slots), 512, SCALE)
    torch.cuda.synchronize()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    some = [0, 1, 2, 3, 100, 255, 256, 511, 512]
    picked = [s[(s >= 0) & (s < pages * 64)] for s in slots[some]]
    vectors = cache.view(-1, 576)
    want = serve_plain.attend(q[some], vectors, 512, SCALE, picked)
    close(out[some], lse[some], want, logit_size(q, vectors, SCALE), 576)
    # a batch of the same rows that is split
    few = dt.attend_selected(q[some], cache, i32(slots[some]), 512, SCALE)
    close(few[0], few[1], want, logit_size(q, vectors, SCALE), 576)
