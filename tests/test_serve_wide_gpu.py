"""Attention behind shared tokens for many heads a workgroup: references that
are outgrown, numbers that are none, tokens that are not there, and every way
that tiles, pages and blocks of lanes can meet."""
import math

import numpy as np
import pytest
import torch

from tests import serve_plain
from tests.test_serve_attend_gpu import SCALE, TYPES, close, i32, logit_size, make
from tests.test_serve_shared_gpu import batch, check, picked

pytestmark = pytest.mark.gpu

DEV = "cuda"
WIDE = dict(max_shared_len=1 << 22)  # a bound by which calls take 128 heads a workgroup (it is one, if not a near one)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("way", [1, -1])
def test_scores_that_rise_and_fall(kind, way):
    """Scores of up to 200 either way, by head, along 1500 tokens: the reference of a part is outgrown many
    times, of some heads at every tile, of others never."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(21)
    page, rows, shared = 64, 9, 1500
    width = -(-(shared + 70) // page)
    table = np.arange(rows * width).reshape(rows, width)
    cache = torch.randn(rows * width, page, 576, generator=g, device=DEV)
    at = torch.arange(rows * width * page, device=DEV) % (width * page)
    cache.view(-1, 576)[:, 512:] = (8.0 * (at if way > 0 else width * page - at) / (width * page))[:, None]
    q = torch.zeros(rows, 16, 576, device=DEV)
    q[..., 512:] = torch.linspace(-6, 6, rows * 16, device=DEV).view(rows, 16, 1)
    cache, q = cache.to(TYPES[kind]), q.to(TYPES[kind])
    lens = shared + np.array([0, 5, 70, 1, 33, 64, 0, 2, 31])
    for kw in (dict(), dict(max_shared_len=1, max_own_len=1), dict(max_shared_len=shared, max_own_len=70), WIDE):
        check(dt, q, cache, lens, table, [0, rows], [shared], 512, page, **kw)


def test_references_outgrown_in_a_long_part():
    """As above, with so many heads that every workgroup has several hundred tokens."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(24)
    page, rows, shared = 64, 24, 3500
    width = -(-(shared + 9) // page)
    table = np.arange(rows * width).reshape(rows, width)
    cache = torch.randn(rows * width, page, 576, generator=g, device=DEV)
    at = torch.arange(rows * width * page, device=DEV) % (width * page)
    cache.view(-1, 576)[:, 512:] = (8.0 * at / (width * page))[:, None]
    q = torch.zeros(rows, 128, 576, device=DEV)
    q[..., 512:] = torch.linspace(-9, 9, rows * 128, device=DEV)[torch.randperm(rows * 128, generator=g, device=DEV)].view(rows, 128, 1)
    lens = np.minimum(np.arange(rows) * 200 - 100, shared + 9)
    check(dt, q.bfloat16(), cache.bfloat16(), lens, table, [0, rows], [shared], 512, page, **WIDE)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("where", [0, 40, 777, 1290])
@pytest.mark.parametrize("kw", [{}, WIDE], ids=["few", "wide"])
def test_an_infinite_or_absent_number(bad, where, kw):
    """One token's first rotary element: heads whose query makes the score -inf do not see the token, others
    give NaN, and rows that end before it know nothing of it."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(22)
    page, rows, shared = 16, 10, 1300
    width = -(-shared // page) + 2
    table = np.arange(rows * width).reshape(rows, width)
    q, cache = make(g, rows, 16, 512, rows * width, page, "bf16")
    sign = torch.ones(rows, 16, device=DEV)
    sign[:, ::2] = -1
    q[..., 512] = sign.bfloat16()
    cache.view(-1, 576)[where, 512] = bad
    lens = np.array([shared + 10, where, 0, shared, where + 1, shared + 20, 3, where + 33, shared, 1])
    sees = torch.as_tensor(lens > where, device=DEV)[:, None].expand(-1, 16)
    out, lse = dt.attend_shared(q, cache, i32(lens), i32(table), i32([0, rows]), i32([shared]), 512, SCALE, **kw)
    torch.cuda.synchronize()
    if math.isnan(bad):
        numbers = ~sees
    else:
        numbers = ~sees | (sign * bad < 0)
    assert torch.isnan(out[~numbers]).all()
    vectors = cache.view(-1, 576).clone()
    vectors[where, 512] = 0.0
    at = [x[x != where] if s else x for x, s in zip(picked(table, np.arange(rows), lens, [0, rows], [shared], page), sees[:, 0].tolist())]
    want = serve_plain.attend(q, vectors, 512, SCALE, at)
    close(out[numbers], lse[numbers], tuple(x[numbers.cpu()] for x in want), logit_size(q, vectors, SCALE), 576)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,page,rows_of,shared,own", [
    (16, 1, [9], [700], [0, 1, 90]),                       # a block and a part of one
    (16, 16, [8, 17], [33, 1000], [31, 32, 33]),
    (40, 4, [5, 4, 6], [95, 96, 97], [300, 0]),            # blocks that end inside a row's heads
    (128, 64, [3, 1, 2], [31, 0, 450], [1, 130]),
    (129, 32, [2], [200], [65]),
    (300, 64, [1, 2], [64, 127], [40]),
])
def test_lanes_tiles_and_pages(kind, heads, page, rows_of, shared, own):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads + page)
    rng = np.random.default_rng(heads + page)
    table, lens, starts, pages = batch(rng, rows_of, shared, own, page)
    q, cache = make(g, sum(rows_of), heads, 512, pages, page, kind)
    for bounds in ((None, None), (1, 1), (1, 5000), (5000, 1), (1 << 22, 1), (1 << 22, 1 << 20)):
        check(dt, q, cache, lens, table, starts, shared, 512, page, max_shared_len=bounds[0], max_own_len=bounds[1])
    # what no row reads may hold anything
    rows = np.arange(len(lens))
    read = np.unique(np.concatenate(picked(table, rows, lens, starts, shared, page)))
    other = torch.full_like(cache, math.nan)
    other.view(-1, 576)[torch.as_tensor(read, device=DEV)] = cache.view(-1, 576)[torch.as_tensor(read, device=DEV)]
    for kw in ({}, WIDE):
        want, got = (dt.attend_shared(q, c, i32(lens), i32(table), i32(starts), i32(shared), 512, SCALE, **kw) for c in (cache, other))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_by_themselves():
    """No shared tokens, and shared ones that nobody has more than."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(23)
    rng = np.random.default_rng(23)
    table, lens, starts, pages = batch(rng, [6, 5], [0, 0], [0, 1, 500, 64], 16)
    q, cache = make(g, 11, 128, 512, pages, 16, "bf16")
    a = check(dt, q, cache, lens, table, starts, [0, 0], 512, 16)
    b = check(dt, q, cache, lens, table, starts, [0, 0], 512, 16, max_shared_len=0)
    assert torch.equal(a[0][lens == 0], b[0][lens == 0]) and (a[0][lens == 0] == 0).all()
    check(dt, q, cache, np.minimum(lens, 300), table, starts, [300, 300], 512, 16, max_own_len=0)
    check(dt, q, cache, np.minimum(lens, 300), table, starts, [300, 300], 512, 16, max_own_len=0, **WIDE)
    check(dt, q, cache, lens, table, starts, [0, 0], 512, 16, max_own_len=1 << 20, **WIDE)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [8, 16, 40, 64, 128])
def test_smaller_vectors(heads, kind):
    """Latent vectors of 256: 128 heads a workgroup, and rows of few, some and all of them."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads)
    rng = np.random.default_rng(heads)
    table, lens, starts, pages = batch(rng, [17, 9], [300, 65], [70, 0, 33], 16)
    q, cache = make(g, 26, heads, 256, pages, 16, kind)
    for kw in (WIDE, dict(WIDE, max_own_len=1 << 18), dict(WIDE, max_own_len=0)):
        lens_of = np.minimum(lens, [300] * 17 + [65] * 9) if kw.get("max_own_len") == 0 else lens
        check(dt, q, cache, lens_of, table, starts, [300, 65], 256, 16, **kw)


def test_jobs_one_after_the_other():
    """So many short groups that every workgroup has several, by the calls with 32, 64 and 128 lanes."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(25)
    rng = np.random.default_rng(25)
    for rows_of, heads, kw in (([1] * 900, 16, {}), ([3] * 900, 16, {}), ([1] * 700, 128, WIDE)):
        shared = rng.integers(0, 90, len(rows_of)).tolist()
        table, lens, starts, pages = batch(rng, rows_of, shared, [0, 3, 40, 1], 32)
        q, cache = make(g, sum(rows_of), heads, 512, pages, 32, "bf16")
        first = check(dt, q, cache, lens, table, starts, shared, 512, 32, **kw)
        again = dt.attend_shared(q, cache, i32(lens), i32(table), i32(starts), i32(shared), 512, SCALE, **kw)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
