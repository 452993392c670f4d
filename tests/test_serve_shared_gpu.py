"""Attention behind shared tokens, absorbed, on the GPU against the definition in
64 bits (tests/serve_plain.py)."""
import math

import numpy as np
import pytest
import torch

from tests import serve_plain
from tests.test_serve_attend_gpu import SCALE, TYPES, close, i32, logit_size, make

pytestmark = pytest.mark.gpu

DEV = "cuda"


def batch(rng, rows_of, shared, own, page):
    """A batch: (table [rows, width], lens, starts, pages). Every row has pages of its own, also in the place of
    what it shares, where only the first row's count."""
    rows = sum(rows_of)
    starts = np.concatenate([[0], np.cumsum(rows_of)])
    lens = np.zeros(rows, dtype=np.int64)
    width = -(-max(max(shared) + max(own), 1) // page) + 2
    pages = rows * width + 1
    table = rng.permutation(pages - 1).reshape(rows, width) + 1
    for g in range(len(rows_of)):
        for r in range(starts[g], starts[g + 1]):
            lens[r] = shared[g] + own[r % len(own)]
    return table, lens, starts, pages


def picked(table, table_rows, lens, starts, shared, page):
    """The cache slots that each row reads."""
    got, most = [], table.shape[1] * page
    for b, n in enumerate(lens):
        g = max(i for i in range(len(starts) - 1) if starts[i] <= b < starts[i + 1])
        j = np.arange(min(max(0, n), most))
        line = np.where(j < shared[g], table_rows[starts[g]], table_rows[b])
        got.append(table[line, j // page] * page + j % page)
    return got


def check(dt, q, cache, lens, table, starts, shared, latent, page, table_rows=None, **kw):
    out, lse = dt.attend_shared(q, cache, i32(lens), i32(table), i32(starts), i32(shared), latent, SCALE,
                                table_rows=None if table_rows is None else i32(table_rows), **kw)
    torch.cuda.synchronize()
    rows = np.arange(len(lens)) if table_rows is None else table_rows
    vectors = cache.view(-1, latent + 64)
    want = serve_plain.attend(q, vectors, latent, SCALE, picked(table, rows, lens, starts, shared, page))
    close(out, lse, want, logit_size(q, vectors, SCALE), latent + 64)
    return out, lse


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,latent,page,rows_of,shared,own", [
    (16, 512, 64, [1], [0], [1]),
    (16, 512, 64, [8], [640], [0, 1, 63, 64, 65, 200]),
    (16, 512, 1, [3, 1, 12], [65, 7, 130], [3, 0, 40]),
    (8, 256, 16, [5, 0, 9], [500, 33, 31], [16, 17]),
    (1, 512, 16, [70], [129], [5, 9, 0]),
    (24, 512, 64, [2, 3], [100, 1000], [70]),
    (32, 256, 64, [1, 1, 1], [64, 0, 300], [20, 64]),
    (40, 512, 16, [7, 2], [333, 64], [31, 2, 0]),
    (64, 512, 128, [3, 1], [257, 512], [129]),
    (100, 512, 64, [2, 2], [200, 63], [65, 0]),
    (128, 512, 64, [4], [1000], [33, 64]),
    (128, 256, 16, [1, 3], [31, 97], [16]),
    (200, 512, 4, [3], [90], [3, 50]),
])
def test_shared(kind, heads, latent, page, rows_of, shared, own):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads * len(own))
    rng = np.random.default_rng(heads + page)
    table, lens, starts, pages = batch(rng, rows_of, shared, own, page)
    q, cache = make(g, sum(rows_of), heads, latent, pages, page, kind)
    first = check(dt, q, cache, lens, table, starts, shared, latent, page)
    # bounds that are too small, or exact, change how the tokens are split and nothing else
    for bounds in ((max(max(shared), 1), max(own)), (1, 1), (70, 1), (1, 300), (100000, 1)):
        check(dt, q, cache, lens, table, starts, shared, latent, page, max_shared_len=bounds[0], max_own_len=bounds[1])
    again = check(dt, q, cache, lens, table, starts, shared, latent, page)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,latent,page,per,lens", [
    (16, 512, 64, 4, [0, 1, 2, 3, 4, 64, 65, 700]),
    (16, 512, 16, 2, [300, 31, 32, 33]),
    (40, 256, 1, 3, [5, 130]),
    (128, 512, 64, 2, [64, 1, 257]),
    (3, 512, 64, 40, [100, 20]),
])
def test_drafted_rows(kind, heads, latent, page, per, lens):
    """Rows of a request, each of which sees one token more than the one before it: the group shares
    all of them. Rows before a request's first token see nothing."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads + per)
    rng = np.random.default_rng(heads)
    n, width = len(lens), -(-max(lens) // page) + 1
    q, cache = make(g, n * per, heads, latent, n * width, page, kind)
    table = rng.permutation(n * width).reshape(n, width)
    row_lens = np.array([x - (per - 1) + i for x in lens for i in range(per)])
    rows, starts = np.arange(n * per) // per, np.arange(n + 1) * per
    for kw in (dict(), dict(max_shared_len=max(lens), max_own_len=0), dict(max_shared_len=1, max_own_len=0), dict(max_own_len=50)):
        check(dt, q, cache, row_lens, table, starts, lens, latent, page, table_rows=rows, **kw)


def test_zero_bounds():
    """No shared tokens: every row's own table from its start. No own ones: nothing past the shared."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(3)
    rng = np.random.default_rng(3)
    table, lens, starts, pages = batch(rng, [3, 4], [100, 37], [20, 0, 5], 16)
    q, cache = make(g, 7, 16, 512, pages, 16, "bf16")
    at = (i32(lens), i32(table), i32(starts), i32([100, 37]), 512, SCALE)
    vectors = cache.view(-1, 576)
    rows = [table[b, np.arange(n) // 16] * 16 + np.arange(n) % 16 for b, n in enumerate(lens)]
    want = serve_plain.attend(q, vectors, 512, SCALE, rows)
    for kw in (dict(max_shared_len=0), dict(max_shared_len=0, max_own_len=60), dict(max_shared_len=0, max_own_len=0)):
        close(*dt.attend_shared(q, cache, *at, **kw), want, logit_size(q, vectors, SCALE), 576)
    out, lse = dt.attend_shared(q, cache, *at, max_own_len=0)
    cut = np.minimum(lens, [100] * 3 + [37] * 4)
    close(out, lse, serve_plain.attend(q, vectors, 512, SCALE, picked(table, np.arange(7), cut, starts, [100, 37], 16)),
          logit_size(q, vectors, SCALE), 576)


def test_lengths_and_starts_at_their_ends():
    """Empty rows, negative lengths, shared lengths past the table and below 0, starts that leave rows out at
    either end, empty groups."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(4)
    rng = np.random.default_rng(4)
    page, width, rows = 16, 5, 9
    table = rng.permutation(rows * width).reshape(rows, width)
    q, cache = make(g, rows, 16, 512, rows * width, page, "bf16")
    lens = np.array([0, -3, 80, 10, 1, 79, 33, 0, 64])
    for starts, shared in (([0, 3, 3, 9], [40, 5, 30]), ([2, 3, 3, 7], [40, 5, 30]), ([0, 9], [10 ** 6]), ([0, 9], [-7]),
                           ([0, 1, 2, 3, 4, 5, 6, 7, 8, 9], [0, 16, 1, 80, 2, 33, 1000, 5, 63]), ([0, 0, 0, 9, 9], [9, 9, 17, 9])):
        real = [0, *starts[1:-1], rows]
        check(dt, q, cache, lens, table, real, shared, 512, page)
        out, lse = dt.attend_shared(q, cache, i32(lens), i32(table), i32(starts), i32(shared), 512, SCALE)
        want, want_lse = dt.attend_shared(q, cache, i32(lens), i32(table), i32(real), i32(shared), 512, SCALE)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # rows longer than the table are cut at its end
    check(dt, q, cache, lens + 500, table, [0, 9], [70], 512, page)


@pytest.mark.parametrize("groups", [63, 64, 65, 130, 4200])
def test_many_groups(groups):
    """Groups are found 64 at a time."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(groups)
    rng = np.random.default_rng(groups)
    rows_of = rng.integers(0, 3, groups)
    rows, page, width = int(rows_of.sum()), 4, 5
    starts = np.concatenate([[0], np.cumsum(rows_of)])
    table = rng.integers(0, 500, (rows, width))
    lens, shared = rng.integers(0, 17, rows), rng.integers(0, 14, groups)
    q, cache = make(g, rows, 2, 256, 500, page, "bf16")
    out, lse = dt.attend_shared(q, cache, i32(lens), i32(table), i32(starts), i32(shared), 256, SCALE)
    group = np.searchsorted(starts, np.arange(rows), side="right") - 1
    rows_read = []
    for b, n in enumerate(lens):
        j = np.arange(n)
        rows_read.append(table[np.where(j < shared[group[b]], starts[group[b]], b), j // page] * page + j % page)
    vectors = cache.view(-1, 320)
    close(out, lse, serve_plain.attend(q, vectors, 256, SCALE, rows_read), logit_size(q, vectors, SCALE), 320)


def test_pages_that_are_not_there():
    """Entries outside the cache, in shared and in own parts, are skipped; a row of nothing else is zeros."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(6)
    rng = np.random.default_rng(6)
    page, width, rows, pages = 16, 8, 6, 30
    table = rng.integers(-20, 50, (rows, width))
    table[0, 1], table[2] = 2 ** 31 - 1, -1
    table[5] = 10 ** 6
    q, cache = make(g, rows, 16, 512, pages, page, "bf16")
    lens, starts, shared = np.array([128, 100, 77, 128, 90, 128]), [0, 2, 5, 6], [60, 50, 0]
    out, lse = dt.attend_shared(q, cache, i32(lens), i32(table), i32(starts), i32(shared), 512, SCALE)
    rows_of = []
    for b, at in enumerate(picked(table, np.arange(rows), lens, starts, shared, page)):
        rows_of.append(at[(at >= 0) & (at < pages * page)])
    assert not len(rows_of[5]) and len(rows_of[0])
    vectors = cache.view(-1, 576)
    close(out, lse, serve_plain.attend(q, vectors, 512, SCALE, rows_of), logit_size(q, vectors, SCALE), 576)


def test_nothing_unseen_is_read():
    """Infinities and NaN in every slot that no row sees, among them what other rows' tables have in the place
    of shared pages, and the rest of pages that end inside a tile."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(8)
    rng = np.random.default_rng(8)
    page, rows_of, shared = 32, [3, 5, 1], [75, 160, 20]
    table, lens, starts, pages = batch(rng, rows_of, shared, [9, 0, 33, 50], page)
    q, cache = make(g, 9, 16, 512, pages, page, "bf16")
    at = picked(table, np.arange(9), lens, starts, shared, page)
    seen = np.zeros(pages * page, dtype=bool)
    seen[np.concatenate(at)] = True
    bad = torch.as_tensor(np.flatnonzero(~seen), device=DEV)
    cache.view(-1, 576)[bad[::2]] = math.nan
    cache.view(-1, 576)[bad[1::2]] = math.inf
    vectors = torch.nan_to_num(cache.view(-1, 576), 0, 0, 0)
    for kw in (dict(), dict(max_shared_len=160, max_own_len=50), dict(max_shared_len=1, max_own_len=1)):
        got = dt.attend_shared(q, cache, i32(lens), i32(table), i32(starts), i32(shared), 512, SCALE, **kw)
        close(*got, serve_plain.attend(q, vectors, 512, SCALE, at), logit_size(q, vectors, SCALE), 576)
    # a group whose rows are all padding reads nothing of what it is said to share
    cache.fill_(math.nan)
    out, lse = dt.attend_shared(q, cache, i32([0] * 9), i32(table), i32(starts), i32(shared), 512, SCALE)
    assert (out == 0).all() and (lse == -math.inf).all()


def test_scores_far_below_zero():
    """Heads whose every score is far below 0, beside rows of their group that see nothing."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(11)
    page, rows = 16, 5
    table = np.arange(rows * 20).reshape(rows, 20)
    for kind in ("bf16", "fp16"):
        cache = torch.randn(rows * 20, page, 576, generator=g, device=DEV).to(TYPES[kind])
        cache[..., 512:] = 8.0
        q = torch.zeros(rows, 16, 576, device=DEV).to(TYPES[kind])
        q[..., 512:] = torch.linspace(-60, 40, rows * 16, device=DEV).view(rows, 16, 1).to(TYPES[kind])
        lens = np.array([200, 0, 170, 0, 300])
        for starts, shared in (([0, 5], [180]), ([0, 2, 5], [64, 300])):
            check(dt, q, cache, lens, table, starts, shared, 512, page)
            check(dt, q, cache, lens, table, starts, shared, 512, page, max_shared_len=300, max_own_len=120)


def test_strides_outputs_and_workspace():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(12)
    rng = np.random.default_rng(12)
    rows_of, shared, page = [4, 2], [300, 100], 16
    table, lens, starts, pages = batch(rng, rows_of, shared, [40, 7], page)
    q, cache = make(g, 6, 16, 512, pages, page, "bf16")
    at = (i32(lens), i32(table), i32(starts), i32(shared), 512, SCALE)
    kw = dict(max_shared_len=300, max_own_len=40)
    want, want_lse = dt.attend_shared(q, cache, *at, **kw)
    wide_q = torch.zeros(6, 17, 640, device=DEV).bfloat16()
    wide_q[:, 1:, 32:608] = q
    wide = torch.full((pages, page + 1, 640), math.nan, device=DEV).bfloat16()
    wide[:, :page, 64:] = cache
    wide_table = torch.full((6, table.shape[1] + 3), -1, dtype=torch.int32, device=DEV)
    wide_table[:, 2:2 + table.shape[1]] = i32(table)
    need = dt.shared_bytes(6, 16, 512, 2, 300, 40)
    assert need > 0
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    work = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaN
    got = dt.attend_shared(wide_q[:, 1:, 32:608], wide[:, :page, 64:], at[0], wide_table[:, 2:2 + table.shape[1]], *at[2:],
                           out=out, lse=lse, workspace=work, **kw)
    assert got[0].data_ptr() == out.data_ptr() and torch.equal(out, want) and torch.equal(lse, want_lse)
    with pytest.raises(dt.DsatopkError) as e:
        dt.attend_shared(q, cache, *at, workspace=work[:need - 16], **kw)
    assert e.value.status == 6


def test_cache_past_32_bits_of_bytes():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(13)
    pages = 60000  # 4.4 GB
    cache = torch.zeros(pages, 64, 576, device=DEV, dtype=torch.bfloat16)
    table = np.array([[pages - 1, 5, pages - 2], [3, pages - 3, 59000], [0, 58999, 7]])
    for p in set(table.flatten().tolist()):
        cache[p] = torch.randn(64, 576, generator=g, device=DEV).bfloat16()
    q = torch.randn(3, 16, 576, generator=g, device=DEV).bfloat16()
    lens, starts, shared = np.array([190, 150, 192]), [0, 3], [100]
    out, lse = dt.attend_shared(q, cache, i32(lens), i32(table), i32(starts), i32(shared), 512, SCALE)
    at = picked(table, np.arange(3), lens, starts, shared, 64)
    every = np.unique(np.concatenate(at))
    vectors = cache.view(-1, 576)[torch.as_tensor(every, device=DEV)]
    want = serve_plain.attend(q, vectors, 512, SCALE, [np.searchsorted(every, x) for x in at])
    close(out, lse, want, logit_size(q, vectors, SCALE), 576)


def test_captured_and_replayed_on_two_streams():
    """Two graphs with workspaces of their own, replayed at once; lengths, groups and queries change between
    replays, within the bounds that the graphs were captured with."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(14)
    rng = np.random.default_rng(14)
    rows, page, width = 12, 16, 40
    table = i32(rng.permutation(rows * width).reshape(rows, width))
    sides = []
    for _ in range(2):
        q, cache = make(g, rows, 16, 512, rows * width, page, "bf16")
        sides.append(dict(q=q, cache=cache, lens=i32([0] * rows), starts=i32([0, 4, 8, 12]), shared=i32([0] * 3), stream=torch.cuda.Stream()))

    def call(s):
        return dt.attend_shared(s["q"], s["cache"], s["lens"], table, s["starts"], s["shared"], 512, SCALE, max_shared_len=500, max_own_len=140)

    for s in sides:
        call(s)
        torch.cuda.synchronize()
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"]):
            s["out"] = call(s)
    for n in range(4):
        for s in sides:
            s["q"].copy_(torch.randn(rows, 16, 576, generator=g, device=DEV).bfloat16())
            s["shared"].copy_(i32(rng.integers(0, 500, 3)))
            s["starts"].copy_(i32([0, *sorted(rng.integers(0, rows + 1, 2)), rows]))
            s["lens"].copy_(i32(rng.integers(0, 640, rows)))
        torch.cuda.synchronize()
        for s in sides:
            with torch.cuda.stream(s["stream"]):
                s["graph"].replay()
        torch.cuda.synchronize()
        for s in sides:
            want = call(s)
            torch.cuda.synchronize()
            assert torch.equal(s["out"][0], want[0]) and torch.equal(s["out"][1], want[1]), n


def test_no_rows_is_no_error():
    import row_top_selection_amd as dt

    q, cache = torch.zeros(0, 16, 576, device=DEV).bfloat16(), torch.zeros(1, 16, 576, device=DEV).bfloat16()
    none = i32([])
    out, lse = dt.attend_shared(q, cache, none, torch.zeros(0, 2, dtype=torch.int32, device=DEV), i32([0]), none, 512, SCALE)
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
    # no pages at all: nothing is there to read
    q = torch.ones(3, 16, 576, device=DEV).bfloat16()
    out, lse = dt.attend_shared(q, cache[:0], i32([5, 9, 0]), i32([[0], [0], [0]]), i32([0, 3]), i32([4]), 512, SCALE)
    assert (out == 0).all() and (lse == -math.inf).all()
