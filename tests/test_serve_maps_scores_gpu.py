"""Page maps and indexer scores on the GPU against their definitions in 64
bits (tests/serve_plain.py)."""
import numpy as np
import pytest
import torch

from tests import serve_plain

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(v):
    return torch.as_tensor(np.asarray(v, dtype=np.int32)).to(DEV)


# -------------------------------------------------------------------------
# page maps


def check_maps(seq_lens, new_lens, page, width, num_free, tokens, seed=0, stride=None):
    import row_top_selection_amd as dt

    rng = np.random.default_rng(seed)
    n = len(seq_lens)
    pool = rng.permutation(n * width + num_free).astype(np.int32)
    table = pool[:n * width].reshape(n, width)
    free = pool[n * width:]
    want = serve_plain.page_maps(seq_lens, new_lens, table, page, free, tokens)
    whole = torch.full((n + 1, stride or width), -7, dtype=torch.int32, device=DEV)
    whole[:n, :width] = i32(table)
    got = dt.page_maps(i32(seq_lens), whole[:n, :width], page, i32(free), tokens,
                       new_lens=None if new_lens is None else i32(new_lens))
    torch.cuda.synchronize()
    for name in ("token_starts", "slots", "table_rows", "row_lens", "counts"):
        assert getattr(got, name).tolist() == list(want[name]), name
    back = whole.cpu().numpy()
    assert (back[:n, :width] == want["table"]).all()
    assert (back[n] == -7).all() and (back[:, width:] == -7).all()


@pytest.mark.parametrize("page", [1, 2, 16, 64, 1 << 20])
@pytest.mark.parametrize("n", [1, 3, 255, 256, 1024, 1025, 2500])
def test_maps_one_token_each(n, page):
    rng = np.random.default_rng(n + page)
    lens = rng.integers(0, 200, n)
    check_maps(lens, None, page, -(-200 // page), n, n + 3, seed=n)


@pytest.mark.parametrize("page", [1, 16, 64])
def test_maps_uneven_prompts(page):
    rng = np.random.default_rng(page)
    lens = np.concatenate([[0, 1, 5, 0, 0, 2500], rng.integers(0, 900, 60), [0, 0, 1]])
    new = np.array([rng.integers(0, x + 1) for x in lens])
    new[5] = 2500
    check_maps(lens, new, page, -(-2500 // page), int(new.sum()) + 9, -(-int(new.sum()) // 64) * 64,
               stride=-(-2500 // page) + 5)


def test_maps_more_requests_than_a_pass_with_prompts():
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 40, 2300)
    new = np.array([rng.integers(0, x + 1) for x in lens])
    check_maps(lens, new, 8, 5, int(new.sum()), int(new.sum()) + 1000)


def test_maps_lengths_that_ask_for_nothing_or_too_much():
    # negative lengths, more new tokens than the length, negative new tokens
    check_maps([-5, 7, 9, 0, 3], [4, 50, -2, 3, 3], 4, 3, 10, 32)


def test_maps_step_that_does_not_fit():
    check_maps([40, 40, 40], [40, 40, 40], 8, 5, 7, 128)     # free list too short
    check_maps([40, 40, 40], [40, 40, 40], 8, 3, 30, 128)    # table too narrow
    check_maps([40, 40, 40], [40, 40, 40], 8, 5, 30, 50)     # more tokens than rows
    check_maps([40, 40, 40], [40, 40, 40], 8, 5, 0, 128)     # nothing free
    check_maps([40], [40], 8, 5, 9, 0)                       # no rows at all
    check_maps([], [], 8, 5, 9, 70)                          # no requests


def test_maps_graph_replays_follow_the_lengths():
    import row_top_selection_amd as dt

    n, page, width = 37, 16, 30
    rng = np.random.default_rng(1)
    lens, table = i32(np.zeros(n)), i32(np.zeros((n, width)))
    free = i32(np.arange(1000, 1000 + n))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out = dt.page_maps(lens, table, page, free, n)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dt.page_maps(lens, table, page, free, n, out=out)
    for step in range(4):
        now, tab = rng.integers(0, 400, n), rng.integers(0, 900, (n, width))
        lens.copy_(i32(now))
        table.copy_(i32(tab))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = serve_plain.page_maps(now, None, tab, page, np.arange(1000, 1000 + n), n)
        assert out.slots.tolist() == want["slots"] and out.counts.tolist() == want["counts"]
        assert (table.cpu().numpy() == want["table"]).all()


# -------------------------------------------------------------------------
# indexer scores

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}


def close_scores(got, want, size, terms):
    """Products are exact in fp32's exponent range; a sum of `terms` fp32
    additions is off by at most terms * 2^-24 of its terms' sizes (here:
    matrix-unit sums over head_dim, then over heads, then one scaling)."""
    got = got.cpu().double()
    inside = torch.isfinite(want) & (size > 0)
    assert torch.equal(got[~inside], want[~inside])
    assert ((got - want).abs() <= terms * 2.0 ** -24 * size)[inside].all(), \
        ((got - want).abs() / size)[inside].max()


def make(g, rows, heads, dim, tokens, kind):
    q = torch.randn(rows, heads, dim, generator=g, device=DEV).to(TYPES[kind])
    w = torch.randn(rows, heads, generator=g, device=DEV)
    keys = torch.randn(*tokens, dim, generator=g, device=DEV).to(TYPES[kind])
    scales = torch.rand(*tokens, generator=g, device=DEV) + 0.5 if kind == "fp8" else None
    return q, w, keys, scales


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("heads,dim,page,lens,per", [
    (64, 128, 64, [0, 1, 63, 64, 65, 255, 256, 257, 1000], 1),
    (1, 64, 16, [5, 300, -3, 17], 1),
    (33, 128, 1, [257, 2], 1),
    (40, 64, 128, [700, 129], 3),
    (128, 128, 32, [511, 90, 1], 2),
])
def test_scores_paged(kind, heads, dim, page, lens, per):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads + dim)
    n, width = len(lens), -(-max(max(lens), 1) // page)
    rows = n * per
    q, w, keys, scales = make(g, rows, heads, dim, (n * width, page), kind)
    table = torch.randperm(n * width, generator=g, device=DEV).view(n, width).to(torch.int32)
    row_lens = [x - (per - 1) + i for x in lens for i in range(per)]
    out = torch.full((rows + 1, width * page + 8), -7.0, device=DEV)
    got = dt.scores_paged(q, w, keys, i32(row_lens), table, key_scales=scales,
                          table_rows=None if per == 1 else i32(np.arange(rows) // per), out=out[:rows])
    torch.cuda.synchronize()
    at = [table[b // per].cpu().long() for b in range(rows)]
    windows = [(0, [int(at[b][j // page]) * page + j % page for j in range(max(0, x))])
               for b, x in enumerate(row_lens)]
    want, size = serve_plain.scores(q, w, keys.view(-1, dim).float(), None if scales is None else scales.view(-1),
                                    windows, torch.full_like(got, -7.0))
    close_scores(got, want, size, dim + heads + 2)
    assert (out[rows] == -7).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("rows,heads,dim", [(1, 64, 128), (70, 24, 128), (513, 64, 64)])
def test_scores_ragged(kind, rows, heads, dim):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(rows)
    rng = np.random.default_rng(rows)
    total = 1237
    q, w, keys, scales = make(g, rows, heads, dim, (total,), kind)
    starts = rng.integers(0, total, rows)
    lens = np.minimum(rng.integers(-2, 900, rows), total - starts)
    starts[0], lens[0] = 0, total
    got = dt.scores_ragged(q, w, keys, i32(lens), i32(starts), key_scales=scales,
                           out=torch.full((rows, 1240), 1e3, device=DEV))
    torch.cuda.synchronize()
    windows = [(int(s), list(range(s, s + max(0, x)))) for s, x in zip(starts, lens)]
    want, size = serve_plain.scores(q, w, keys.float(), scales, windows, torch.full_like(got, 1e3))
    close_scores(got, want, size, dim + heads + 2)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("heads,dim", [(8, 64), (40, 128), (70, 64)])
def test_scores_of_many_rows_paged(kind, heads, dim):
    """Batches whose workgroups go over several rows: tables that change inside
    a group, rows that a tile does not reach, empty rows."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads)
    rng = np.random.default_rng(heads)
    n, per, page, width = 1200, 2, 16, 44
    rows = n * per
    q, w, keys, scales = make(g, rows, heads, dim, (400, page), kind)
    table = rng.integers(0, 400, (n, width))
    lens = rng.integers(-1, width * page + 1, rows)
    lens[rng.random(rows) < 0.3] = 0
    out = dt.scores_paged(q, w, keys, i32(lens), i32(table), key_scales=scales,
                          table_rows=i32(np.arange(rows) // per),
                          out=torch.full((rows, width * page), -7.0, device=DEV))
    torch.cuda.synchronize()
    some = np.concatenate([np.arange(12), rng.permutation(rows)[:60], [rows - 1]])
    windows = []
    for b in some:
        j = np.arange(max(0, lens[b]))
        windows.append((0, table[b // per][j // page] * page + j % page))
    want, size = serve_plain.scores(q[some], w[some], keys.view(-1, dim).float(),
                                    None if scales is None else scales.view(-1), windows,
                                    torch.full((len(some), width * page), -7.0))
    close_scores(out[torch.as_tensor(some, device=DEV)], want, size, dim + heads + 2)
    # every row, by the kernel itself a few rows at a time
    for first in (0, 1111, rows - 7):
        part = slice(first, first + 7)
        few = dt.scores_paged(q[part], w[part], keys, i32(lens[part]), i32(table), key_scales=scales,
                              table_rows=i32(np.arange(rows)[part] // per),
                              out=torch.full((7, width * page), -7.0, device=DEV))
        assert torch.equal(few, out[part])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_scores_of_many_rows_ragged(kind):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(77)
    rng = np.random.default_rng(77)
    rows, total = 5000, 2100
    q, w, keys, scales = make(g, rows, 16, 128, (total,), kind)
    starts = np.sort(rng.integers(0, total, rows))
    lens = np.minimum(rng.integers(-2, 900, rows), total - starts)
    out = dt.scores_ragged(q, w, keys, i32(lens), i32(starts), key_scales=scales,
                           out=torch.full((rows, total), 1e3, device=DEV))
    torch.cuda.synchronize()
    some = np.concatenate([np.arange(70), rng.permutation(rows)[:60], [rows - 1]])
    windows = [(int(starts[b]), np.arange(starts[b], starts[b] + max(0, lens[b]))) for b in some]
    want, size = serve_plain.scores(q[some], w[some], keys.float(), scales, windows,
                                    torch.full((len(some), total), 1e3))
    close_scores(out[torch.as_tensor(some, device=DEV)], want, size, 128 + 16 + 2)


def test_scores_with_strided_inputs():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(3)
    q, w, keys, _ = make(g, 5, 20, 128, (6, 16), "bf16")
    wide_q = torch.full((5, 24, 192), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide_q[:, :20, :128] = q
    wide_k = torch.full((6, 16, 160), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide_k[..., 8:136] = keys
    wide_w = torch.full((5, 31), float("nan"), device=DEV)
    wide_w[:, 3:23] = w
    table = i32([[0, 3], [1, 1], [2, 0], [5, 4], [4, 2]])
    lens = i32([32, 17, 1, 30, 0])
    a = dt.scores_paged(q, w, keys, lens, table, out=torch.zeros(5, 32, device=DEV))
    b = dt.scores_paged(wide_q[:, :20, :128], wide_w[:, 3:23], wide_k[..., 8:136], lens, table,
                        out=torch.zeros(5, 32, device=DEV))
    assert torch.equal(a, b) and torch.isfinite(a).all() and a.abs().sum() > 0


def test_scores_never_read_what_is_not_there():
    """Pages outside the cache read as keys of score 0; NaN in other pages, in
    the rest of a window's last page and behind the window stays there."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(4)
    q, w, keys, _ = make(g, 2, 64, 128, (8, 16), "bf16")
    keys[5] = float("nan")
    keys[3, 9:] = float("inf")
    table = i32([[2, -1, 8, 3], [1 << 30, 0, 3, 5]])
    out = dt.scores_paged(q, w, keys, i32([57, 41]), table, out=torch.full((2, 64), -7.0, device=DEV))
    torch.cuda.synchronize()
    pages = [[2, -1, -1, 3], [-1, 0, 3, 5]]
    windows = [(0, [p[j // 16] * 16 + j % 16 if p[j // 16] >= 0 else -1 for j in range(n)])
               for p, n in zip(pages, (57, 41))]
    clean = torch.nan_to_num(keys.view(-1, 128).float(), nan=9.0, posinf=9.0)
    want, size = serve_plain.scores(q, w, clean, None, windows, torch.full_like(out, -7.0))
    close_scores(out, want, size, 194)


def test_scores_infinite_and_nan_keys_stay_in_their_columns():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(5)
    q, w, keys, _ = make(g, 1, 64, 128, (300,), "bf16")
    ref = dt.scores_ragged(q, w, keys, i32([300]), i32([0])).clone()
    keys[7] = float("nan")
    keys[201] = float("inf")
    got = dt.scores_ragged(q, w, keys, i32([300]), i32([0]))
    rest = torch.ones(300, dtype=torch.bool, device=DEV)
    rest[7] = rest[201] = False
    assert torch.equal(got[0, :300][rest], ref[0, :300][rest])


def test_scores_empty_batches():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(6)
    q, w, keys, _ = make(g, 0, 64, 128, (300,), "bf16")
    assert dt.scores_ragged(q, w, keys, i32([]), i32([])).shape[0] == 0
    q, w, keys, _ = make(g, 3, 64, 128, (4, 16), "bf16")
    out = torch.full((3, 64), 5.0, device=DEV)
    dt.scores_paged(q, w, keys, i32([0, 0, -1]), i32(np.zeros((3, 4))), out=out)
    torch.cuda.synchronize()
    assert (out == 5).all()


def test_scores_feed_the_top_k():
    """The selection over the kernel's scores is the selection over them."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(7)
    q, w, keys, _ = make(g, 4, 64, 128, (4 * 16, 64), "bf16")
    table = torch.randperm(64, generator=g, device=DEV).view(4, 16).to(torch.int32)
    lens = i32([1024, 700, 130, 64])
    out = dt.scores_paged(q, w, keys, lens, table)
    slots = dt.paged(out, lens, table, 64, 128)
    torch.cuda.synchronize()
    for b, n in enumerate(lens.tolist()):
        order = torch.sort(out[b, :n], descending=True, stable=True).indices[:128].cpu()
        pages = table[b].cpu().long()[order // 64] * 64 + order % 64
        got = slots[b].cpu()
        assert sorted(got[got >= 0].tolist()) == sorted(pages.tolist())
