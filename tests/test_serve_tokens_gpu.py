"""Every token of a row is attended to, once.

Counting: with queries of zeros all weights are the same, a power of two, and
a value of 1 in one element of each token's vector makes output element c the
share of the row's tokens whose vector has it there. Sums of such weights are
exact in fp32, so that only the division (2^-22), the rounding of the output
and the logarithm are left: one token left out, or read twice, exceeds the
tolerance in rows of 20000.

Weighing: queries with DIMS elements other than 0, so that a logit is a sum
of DIMS products and off by (DIMS + 4) * 2^-24 of its size at most, taken by
row and head: a tile left out exceeds the tolerance in rows of 9000, as do
single tokens of more than some 1e-4 of the weights.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DIMS = 8


def i32(v):
    return torch.as_tensor(np.asarray(v, dtype=np.int32)).to(DEV)


def check_counts(out, lse, counts):
    """counts float64 [rows, elements]: tokens of each row by the element that is 1; all heads alike."""
    n = counts.sum(1, keepdim=True)
    want = torch.where(n > 0, counts / n.clamp(min=1), 0.0)[:, None]
    bound = want * (torch.finfo(out.dtype).eps / 2 + 2.0 ** -21) + torch.finfo(out.dtype).smallest_normal * torch.finfo(out.dtype).eps / 2
    assert ((out.double() - want).abs() <= bound).all(), ((out.double() - want).abs() / bound.clamp(min=1e-30)).max()
    total = torch.log(n).expand(lse.shape)
    seen = torch.isfinite(total)
    assert (lse[~seen] == -math.inf).all()
    assert ((lse.double() - total)[seen].abs() <= 2.0 ** -21 * (1 + total[seen].abs())).all()


def check_weights(out, lse, logits, size, values, dtype):
    """One row's head: logits float64 [n], size: the largest sum of its products' sizes, values float64 [n, dim]."""
    n = logits.numel()
    want_lse = torch.logsumexp(logits, 0)
    w = torch.exp(logits - want_lse)
    want, mean = w @ values, w @ values.abs()
    info = torch.finfo(dtype)
    half = info.eps / 2
    off = (DIMS + 4) * 2.0 ** -24 * size + 2.0 ** -21  # exp2 and log2: a few steps each
    sums = (n / 16 + 64) * 2.0 ** -24                  # additions behind each other, of a lane and of parts
    lost = n * 2.0 ** -35 * float(values.abs().max()) if dtype == torch.float16 else 0.0
    bound = mean * (math.expm1(2 * off) + half * (1 + half) + 2 * sums) + want.abs() * half + lost + info.smallest_normal * half
    assert ((out.double() - want).abs() <= bound).all(), ((out.double() - want).abs() / bound).max()
    assert abs(float(lse.double() - want_lse)) <= off + sums + 2.0 ** -21 * (1 + abs(float(want_lse)))


def coded(tokens, width, kind, g):
    """[tokens, width + 64]: token t has a 1 at t % width, and anything in the rotary part."""
    x = torch.zeros(tokens, width + 64, device=DEV)
    t = torch.arange(tokens, device=DEV)
    x[t, t % width] = 1.0
    x[:, width:] = torch.randn(tokens, 64, generator=g, device=DEV)
    return x.to(TYPES[kind])


def counts_of(picked, width):
    return torch.stack([torch.bincount(p % width, minlength=width) for p in picked]).double()


HEADS = [(1, 256), (16, 512), (24, 256), (32, 512), (40, 512), (64, 256), (70, 512), (128, 512), (200, 256)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,latent", HEADS)
@pytest.mark.parametrize("lens", [[20000, 3, 9001], [12000, 0], [9999], [33, 64, 65, 31, 32, 1, 127, 128, 129], [700] * 5 + [701] * 4,
                                  list(range(2030, 2100))])
def test_paged_counts(kind, heads, latent, lens):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads + len(lens))
    page, pages = 16, 300
    cache = coded(pages * page, latent, kind, g).view(pages, page, latent + 64)
    width = -(-max(lens) // page)
    table = torch.randint(0, pages, (len(lens), width), generator=g, device=DEV).to(torch.int32)
    q = torch.zeros(len(lens), heads, latent + 64, dtype=TYPES[kind], device=DEV)
    at = [(table[b].long()[:, None] * page + torch.arange(page, device=DEV)).flatten()[:n] for b, n in enumerate(lens)]
    counts = counts_of(at, latent)
    for bound in (None, 100, max(lens)):
        check_counts(*dt.attend_paged(q, cache, i32(lens), table, latent, 0.1, max_seq_len=bound), counts)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,latent", HEADS)
@pytest.mark.parametrize("rows,k", [(1, 2048), (2, 2047), (3, 33), (9, 130), (70, 513), (300, 190)])
def test_selected_counts(kind, heads, latent, rows, k):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(rows + k)
    rng = np.random.default_rng(rows + k + heads)
    cache = coded(4096, latent, kind, g).view(64, 64, latent + 64)
    slots = rng.integers(0, 4096, (rows, k))
    if rows > 2:  # holes anywhere, nothing from somewhere on, and nothing at all
        slots[1::3][rng.random(slots[1::3].shape) < 0.3] = -1
        slots[2::3][np.arange(k) >= rng.integers(0, k, len(slots[2::3]))[:, None]] = -1
        slots[2, 1:], slots[-1] = 4096, -1
    q = torch.zeros(rows, heads, latent + 64, dtype=TYPES[kind], device=DEV)
    at = [torch.as_tensor(s[(s >= 0) & (s < 4096)]).to(DEV) for s in slots]
    check_counts(*dt.attend_selected(q, cache, i32(slots), latent, 0.1), counts_of(at, latent))


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,latent", HEADS)
@pytest.mark.parametrize("lens", [[9000, 5], [4001, 100, 2, 3000], [515] * 70])
def test_paged_weights(kind, heads, latent, lens):
    """Logits between about -5 and 5."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads + len(lens))
    page, pages, dim = 16, 300, latent + 64
    cache = torch.randn(pages, page, dim, generator=g, device=DEV).to(TYPES[kind])
    table = torch.randint(0, pages, (len(lens), -(-max(lens) // page)), generator=g, device=DEV).to(torch.int32)
    q = torch.zeros(len(lens), heads, dim, device=DEV)
    for b in range(len(lens)):  # other elements for each row, of the rotary part too
        which = torch.randperm(dim, generator=g, device=DEV)[:DIMS]
        which[0] = latent + b % 64
        q[b, :, which] = torch.randn(heads, DIMS, generator=g, device=DEV)
    q = q.to(TYPES[kind])
    out, lse = dt.attend_paged(q, cache, i32(lens), table, latent, 0.6)
    for b in sorted({0, 1, len(lens) - 1}):
        at = (table[b].long()[:, None] * page + torch.arange(page, device=DEV)).flatten()[:lens[b]]
        x = cache.view(-1, dim)[at].double()
        for h in sorted({0, heads // 2, heads - 1}):
            logits = x @ q[b, h].double() * 0.6
            size = float((x.abs() @ q[b, h].double().abs()).max() * 0.6)
            check_weights(out[b, h], lse[b, h], logits, size, x[:, :latent], TYPES[kind])


EXPANDED = [  # queries and keys of each request, heads
    ([1], [1], 1), ([1, 1, 1], [1, 64, 65], 3), ([128, 129, 31], [128, 129, 31], 2), ([5, 0, 70], [200, 9, 70], 1),
    ([2, 130, 1], [3000, 2050, 1], 1), ([40, 0, 7], [5000, 10, 600], 2), ([1], [20000], 1), ([164, 100], [4906, 4001], 1),
    ([515, 300, 1, 600, 512], [517, 333, 65, 631, 512], 64), ([1024, 1000], [9000, 8191], 32),
    ([10, 40, 3, 140], [4, 0, 3, 70], 2), ([777, 400, 31], [777, 400, 31], 16),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,k_lens,heads", EXPANDED)
def test_expanded_counts(kind, causal, q_lens, k_lens, heads):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(sum(q_lens))
    qs, ks = np.concatenate([[0], np.cumsum(q_lens)]), np.concatenate([[0], np.cumsum(k_lens)])
    q = torch.zeros(qs[-1], heads, 192, dtype=TYPES[kind], device=DEV)
    k = torch.randn(ks[-1], heads, 128, generator=g, device=DEV).to(TYPES[kind])
    rope = torch.randn(ks[-1], 64, generator=g, device=DEV).to(TYPES[kind])
    v = torch.zeros(ks[-1], heads, 128, dtype=TYPES[kind], device=DEV)
    j = torch.arange(ks[-1], device=DEV)
    v[j, :, j % 128] = 1.0
    out, lse = dt.attend_expanded(q, k, v, rope, i32(qs), i32(ks), max(q_lens), 0.1, causal=causal)
    ends, firsts = [], []
    for m, n, first in zip(q_lens, k_lens, ks):
        ends += [min(n, max(0, n - m + i + 1)) if causal else n for i in range(m)]
        firsts += [int(first)] * m
    first, end = (torch.as_tensor(x, device=DEV)[:, None] for x in (firsts, ends))
    c = torch.arange(128, device=DEV)
    # keys j < x with j % 128 == c, for the row's last key and its first
    counts = ((first + end - c + 127) // 128 - (first - c + 127) // 128).double()
    check_counts(out, lse, counts)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("q_lens,k_lens,heads", EXPANDED[:-2] + EXPANDED[-1:])
def test_expanded_weights(kind, q_lens, k_lens, heads):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(sum(q_lens) + 1)
    qs, ks = np.concatenate([[0], np.cumsum(q_lens)]), np.concatenate([[0], np.cumsum(k_lens)])
    q = torch.zeros(qs[-1], heads, 192, device=DEV)
    for h in range(heads):
        which = torch.randperm(192, generator=g, device=DEV)[:DIMS]
        which[0] = 128 + h % 64
        q[:, h, which] = torch.randn(int(qs[-1]), DIMS, generator=g, device=DEV)
    q = q.to(TYPES[kind])
    k, v = (torch.randn(ks[-1], heads, 128, generator=g, device=DEV).to(TYPES[kind]) for _ in range(2))
    rope = torch.randn(ks[-1], 64, generator=g, device=DEV).to(TYPES[kind])
    out, lse = dt.attend_expanded(q, k, v, rope, i32(qs), i32(ks), max(q_lens), 0.6)
    for r, (m, n) in enumerate(zip(q_lens, k_lens)):
        for h in sorted({0, heads // 2, heads - 1}):
            keys = torch.cat([k[ks[r]:ks[r + 1], h], rope[ks[r]:ks[r + 1]]], dim=1).double()
            for i in sorted({0, m // 2, m - 2, m - 1} & set(range(m))):
                end = n - m + i + 1
                if end < 1:
                    continue
                query = q[qs[r] + i, h].double()
                size = float((keys[:end].abs() @ query.abs()).max() * 0.6)
                check_weights(out[qs[r] + i, h], lse[qs[r] + i, h], keys[:end] @ query * 0.6, size,
                              v[ks[r]:ks[r] + end, h].double(), TYPES[kind])


def test_tables_much_wider_than_the_rows():
    """A table of the longest context, as a captured step has it: what it
    holds behind the rows' ends is not read as tokens."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(8)
    page, pages, width, latent = 64, 70, 2048, 512
    lens = [4000, 1, 0, 64, 65, 777, 131072 // 2, 4100]
    cache = coded(pages * page, latent, "bf16", g).view(pages, page, latent + 64)
    table = torch.randint(-5, 2 * pages, (len(lens), width), generator=g, device=DEV).to(torch.int32)
    for b, n in enumerate(lens):
        table[b, :-(-n // page)] %= pages
    at = [(table[b].long()[:, None] * page + torch.arange(page, device=DEV)).flatten()[:n] for b, n in enumerate(lens)]
    q = torch.zeros(len(lens), 16, latent + 64, dtype=torch.bfloat16, device=DEV)
    for bound in (None, max(lens)):
        check_counts(*dt.attend_paged(q, cache, i32(lens), table, latent, 0.1, max_seq_len=bound),
                     counts_of([p.clamp(0, pages * page - 1) for p in at], latent))
    # scores: the same bits as over a table that ends with the row, and nothing behind
    qi = torch.randn(len(lens), 64, 128, generator=g, device=DEV).to(torch.bfloat16)
    w, keys = torch.randn(len(lens), 64, generator=g, device=DEV), torch.randn(pages, page, 128, generator=g, device=DEV)
    keys = keys.to(torch.bfloat16)
    wide = dt.scores_paged(qi, w, keys, i32(lens), table, out=torch.full((len(lens), width * page), -7.0, device=DEV))
    for b, n in enumerate(lens):
        cols = max(1, -(-n // page))
        one = dt.scores_paged(qi[b:b + 1], w[b:b + 1], keys, i32([n]), table[b:b + 1, :cols].contiguous(),
                              out=torch.full((1, cols * page), -7.0, device=DEV))
        assert torch.equal(wide[b, :n], one[0, :n])
        assert (wide[b, n:] == -7).all()
