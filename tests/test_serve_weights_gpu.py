"""Softmax weights of both attention forms far below the largest one, against
the definition in 64 bits (tests/serve_plain.py).

In half precision a weight is held to 2^-11 of itself or, where that is more,
to 2^-35 of its row's largest weight: many small weights beside a large one
whose value is small still make the output that they should."""
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


def close(got, want, logit_size, dim, tokens, value):
    """out and lse of rows whose logits are at most `logit_size` and values at
    most `value`.

    off: a logit's error, `dim` fp32 additions and three roundings of its size,
    beside exp2's and log2's own 2^-20; it shifts a weight and the weights' sum
    by e^off each. A weight is rounded to half a step of the type, in half
    precision at least to 2^-35 of the largest weight (1, at most, of the sum);
    the output to half a step, below the normal range to half of its
    smallest. Sums over tokens in fp32: 2^-16 of the values' sizes."""
    out, lse = got[0].cpu().double(), got[1].cpu().double()
    want_out, want_lse, size = want
    off = (dim + 4) * 2.0 ** -24 * logit_size + 2.0 ** -20
    info = torch.finfo(got[0].dtype)
    half = info.eps / 2
    lost = tokens * 2.0 ** -35 * value if got[0].dtype == torch.float16 else 0.0
    bound = size * (math.expm1(2 * off) + half * (1 + half) + 2.0 ** -16) + lost + want_out.abs() * half
    bound = bound + info.smallest_normal * half
    assert torch.isfinite(out).all()
    assert ((out - want_out).abs() <= bound).all(), ((out - want_out).abs() / bound).max()
    assert ((lse - want_lse).abs() <= off + 2.0 ** -20 * (1 + want_lse.abs())).all()


# Logits of a row's tokens, by the number of them, and the tokens whose values are 0.
def tail(n, by):
    """One token `by` above all others, in the middle; its value is 0."""
    logits = np.zeros(n)
    logits[n // 2] = by
    return logits, [n // 2]


def spread(n, by):
    """Logits evenly over 0 .. by, the largest first; the upper half has no value."""
    logits = np.linspace(by, 0.0, n)
    return logits, np.arange(n // 2)


def growing(n, by):
    """The same, the largest last."""
    return np.linspace(0.0, by, n), np.arange(n - n // 2, n)


CASES = [(tail, 9.0), (tail, 15.0), (tail, 17.0), (tail, 18.5), (tail, 21.0), (spread, 20.0), (growing, 20.0),
         (growing, 300.0), (spread, 0.0), (growing, 3.0)]


def values_and_logits(g, kind, n, case, width):
    """(values [n, width], the logits as the type holds them)."""
    logits, none = case[0](n, case[1])
    v = torch.randn(n, width, generator=g, device=DEV).abs() + 0.5  # of one sign: nothing cancels
    v[torch.as_tensor(none, device=DEV, dtype=torch.long)] = 0.0
    return v.to(TYPES[kind]), torch.as_tensor(logits, device=DEV).to(TYPES[kind])


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0].__name__}{c[1]:g}")
@pytest.mark.parametrize("rows,heads,latent", [(1, 16, 512), (2, 3, 256), (3, 30, 512), (2, 50, 512), (2, 128, 256),
                                               (600, 16, 256)])
def test_selected_small_weights(rows, heads, latent, case):
    import row_top_selection_amd as dt

    n = 4000 if rows < 600 else 400
    for kind in ("fp16", "bf16"):
        g = torch.Generator(DEV).manual_seed(n + heads)
        v, logits = values_and_logits(g, kind, n, case, latent)
        cache = torch.zeros(1, 4096, latent + 64, dtype=TYPES[kind], device=DEV)
        cache[0, :n, :latent], cache[0, :n, latent + 5] = v, logits
        q = torch.zeros(rows, heads, latent + 64, dtype=TYPES[kind], device=DEV)
        q[..., latent + 5] = 1.0
        slots = i32(np.tile(np.arange(n), (rows, 1)))
        got = dt.attend_selected(q, cache, slots, latent, 1.0)
        want = serve_plain.attend(q[:1, :1], cache[0], latent, 1.0, [np.arange(n)])
        close(got, want, case[1], latent + 64, n, float(v.max()))


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0].__name__}{c[1]:g}")
@pytest.mark.parametrize("queries,heads,keys", [(1, 1, 9000), (150, 2, 700), (33, 2, 2100), (520, 64, 520)])
def test_expanded_small_weights(queries, heads, keys, case):
    """Few queries of many keys (split), narrow workgroups, and wide ones."""
    import row_top_selection_amd as dt

    for kind in ("fp16", "bf16"):
        g = torch.Generator(DEV).manual_seed(keys + queries)
        v, logits = values_and_logits(g, kind, keys, case, 128)
        value = v[:, None].expand(keys, heads, 128).contiguous()
        k = torch.zeros(keys, heads, 128, dtype=TYPES[kind], device=DEV)
        rope = torch.zeros(keys, 64, dtype=TYPES[kind], device=DEV)
        rope[:, 9] = logits
        q = torch.zeros(queries, heads, 192, dtype=TYPES[kind], device=DEV)
        q[..., 128 + 9] = 1.0
        got = dt.attend_expanded(q, k, value, rope, i32([0, queries]), i32([0, keys]), queries, 1.0, causal=False)
        want = serve_plain.expand(q[:1, :1], k[:, :1], value[:, :1], rope, [0, 1], [0, keys], 1.0, False)
        close(got, want, case[1], 192, keys, float(v.max()))
