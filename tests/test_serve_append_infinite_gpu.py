"""Cache writes: elements that are not turned are what they were beside infinite
ones and NaN, and a turned one depends on its own pair only."""
import math

import numpy as np
import pytest
import torch

from tests import append_plain as plain
from tests.test_serve_append_gpu import TYPES, bits, i32, rand

pytestmark = pytest.mark.gpu

BAD = [math.inf, -math.inf, math.nan]


def some_bad(g, kind, *shape):
    """Random numbers, one in eight of them infinite or NaN."""
    x = rand(g, kind, *shape)
    pick = torch.randint(0, 24, shape, generator=g, device="cuda")
    for i, v in enumerate(BAD):
        x[pick == i] = v
    return x


def turned(x, row_lens, positions, cos_sin, near):
    """(expected [tokens, ..., 64] by IEEE rules in 32 bits, whether an element of the pair is not finite)."""
    x = x.float().cpu()
    want, odd = x.clone(), torch.zeros(x.shape, dtype=torch.bool)
    for t, n in enumerate(row_lens):
        if not 0 < n <= positions:
            continue
        a, b = (slice(0, 64, 2), slice(1, 64, 2)) if near else (slice(0, 32), slice(32, 64))
        cos, sin = cos_sin[n - 1, :32].cpu(), cos_sin[n - 1, 32:].cpu()
        p, q = x[t, ..., a], x[t, ..., b]
        want[t, ..., a], want[t, ..., b] = p * cos - q * sin, p * sin + q * cos
        odd[t, ..., a] = odd[t, ..., b] = ~(torch.isfinite(p) & torch.isfinite(q))
    return want, odd


def same(got, want, odd, before):
    """Not finite where a pair is not, finite where it is, and bit for bit what they were where nothing turns."""
    got = got.float().cpu()
    real = torch.isfinite(want) & ~odd
    # two products and a sum in fp32, one rounding
    half = 2.0 ** -8
    assert torch.isfinite(got[real]).all() and ((got - want)[real].abs() <= half * want[real].abs() + 2.0 ** -18).all()
    assert (~torch.isfinite(got[odd])).all()
    still = ~torch.isfinite(want) & ~odd
    assert torch.equal(torch.isnan(got[still]), torch.isnan(before[still]))
    whole = still & ~torch.isnan(before)
    assert torch.equal(got[whole], before[whole])


@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_index(kind, dim, near):
    import row_top_selection_amd as dt

    g = torch.Generator("cuda").manual_seed(dim)
    tokens, heads, positions = 40, 5, 30
    lens = np.arange(tokens) - 2  # no position before the third, nor from the 33rd on
    cos_sin = plain.angles(positions).cuda()
    cos_sin[:, 32:].clamp_(min=2.0 ** -10)  # (a sine of 0 would make NaN of an infinite partner by the formula)
    x, q = some_bad(g, kind, tokens, dim), some_bad(g, kind, tokens, heads, dim)
    keys = torch.zeros(3, 16, dim, device="cuda").to(TYPES[kind])
    slots = np.arange(tokens)
    q_out, _ = dt.append_index(x, keys, i32(slots), i32(lens), cos_sin, q=q, interleaved=near)
    torch.cuda.synchronize()
    cached = (lens > 0) & (lens <= positions)
    stored = keys.view(-1, dim)[torch.as_tensor(slots[cached], device="cuda")]
    mine = x[torch.as_tensor(cached, device="cuda")]
    # behind the rotary part, and without a position, nothing changes
    assert torch.equal(bits(stored[:, 64:]), bits(mine[:, 64:])) and torch.equal(bits(q_out[..., 64:]), bits(q[..., 64:]))
    none = torch.as_tensor(~cached, device="cuda")
    assert torch.equal(bits(q_out[none]), bits(q[none]))
    want, odd = turned(mine[:, :64], lens[cached], positions, cos_sin, near)
    same(stored[:, :64], want, odd, mine[:, :64].float().cpu())
    want, odd = turned(q[..., :64], lens, positions, cos_sin, near)
    same(q_out[..., :64], want, odd, q[..., :64].float().cpu())


@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("latent", [256, 512])
def test_latent(kind, latent, near):
    import row_top_selection_amd as dt

    g = torch.Generator("cuda").manual_seed(latent)
    tokens, heads, positions = 40, 5, 30
    lens = np.arange(tokens) - 2
    cos_sin = plain.angles(positions).cuda()
    cos_sin[:, 32:].clamp_(min=2.0 ** -10)
    x, q = some_bad(g, kind, tokens, latent + 64), some_bad(g, kind, tokens, heads, 64)
    cache, out = torch.zeros(3, 16, latent + 64, device="cuda").to(TYPES[kind]), torch.empty_like(x)
    q_out = dt.append_latent(x, cache, i32(np.arange(tokens)), i32(lens), cos_sin, q_rope=q, out=out, interleaved=near)
    torch.cuda.synchronize()
    assert torch.equal(bits(out[:, :latent]), bits(x[:, :latent]))
    none = torch.as_tensor((lens <= 0) | (lens > positions), device="cuda")
    assert torch.equal(bits(out[none]), bits(x[none])) and torch.equal(bits(q_out[none]), bits(q[none]))
    for got, was in ((out[:, latent:], x[:, latent:]), (q_out, q)):
        want, odd = turned(was, lens, positions, cos_sin, near)
        same(got, want, odd, was.float().cpu())
