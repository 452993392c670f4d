"""The cache writes' definitions in 64 bits on the CPU (test helper; shares no
code with the library), with what fp32 may be off by."""
from __future__ import annotations

import torch

ROPE = 64


def angles(positions, base=10000.0):
    """float32 [positions, 64]: cosines, sines."""
    at = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-torch.arange(32, dtype=torch.float64) / 32)
    return torch.cat([at.cos(), at.sin()], 1).float()


def turn(x, size, row_lens, cos_sin, interleaved):
    """(turned, size of its terms) of x [tokens, ..., 64], `size` that of its elements."""
    x, size, table = x.clone(), size.clone(), cos_sin.double().cpu()
    for t, n in enumerate(row_lens):
        if not 0 < n <= table.shape[0]:
            continue
        for i in range(32):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
            cos, sin = table[n - 1, i], table[n - 1, 32 + i]
            p, q, u, v = (y[t, ..., j].clone() for y in (x, size) for j in (a, b))
            x[t, ..., a], x[t, ..., b] = p * cos - q * sin, p * sin + q * cos
            size[t, ..., a], size[t, ..., b] = u * cos.abs() + v * sin.abs(), u * sin.abs() + v * cos.abs()
    return x, size


def latent(x, weight, eps, row_lens, cos_sin, interleaved, latent_dim):
    """(vectors, what they may be off by in fp32).

    The sum of squares is 8 terms a lane and 6 sums over lanes, off by 14 half
    steps (2^-24 each) of itself; the mean, eps, the root, its inverse and two
    products are one each, a root halves what was off before: under 2^-19. A
    turned element is two products and a sum, under 2^-22 of its terms' size."""
    x = x.double().cpu()
    body = x[:, :latent_dim]
    off = torch.zeros_like(x)
    if weight is not None:
        body = body / ((body ** 2).mean(1, keepdim=True) + eps).sqrt() * weight.double().cpu()
        off[:, :latent_dim] = body.abs() * 2.0 ** -19
    rope, size = turn(x[:, latent_dim:], x[:, latent_dim:].abs(), row_lens, cos_sin, interleaved)
    off[:, latent_dim:] = size * 2.0 ** -22
    return torch.cat([body, rope], 1), off


def index(x, weight, bias, eps, row_lens, cos_sin, interleaved):
    """(vectors, what they may be off by) of keys or queries [..., dim], before any rounding.

    The mean is off by under 16 half steps of the mean size m, and so is every
    difference from it; that moves the deviation by as much, which a difference
    is divided by: (|x| + m) * (1 + m / deviation) * 2^-18 covers both and the
    products behind them."""
    x = x.double().cpu()
    off = torch.zeros_like(x)
    if weight is not None:
        mean, m = x.mean(-1, keepdim=True), x.abs().mean(-1, keepdim=True)
        by = 1 / ((x - mean).pow(2).mean(-1, keepdim=True) + eps).sqrt()
        w, b = weight.double().cpu(), bias.double().cpu()
        off = ((x.abs() + m) * by * w.abs() * (1 + m * by) + b.abs()) * 2.0 ** -18
        x = (x - mean) * by * w + b
    rope, size = turn(x[..., :ROPE], x[..., :ROPE].abs(), row_lens, cos_sin, interleaved)
    _, moved = turn(x[..., :ROPE], off[..., :ROPE], row_lens, cos_sin, interleaved)
    return torch.cat([rope, x[..., ROPE:]], -1), torch.cat([moved + size * 2.0 ** -22, off[..., ROPE:]], -1)


def close(got, want, off, what=""):
    """got, in its own type, rounded once from a number within `off` of want."""
    half = torch.finfo(got.dtype).eps / 2
    bound = (want.abs() + off) * half + off + torch.finfo(got.dtype).smallest_normal * half
    far = (got.double().cpu() - want).abs()
    assert (far <= bound).all(), (what, float((far / bound).max()))


def close8(got, scale, want, off, what=""):
    """e4m3 numbers and their scales [...] against vectors: the scale is the largest element / 448, a
    number is off by half a step (2^-4 of itself, half of the smallest number 2^-9 below the normal ones)."""
    most = want.abs().amax(-1).clamp(min=2.0 ** -100)
    loose = (off.amax(-1) + most * 2.0 ** -22)
    scale = scale.double().cpu()
    assert ((scale * 448 - most).abs() <= loose).all(), what
    got = got.float().double().cpu() * scale[..., None]
    # y / s carries the scale's and the inverse's own two roundings
    bound = want.abs() * (2.0 ** -4 + 2.0 ** -21) + scale[..., None] * 2.0 ** -10 + off * (1 + 2.0 ** -3)
    far = (got - want).abs()
    assert (far <= bound).all(), (what, float((far / bound.clamp(min=1e-300)).max()))
