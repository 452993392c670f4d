"""The serving operators' definitions, in plain loops and 64 bits on the CPU
(test helper; shares no code with the library)."""
from __future__ import annotations

import numpy as np
import torch


def page_maps(seq_lens, new_lens, table, page_size, free, num_tokens):
    """(table, token_starts, slots, table_rows, row_lens, counts) as lists and arrays."""
    table = np.array(table, dtype=np.int64)
    starts, slots, rows, lens = [0], [], [], []
    tokens = pages = 0
    for r, length in enumerate(seq_lens):
        length = max(int(length), 0)
        new = min(1, length) if new_lens is None else min(max(int(new_lens[r]), 0), length)
        held = -(-(length - new) // page_size)
        opened = {}
        for e in range(held, -(-length // page_size)):
            opened[e] = int(free[pages]) if pages < len(free) else -1
            pages += 1
        for pos in range(length - new, length):
            if tokens < num_tokens:
                e = pos // page_size
                page = -1
                if e < table.shape[1]:
                    if e in opened:
                        page = opened[e]
                        if pos % page_size == 0:
                            table[r, e] = page
                    else:
                        page = int(table[r, e])
                slot = page * page_size + pos % page_size
                slots.append(-1 if page < 0 or slot >= 2 ** 31 else slot)
                rows.append(r)
                lens.append(pos + 1)
            tokens += 1
        starts.append(tokens)
    pad = num_tokens - len(slots)
    return dict(table=table, token_starts=starts, slots=slots + [-1] * pad,
                table_rows=rows + [0] * pad, row_lens=lens + [0] * pad, counts=[tokens, pages])


def scores(q, weights, keys, scales, windows, out):
    """windows[b] = (first column, key row of each column of the window, -1: no
    key). Returns (64-bit scores in out's shape, bound on the sums' sizes)."""
    want = out.double().cpu().clone()
    size = torch.zeros_like(want)
    q, weights, keys = q.cpu().double(), weights.cpu().double(), keys.cpu().double()
    for b, (first, at) in enumerate(windows):
        at = torch.as_tensor(at, dtype=torch.int64)
        if not at.numel():
            continue
        k = keys[at.clamp(min=0)] * (at >= 0)[:, None]
        s = torch.ones(at.numel(), dtype=torch.float64) if scales is None else scales.cpu().double()[at.clamp(min=0)]
        dots = q[b] @ k.T
        want[b, first:first + at.numel()] = (weights[b][:, None] * dots.clamp(min=0)).sum(0) * s
        # what fp32 rounding is relative to: every product and partial sum by its size
        size[b, first:first + at.numel()] = (weights[b].abs()[:, None] * (q[b].abs() @ k.abs().T)).sum(0) * s.abs()
    return want, size


def attend(q, vectors, latent, scale, picked):
    """Absorbed latent attention: picked[b] = rows of vectors that query row b
    reads. Returns 64-bit (out, lse, mean size of the values by weight)."""
    q, vectors = q.cpu().double(), vectors.cpu().double()
    rows, heads, _ = q.shape
    out = torch.zeros(rows, heads, latent, dtype=torch.float64)
    size = torch.zeros_like(out)
    lse = torch.full((rows, heads), -float("inf"), dtype=torch.float64)
    for b, at in enumerate(picked):
        at = torch.as_tensor(at, dtype=torch.int64)
        if not at.numel():
            continue
        x = vectors[at]
        logits = (q[b] @ x.T) * scale
        lse[b] = torch.logsumexp(logits, -1)
        w = torch.exp(logits - lse[b][:, None])
        out[b] = w @ x[:, :latent]
        size[b] = w @ x[:, :latent].abs()
    return out, lse, size


def expand(q, k, v, k_rope, q_starts, k_starts, scale, causal=True):
    """Expanded latent attention in 64 bits: (out, lse, size of the values by weight)."""
    q, k, v, k_rope = (t.cpu().double() for t in (q, k, v, k_rope))
    tokens, heads, _ = q.shape
    out = torch.zeros(tokens, heads, v.shape[-1], dtype=torch.float64)
    size = torch.zeros_like(out)
    lse = torch.full((tokens, heads), -float("inf"), dtype=torch.float64)
    for r in range(len(q_starts) - 1):
        a, b, c, d = q_starts[r], q_starts[r + 1], k_starts[r], k_starts[r + 1]
        for i in range(a, b):
            end = c + min(d - c, max(0, (i - a) + (d - c) - (b - a) + 1)) if causal else d
            if end <= c:
                continue
            for h in range(heads):
                key = torch.cat([k[c:end, h], k_rope[c:end]], dim=1)
                logits = key @ q[i, h] * scale
                lse[i, h] = torch.logsumexp(logits, -1)
                w = torch.exp(logits - lse[i, h])
                out[i, h] = w @ v[c:end, h]
                size[i, h] = w @ v[c:end, h].abs()
    return out, lse, size
