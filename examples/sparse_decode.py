"""One layer of sparse latent attention, from prompts to tokens.

A batch of prompts is read with the expanded form; their latent vectors and
indexer keys are left in paged caches. Then tokens are decoded, each step
captured once in a HIP graph and replayed:

    page_maps        pages and slots of the step's tokens, the top-k's row arguments
    append_latent    the new tokens' latent vectors, normalised and turned, into their
                     slots, and the queries' rotary parts
    append_index     the same for the indexer's keys and queries
    scores_paged     the indexer's scores of every cached token
    plan, paged      the top-k, as cache slots
    attend_selected  attention over the selected slots

Weights and inputs are random: the example shows how the calls fit together.

    python examples/sparse_decode.py [--requests 8] [--prompt 700] [--steps 8]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import row_top_selection_amd as dt  # noqa: E402

LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128
INDEX_HEADS, INDEX_DIM = 64, 128
PAGE = 64


class Layer:
    """Random projections of a hidden state, and the caches."""

    def __init__(self, hidden, heads, pages, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-2] ** -0.5).bfloat16()

        self.heads = heads
        self.to_q = weight(hidden, heads * (NOPE + ROPE))
        self.to_latent = weight(hidden, LATENT + ROPE)
        self.up_k = weight(heads, NOPE, LATENT) * (NOPE / LATENT) ** 0.5
        self.up_v = weight(heads, LATENT, VALUE)
        self.to_index_q = weight(hidden, INDEX_HEADS * INDEX_DIM)
        self.to_index_k = weight(hidden, INDEX_DIM)
        self.to_index_w = weight(hidden, INDEX_HEADS)
        self.scale = (NOPE + ROPE) ** -0.5
        self.norm = 1 + 0.1 * torch.randn(LATENT, generator=g, device=device)
        self.index_norm = 1 + 0.1 * torch.randn(INDEX_DIM, generator=g, device=device)
        self.index_bias = 0.1 * torch.randn(INDEX_DIM, generator=g, device=device)
        angles = torch.arange(pages * PAGE, device=device)[:, None] * 10000.0 ** (-torch.arange(32, device=device) / 32)
        self.angles = torch.cat([angles.cos(), angles.sin()], dim=1)
        bf = dict(dtype=torch.bfloat16, device=device)
        self.cache = torch.zeros(pages, PAGE, LATENT + ROPE, **bf)
        self.index_keys = torch.zeros(pages, PAGE, INDEX_DIM, **bf)

    def write(self, x, maps, q_rope, q_out, index_q=None):
        """The tokens' latent vectors and indexer keys go to their slots, and the queries' rotary parts to q_out:
        the vectors, and the indexer's queries."""
        latent = x @ self.to_latent
        dt.append_latent(latent, self.cache, maps.slots, maps.row_lens, self.angles, weight=self.norm, q_rope=q_rope,
                         q_out=q_out, out=latent)
        index = dt.append_index(x @ self.to_index_k, self.index_keys, maps.slots, maps.row_lens, self.angles,
                                weight=self.index_norm, bias=self.index_bias, q=index_q)
        return latent, index and index[0]

    def prompt(self, x, starts, longest, maps):
        """Causal attention of whole prompts, expanded: [tokens, heads, VALUE]."""
        tokens = x.shape[0]
        q = (x @ self.to_q).view(tokens, self.heads, NOPE + ROPE)
        latent, _ = self.write(x, maps, q[..., NOPE:], q[..., NOPE:])
        up = torch.cat([self.up_k, self.up_v.transpose(1, 2)], dim=1)  # [heads, NOPE + VALUE, LATENT]
        kv = (latent[:, :LATENT] @ up.reshape(-1, LATENT).t().contiguous()).view(tokens, self.heads, NOPE + VALUE)
        out, _ = dt.attend_expanded(q, kv[..., :NOPE], kv[..., NOPE:], latent[:, LATENT:], starts,
                                    starts, longest, self.scale)
        return out

    def step(self, x, lens, table, free, k, buffers):
        """One token for every request: [requests, heads, VALUE], and what was selected."""
        n = x.shape[0]
        maps = dt.page_maps(lens, table, PAGE, free, n)
        q = (x @ self.to_q).view(n, self.heads, NOPE + ROPE)
        absorbed = torch.empty(n, self.heads, LATENT + ROPE, dtype=x.dtype, device=x.device)
        _, index_q = self.write(x, maps, q[..., NOPE:], absorbed[..., LATENT:],
                                (x @ self.to_index_q).view(n, INDEX_HEADS, INDEX_DIM))
        scores = dt.scores_paged(index_q, (x @ self.to_index_w).float(), self.index_keys, maps.row_lens, table,
                                 table_rows=maps.table_rows, out=buffers["scores"])
        plan = dt.plan(maps.row_lens, k)
        slots = dt.paged(scores, maps.row_lens, table, PAGE, k, plan=plan, table_rows=maps.table_rows)
        # the keys' projection is absorbed into the queries, the values' into the output
        absorbed[..., :LATENT] = torch.bmm(q[..., :NOPE].transpose(0, 1).contiguous(), self.up_k).transpose(0, 1)
        out, _ = dt.attend_selected(absorbed, self.cache, slots, LATENT, self.scale)
        return torch.bmm(out.transpose(0, 1).contiguous(), self.up_v).transpose(0, 1), slots


def turned(layer, x, position):
    """x [..., ROPE] by the position's angles: element i and i + 32 are a pair."""
    cos, sin = layer.angles[position].split(32)
    a, b = x.split(32, dim=-1)
    return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)


def plain_step(layer, x, length, table_row, slots):
    """The step of one request from the definition, in fp32, over the given slots."""
    q = (x @ layer.to_q).view(layer.heads, NOPE + ROPE).float()
    q[:, NOPE:] = turned(layer, q[:, NOPE:], length - 1)
    # the new token's vector has been cached
    new = (x[None] @ layer.to_latent)[0].float()
    body = new[:LATENT] * (new[:LATENT].square().mean() + 1e-6).rsqrt() * layer.norm
    new = torch.cat([body, turned(layer, new[LATENT:], length - 1)])
    cached = layer.cache[table_row[(length - 1) // PAGE].long(), (length - 1) % PAGE].float()
    assert float((cached - new).abs().max() / new.abs().max()) < 0.02
    vectors = layer.cache.view(-1, LATENT + ROPE)[slots[slots >= 0].long()].float()
    keys = torch.einsum("tc,hdc->thd", vectors[:, :LATENT], layer.up_k.float())
    logits = torch.einsum("hd,thd->ht", q[:, :NOPE], keys) + q[:, NOPE:] @ vectors[:, LATENT:].t()
    weights = torch.softmax(logits * layer.scale, dim=-1)
    return torch.einsum("ht,tc,hcd->hd", weights, vectors[:, :LATENT], layer.up_v.float())


def main(requests=8, prompt=700, steps=8, k=256, heads=16, hidden=1024, check=True, say=print):
    device = "cuda"
    g = torch.Generator(device=device).manual_seed(1)
    most = prompt + steps
    width = -(-most // PAGE)
    layer = Layer(hidden, heads, requests * width)
    table = torch.full((requests, width), -1, dtype=torch.int32, device=device)
    free = torch.randperm(requests * width, generator=g, device=device).to(torch.int32)

    # prompts of uneven lengths
    prompt_lens = [max(1, prompt - 37 * r) for r in range(requests)]
    lens = torch.tensor(prompt_lens, dtype=torch.int32, device=device)
    tokens = sum(prompt_lens)
    x = torch.randn(tokens, hidden, generator=g, device=device).bfloat16()
    maps = dt.page_maps(lens, table, PAGE, free, tokens, new_lens=lens)
    layer.prompt(x, maps.token_starts, max(prompt_lens), maps)
    free = free[int(maps.counts[1]):].clone()

    # one decode step, captured; its inputs are static buffers
    x = torch.zeros(requests, hidden, dtype=torch.bfloat16, device=device)
    buffers = {"scores": torch.empty(requests, width * PAGE, device=device)}
    now = lens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # once outside the graph: libraries set themselves up
        layer.step(x, torch.zeros_like(lens), table, free, k, buffers)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, slots = layer.step(x, now, table, free, k, buffers)

    worst = 0.0
    for step in range(steps):
        x.copy_(torch.randn(requests, hidden, generator=g, device=device).bfloat16())
        opened = int(((now + PAGE) // PAGE - (now + PAGE - 1) // PAGE).sum())  # pages that this step opens
        now.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        free.copy_(torch.cat([free[opened:], free[:opened]]))
        if check:
            for r in range(requests):
                want = plain_step(layer, x[r], int(now[r]), table[r], slots[r])
                worst = max(worst, float((out[r].float() - want).abs().max() / want.abs().max()))
                assert int((slots[r] >= 0).sum()) == min(k, int(now[r]))
    say(f"{requests} requests, {steps} steps: last lengths {now.tolist()}, largest difference from the "
        f"definition {worst:.2e} of the largest output")
    assert math.isfinite(worst) and worst < 0.05
    return worst


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("requests", 8), ("prompt", 700), ("steps", 8), ("k", 256), ("heads", 16)):
        parser.add_argument("--" + name, type=int, default=value)
    main(**vars(parser.parse_args()))
