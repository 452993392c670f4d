"""A batch of requests behind common prompts, with all of the operators: the prompts and
what follows them are cached and read in their expanded form, then tokens are
decoded, selected and not, each against the definition over what is cached."""
import numpy as np
import pytest
import torch

from tests import append_plain, serve_plain
from tests.test_serve_attend_gpu import SCALE, close, i32, logit_size
from tests.test_serve_behind_gpu import definition

pytestmark = pytest.mark.gpu

DEV = "cuda"
LATENT, PAGE, HEADS = 512, 16, 16


def near(got, want, off):
    half = torch.finfo(got.dtype).eps / 2
    assert ((got.double().cpu() - want).abs() <= off + (want.abs() + off) * half).all()


def append(dt, g, cache, keys, maps, table_of_angles, norm):
    """New tokens, cached: (latent vectors, rotary parts of queries, indexer queries)."""
    n = maps.slots.numel()
    x = torch.randn(n, LATENT + 64, generator=g, device=DEV).bfloat16()
    q = torch.randn(n, HEADS, LATENT + 64, generator=g, device=DEV).bfloat16()
    turned = q.clone()
    lens = maps.row_lens.tolist()
    want, off = append_plain.latent(x, norm, 1e-6, lens, table_of_angles, False, LATENT)
    dt.append_latent(x, cache, maps.slots, maps.row_lens, table_of_angles, weight=norm, q_rope=q[..., LATENT:], q_out=turned[..., LATENT:], out=x)
    k, i = torch.randn(n, 128, generator=g, device=DEV).bfloat16(), torch.randn(n, 8, 128, generator=g, device=DEV).bfloat16()
    i, _ = dt.append_index(k, keys, maps.slots, maps.row_lens, table_of_angles, q=i)
    near(x, want, off)
    at = maps.slots.long()
    assert torch.equal(cache.view(-1, LATENT + 64)[at], x)
    return x, turned, i


def test_requests_behind_common_prompts():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(31)
    rng = np.random.default_rng(31)
    prompts, group = [96, 32, 160], np.array([0, 0, 0, 1, 2, 2, 2])   # whole pages, so that requests can share them
    rows, width, pages = len(group), 20, 200
    starts = [0, 3, 4, 7]
    cache = torch.zeros(pages, PAGE, LATENT + 64, device=DEV).bfloat16()
    keys = torch.zeros(pages, PAGE, 128, device=DEV).bfloat16()
    angles, norm = append_plain.angles(width * PAGE).to(DEV), torch.rand(LATENT, generator=g, device=DEV) + 0.5
    free = i32(rng.permutation(pages))

    # the prompts
    lens = i32(prompts)
    prompt_table = i32(np.full((3, width), -1))
    maps = dt.page_maps(lens, prompt_table, PAGE, free, sum(prompts), new_lens=lens)
    shared_x, _, _ = append(dt, g, cache, keys, maps, angles, norm)
    free = free[int(maps.counts[1]):]

    # what each request asks, behind its prompt
    table = prompt_table[torch.as_tensor(group, device=DEV)].clone()
    new = np.array([5, 1, 40, 17, 33, 2, 9])
    lens = np.array(prompts)[group] + new
    maps = dt.page_maps(i32(lens), table, PAGE, free, int(new.sum()), new_lens=i32(new))
    x, _, _ = append(dt, g, cache, keys, maps, angles, norm)
    free = free[int(maps.counts[1]):]
    vectors = torch.cat([shared_x, x])
    up = torch.randn(LATENT, HEADS * 256, generator=g, device=DEV).bfloat16() * LATENT ** -0.5
    kv = (vectors[:, :LATENT] @ up).view(-1, HEADS, 256)
    q = torch.randn(len(x), HEADS, 192, generator=g, device=DEV).bfloat16()
    before = np.concatenate([[0], np.cumsum(prompts)])
    q_starts = np.concatenate([[0], np.cumsum(new)])
    at = (q_starts, q_starts + sum(prompts), before[group], np.array(prompts)[group])
    tensors = (q, kv[..., :128], kv[..., 128:], vectors[:, LATENT:])
    out, lse = dt.attend_expanded_shared(*tensors, *(i32(v) for v in at), SCALE)
    size = float((q.float().abs().amax((0, 1)) * torch.cat([kv[..., :128].float().abs().amax((0, 1)), vectors[:, LATENT:].float().abs().amax(0)])).sum() * SCALE)
    close(out, lse, definition(*tensors, *(list(map(int, v)) for v in at)), size, 192)

    # tokens: in a graph, with the pages that they open
    step = dict(lens=i32(lens), free=free.clone(), out=None)
    group_starts, shared = i32(starts), i32(prompts)
    x0, q0 = torch.zeros(rows, LATENT + 64, device=DEV).bfloat16(), torch.zeros(rows, HEADS, LATENT + 64, device=DEV).bfloat16()
    iq, ik, w = torch.zeros(rows, 8, 128, device=DEV).bfloat16(), torch.zeros(rows, 128, device=DEV).bfloat16(), torch.rand(rows, 8, generator=g, device=DEV)

    def decode():
        maps = dt.page_maps(step["lens"], table, PAGE, step["free"], rows)
        turned = q0.clone()
        dt.append_latent(x0, cache, maps.slots, maps.row_lens, angles, weight=norm, q_rope=q0[..., LATENT:], q_out=turned[..., LATENT:])
        i, _ = dt.append_index(ik, keys, maps.slots, maps.row_lens, angles, q=iq)
        scores = dt.scores_paged(i, w, keys, maps.row_lens, table, table_rows=maps.table_rows)
        slots = dt.paged(scores, maps.row_lens, table, PAGE, 64, table_rows=maps.table_rows)
        some = dt.attend_selected(turned, cache, slots, LATENT, SCALE)
        every = dt.attend_shared(turned, cache, maps.row_lens, table, group_starts, shared, LATENT, SCALE, table_rows=maps.table_rows)
        return maps, turned, slots, some, every, dt.attend_paged(turned, cache, maps.row_lens, table, LATENT, SCALE, table_rows=maps.table_rows)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        keep, step["lens"] = step["lens"], i32([0] * rows)
        decode()
        step["lens"] = keep
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        maps, turned, slots, some, every, one = decode()
    for n in range(5):
        x0.copy_(torch.randn(rows, LATENT + 64, generator=g, device=DEV).bfloat16())
        q0.copy_(torch.randn(rows, HEADS, LATENT + 64, generator=g, device=DEV).bfloat16())
        iq.copy_(torch.randn(rows, 8, 128, generator=g, device=DEV).bfloat16())
        ik.copy_(torch.randn(rows, 128, generator=g, device=DEV).bfloat16())
        step["lens"].add_(1)
        graph.replay()
        torch.cuda.synchronize()
        lens = lens + 1
        taken = int(maps.counts[1])
        step["free"].copy_(torch.cat([step["free"][taken:], step["free"][:taken]]))
        flat, at = cache.view(-1, LATENT + 64), table.cpu().numpy()
        want, off = append_plain.latent(x0, norm, 1e-6, lens.tolist(), angles, False, LATENT)
        near(flat[maps.slots.long()], want, off)
        want, size = append_plain.turn(q0[..., LATENT:].double().cpu(), q0[..., LATENT:].double().cpu().abs(), lens.tolist(), angles, False)
        near(turned[..., LATENT:], want, size * 2.0 ** -22)
        every_at = [at[r, np.arange(m) // PAGE] * PAGE + np.arange(m) % PAGE for r, m in enumerate(lens)]
        size = logit_size(turned, flat, SCALE)
        want = serve_plain.attend(turned, flat, LATENT, SCALE, every_at)
        close(*every, want, size, LATENT + 64)
        close(*one, want, size, LATENT + 64)
        picked = [[s for s in row if s >= 0] for row in slots.tolist()]
        assert all(len(set(p)) == min(64, m) and set(p) <= set(e.tolist()) for p, e, m in zip(picked, every_at, lens))
        close(*some, serve_plain.attend(turned, flat, LATENT, SCALE, picked), size, LATENT + 64)
