"""Attention behind shared tokens, 128 heads a workgroup: rows that end early cost
nothing once a reference has been outgrown."""
import math

import pytest
import torch

from tests.test_serve_attend_gpu import SCALE, TYPES, i32

pytestmark = pytest.mark.gpu


def times(*calls):
    """The shortest time of each call (us, among ten others), the calls taken in turn."""
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = [math.inf] * len(calls)
    for _ in range(9):
        for i, call in enumerate(calls):
            call()
            begin.record()
            for _ in range(10):
                call()
            end.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], begin.elapsed_time(end) * 100)
    return best


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_rows_that_end_before_a_new_reference(kind):
    """Scores grow by 20 at token 128 of 1024. Every second row ends before that, in the same waves as those
    that see all: less work than if all see all, and no other result for these."""
    import row_top_selection_amd as dt

    g = torch.Generator("cuda").manual_seed(1)
    rows, shared, page = 2048, 1024, 64
    cache = torch.randn(shared // page, page, 576, generator=g, device="cuda")
    cache.view(-1, 576)[:, 512] = torch.arange(shared, device="cuda") >= 128
    q = 0.1 * torch.randn(rows, 16, 576, generator=g, device="cuda")
    q[..., 512] = 20 / SCALE
    cache, q = cache.to(TYPES[kind]), q.to(TYPES[kind])
    table = torch.arange(shared // page, device="cuda", dtype=torch.int32).expand(rows, -1).contiguous()
    whole = torch.full((rows,), shared, dtype=torch.int32, device="cuda")
    uneven = whole.clone()
    uneven[::2] = 40

    def call(lens):
        return dt.attend_shared(q, cache, lens, table, i32_starts, i32_shared, 512, SCALE, max_shared_len=shared, max_own_len=0)

    i32_starts, i32_shared = i32([0, rows]), i32([shared])
    (out, lse), (want, want_lse) = call(uneven), call(whole)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and not math.isinf(float(lse.min()))
    assert torch.equal(out[1::2], want[1::2]) and torch.equal(lse[1::2], want_lse[1::2])
    of_uneven, of_whole = times(lambda: call(uneven), lambda: call(whole))
    assert of_uneven < 1.5 * of_whole, (of_uneven, of_whole)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_a_row_that_is_no_number(kind):
    """The queries of one row in eight are NaN: the others get what they get without them, in the same time."""
    import row_top_selection_amd as dt

    g = torch.Generator("cuda").manual_seed(2)
    rows, shared, page = 2048, 1024, 64
    cache = torch.randn(shared // page, page, 576, generator=g, device="cuda").to(TYPES[kind])
    q = (0.1 * torch.randn(rows, 16, 576, generator=g, device="cuda")).to(TYPES[kind])  # (references hold for all tokens)
    odd = q.clone()
    odd[::8] = math.nan
    table = torch.arange(shared // page, device="cuda", dtype=torch.int32).expand(rows, -1).contiguous()
    at = (i32([shared] * rows), table, i32([0, rows]), i32([shared]), 512, SCALE)

    def call(queries):
        return dt.attend_shared(queries, cache, *at, max_shared_len=shared, max_own_len=0)

    (out, lse), (want, want_lse) = call(odd), call(q)
    torch.cuda.synchronize()
    numbers = torch.arange(rows, device="cuda") % 8 != 0
    assert torch.equal(out[numbers], want[numbers]) and torch.equal(lse[numbers], want_lse[numbers])
    assert torch.isnan(out[~numbers]).all() and torch.isnan(lse[~numbers]).all()
    of_odd, of_all = times(lambda: call(odd), lambda: call(q))
    assert of_odd < 1.5 * of_all, (of_odd, of_all)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("spread", [1.7, 3.5, 7.0])
def test_scores_that_spread_far(kind, spread):
    """Random scores that spread by 1.7 to 7 outgrow references again and again. That may cost as much again as the
    call itself (half precision), but not several times as much, as where every tile is begun anew."""
    import row_top_selection_amd as dt

    g = torch.Generator("cuda").manual_seed(3)
    rows, shared, page = 64, 16384, 64
    cache = torch.randn(shared // page, page, 576, generator=g, device="cuda").to(TYPES[kind])
    q = torch.randn(rows, 16, 576, generator=g, device="cuda") / (SCALE * 24)  # scores of size 1
    table = torch.arange(shared // page, device="cuda", dtype=torch.int32).expand(rows, -1).contiguous()
    at = (i32([shared] * rows), table, i32([0, rows]), i32([shared]), 512, SCALE)

    def call(queries):
        return dt.attend_shared(queries, cache, *at, max_shared_len=shared, max_own_len=0)

    near, far = (0.4 * q).to(TYPES[kind]), (spread * q).to(TYPES[kind])
    of_near, of_far = times(lambda: call(near), lambda: call(far))
    assert of_far < 3 * of_near, (of_far, of_near)
