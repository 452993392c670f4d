"""Attention behind shared tokens, workgroups whose waves take different tokens of
a tile: a row that ends among another wave's needs no references."""
import pytest
import torch

from tests.test_serve_attend_gpu import SCALE, TYPES, i32
from tests.test_serve_wide_time_gpu import times

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_rows_that_end_in_the_first_tile(kind):
    """Groups of two rows, of which one ends after 5 tokens of 2048: no other result for the other one, and no
    more time than if both see all."""
    import row_top_selection_amd as dt

    g = torch.Generator("cuda").manual_seed(1)
    groups, shared, page, rows = 512, 2048, 64, 1024
    cache = torch.randn(shared // page, page, 576, generator=g, device="cuda").to(TYPES[kind])
    q = torch.randn(rows, 16, 576, generator=g, device="cuda").to(TYPES[kind])
    table = torch.arange(shared // page, device="cuda", dtype=torch.int32).expand(rows, -1).contiguous()
    whole = torch.full((rows,), shared, dtype=torch.int32, device="cuda")
    uneven = whole.clone()
    uneven[1::2] = 5
    starts, lens_shared = i32(range(0, rows + 1, 2)), i32([shared] * groups)

    def call(lens):
        return dt.attend_shared(q, cache, lens, table, starts, lens_shared, 512, SCALE, max_shared_len=shared, max_own_len=0)

    (out, lse), (want, want_lse) = call(uneven), call(whole)
    short, short_lse = dt.attend_paged(q, cache, i32([5] * rows), table, 512, SCALE, max_seq_len=5)
    torch.cuda.synchronize()
    # weights are rounded after a reference is found, which may be another one: half a step each, and the results'
    size = cache[0, :5, :512].float().abs().max()
    assert torch.equal(out[::2], want[::2]) and torch.equal(lse[::2], want_lse[::2])
    assert ((out[1::2].float() - short[1::2].float()).abs() <= 4 * torch.finfo(TYPES[kind]).eps * size).all()
    assert ((lse[1::2] - short_lse[1::2]).abs() <= 1e-4).all()
    of_uneven, of_whole = times(lambda: call(uneven), lambda: call(whole))
    # looking for references takes 12% of a tile
    assert of_uneven < 1.07 * of_whole, (of_uneven, of_whole)
