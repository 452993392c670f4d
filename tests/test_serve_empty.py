"""Tensors without entries in the serving operators: torch gives them a null
pointer, which is no error where nothing of them is read."""
import numpy as np
import pytest
import torch

import row_top_selection_amd as dt
from tests.test_serve_refusals import RAGGED, call


@pytest.fixture(scope="module")
def lib():
    return dt.lib()


def test_no_keys_are_no_error(lib):
    # nothing is launched: there is no column to write
    assert call(lib.dsatopk_scores_ragged, RAGGED, dict(n=0, keys=None)) == 0
    assert call(lib.dsatopk_scores_ragged, RAGGED, dict(n=0, keys=None, out=None, columns=0, out_stride=0)) == 0
    assert call(lib.dsatopk_scores_ragged, RAGGED, dict(keys=None)) == 1
    assert call(lib.dsatopk_scores_ragged, RAGGED, dict(out=None)) == 1


def i32(v):
    return torch.as_tensor(np.asarray(v, dtype=np.int32)).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float8_e4m3fn])
def test_scores_of_an_empty_cache(kind):
    q, w = torch.ones(3, 64, 128, device="cuda").to(kind), torch.ones(3, 64, device="cuda")
    scales = torch.ones(0, 16, device="cuda")
    out = torch.full((3, 64), 5.0, device="cuda")
    for s in (None, scales):
        got = dt.scores_paged(q, w, torch.ones(0, 16, 128, device="cuda").to(kind), i32([0, 64, 9]), i32(np.zeros((3, 4))),
                              key_scales=s, out=out.clone())
        # pages that are not there score 0
        want = torch.full((3, 64), 5.0, device="cuda")
        want[1], want[2, :9] = 0.0, 0.0
        assert torch.equal(got, want)
    for s in (None, scales[:, 0].contiguous()):
        got = dt.scores_ragged(q, w, torch.ones(0, 128, device="cuda").to(kind), i32([0, 7, 9]), i32([0, 0, 3]),
                               key_scales=s, out=out.clone())
        assert torch.equal(got, out)
    assert dt.scores_ragged(q, w, torch.ones(0, 128, device="cuda").to(kind), i32([0] * 3), i32([0] * 3)).shape[0] == 3
    none = torch.empty(3, 0, device="cuda")
    assert dt.scores_ragged(q, w, torch.ones(8, 128, device="cuda").to(kind), i32([8] * 3), i32([0] * 3), out=none) is none


@pytest.mark.gpu
@pytest.mark.parametrize("requests", [1, 3])
def test_page_maps_of_a_table_without_columns(requests):
    """Every new token is past the table's width: counted, without a slot."""
    from tests import serve_plain

    lens, free = [5, 0, 9][:requests], np.arange(20)
    table = torch.empty(requests, 0, dtype=torch.int32, device="cuda")
    got = dt.page_maps(i32(lens), table, 4, i32(free), 16, new_lens=i32(lens))
    want = serve_plain.page_maps(lens, lens, np.zeros((requests, 0)), 4, free, 16)
    for name in ("token_starts", "slots", "table_rows", "row_lens", "counts"):
        assert getattr(got, name).tolist() == list(want[name]), name


@pytest.mark.gpu
def test_a_table_of_more_positions_than_a_row_may_have():
    """2048 pages of 2^20 tokens: no row is that long, and the call's default
    bound on the rows is no reason to refuse it."""
    cache = torch.zeros(1, 1 << 20, 320, dtype=torch.bfloat16, device="cuda")
    cache[0, :9, 3] = 2.0
    q = torch.zeros(1, 4, 320, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, 2048, dtype=torch.int32, device="cuda")
    out, lse = dt.attend_paged(q, cache, i32([9]), table, 256, 0.1)
    assert (out[..., 3] == 2).all() and (lse - np.log(9)).abs().max() < 1e-6
