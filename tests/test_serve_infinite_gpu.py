"""Indexer scores of infinite keys and queries: what the formula gives, for
every number of heads."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}


def i32(v):
    return torch.as_tensor(np.asarray(v, dtype=np.int32)).to(DEV)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [1, 20, 31, 32, 33, 64, 65, 100, 128])
def test_infinite_keys_of_any_number_of_heads(kind, heads):
    """A key with an infinite element that all heads' queries meet with a
    positive one: all heads' products are infinite, and so is the score; a
    negative infinity leaves no head anything, and a score of 0."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads)
    q = torch.randn(2, heads, 128, generator=g, device=DEV).to(TYPES[kind])
    q[..., 40] = 1.5
    w = torch.rand(2, heads, generator=g, device=DEV) + 0.1
    w[1] *= -1
    keys = torch.randn(300, 128, generator=g, device=DEV).to(TYPES[kind])
    plain = dt.scores_ragged(q, w, keys, i32([300, 300]), i32([0, 0])).clone()
    keys[7, 40], keys[201, 40], keys[290, 3] = math.inf, -math.inf, math.nan
    got = dt.scores_ragged(q, w, keys, i32([300, 300]), i32([0, 0]))
    table = i32([[0], [0]])
    paged = dt.scores_paged(q, w, torch.cat([keys, keys[:212]]).view(1, 512, 128), i32([300, 300]), table)
    for out in (got[:, :300], paged[:, :300]):
        assert out[:, 7].tolist() == [math.inf, -math.inf]
        assert out[:, 201].tolist() == [0.0, 0.0]
        assert torch.isnan(out[:, 290]).all()
        rest = torch.ones(300, dtype=torch.bool, device=DEV)
        rest[[7, 201, 290]] = False
        assert torch.equal(out[:, rest], plain[:, :300][:, rest])


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("scaled", [False, True])
def test_absent_pages_score_0_whatever_the_query(kind, scaled):
    """Columns of a page outside the cache have the score 0, also for rows
    whose queries or weights hold infinities and NaN."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(3)
    q = torch.randn(4, 24, 64, generator=g, device=DEV)
    w = torch.rand(4, 24, generator=g, device=DEV)
    q[1, 3, 5], w[2, 0], w[3, 1] = math.nan, math.inf, math.nan
    if kind != "fp8":
        q[0, 0, 0] = math.inf
    keys = torch.randn(3, 16, 64, generator=g, device=DEV).to(TYPES[kind])
    scales = torch.rand(3, 16, generator=g, device=DEV) if scaled else None
    table = i32([[0, -1, 2, 3]] * 4)
    out = dt.scores_paged(q.to(TYPES[kind]), w, keys, i32([60] * 4), table, key_scales=scales,
                          out=torch.full((4, 64), -7.0, device=DEV))
    assert (out[:, 16:32] == 0).all() and (out[:, 48:60] == 0).all()
    assert (out[:, 60:] == -7).all()
