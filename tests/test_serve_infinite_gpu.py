"""Indexer scores of infinite keys: what the formula gives, for every number
of heads."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


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
