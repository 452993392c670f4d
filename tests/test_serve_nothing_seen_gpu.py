"""Rows and queries that see nothing get zeros and -inf, also where others of their
workgroup see infinite numbers."""
import math

import pytest
import torch

from tests.test_serve_attend_gpu import SCALE, TYPES, i32, make
from tests.test_serve_behind_gpu import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("heads,latent,rows,kw", [
    (16, 512, 2, {}), (16, 512, 4, {}), (16, 512, 8, dict(max_shared_len=1 << 22)), (128, 512, 3, dict(max_shared_len=1 << 22)),
    (16, 256, 4, {}), (16, 256, 8, dict(max_shared_len=1 << 22)), (8, 512, 3, dict(max_own_len=0)),
])
@pytest.mark.parametrize("shared", [20, 1000])
def test_rows(kind, bad, heads, latent, rows, kw, shared):
    """Every second row is padding; the others share a token that is not finite. In one part, and in several."""
    import row_top_selection_amd as dt

    g = torch.Generator("cuda").manual_seed(rows)
    width = -(-shared // 16) + 1
    q, cache = make(g, rows, heads, latent, rows * width, 16, kind)
    cache.view(-1, latent + 64)[7, :latent] = bad
    lens = i32([shared if r % 2 else 0 for r in range(rows)])
    table = torch.arange(rows * width, device="cuda", dtype=torch.int32).view(rows, width)
    out, lse = dt.attend_shared(q, cache, lens, table, i32([0, rows]), i32([shared]), latent, SCALE, **kw)
    torch.cuda.synchronize()
    assert (out[::2] == 0).all() and (lse[::2] == -math.inf).all()
    assert not torch.isfinite(out[1::2]).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("shared_form", [False, True])
def test_queries(kind, bad, shared_form):
    """Prompts of more queries than keys: the first ones see none, and the keys' values are not finite."""
    import row_top_selection_amd as dt

    g = torch.Generator("cuda").manual_seed(1)
    q, k, v, rope = inputs(g, 60, 30, 3, kind)
    v[:] = bad
    q_starts, k_starts = i32([0, 40, 60]), i32([0, 25, 30])
    if shared_form:
        out, lse = dt.attend_expanded_shared(q, k, v, rope, q_starts, k_starts, i32([0, 0]), i32([0, 0]), SCALE)
    else:
        out, lse = dt.attend_expanded(q, k, v, rope, q_starts, k_starts, 40, SCALE)
    torch.cuda.synchronize()
    none = torch.zeros(60, dtype=torch.bool, device="cuda")
    none[:15] = none[40:55] = True
    assert (out[none] == 0).all() and (lse[none] == -math.inf).all()
    assert not torch.isfinite(out[~none]).any()
