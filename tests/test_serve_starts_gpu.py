"""Attention behind shared tokens with starts of groups that do not rise, which
no caller should give: what is read and written stays in the workspace."""
import pytest
import torch

from tests.test_serve_attend_gpu import SCALE, i32, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("starts,shared", [
    ([0, 7, 6, 2, 8], [0, 100, 100, 100]),  # rows 2 to 5 are before the group that a search for theirs ends at
    ([0, 8, 5, 3, 1, 8], [0, 33, 1, 90, 70]),
    ([5, 9, -4, 1, 0], [100, 0, 100, 64]),
])
@pytest.mark.parametrize("kw", [{}, dict(max_shared_len=1, max_own_len=1), dict(max_shared_len=1 << 22)])
def test_nothing_before_the_workspace_is_read(starts, shared, kw):
    """The workspace holds zeros, by which a block that nobody has numbered has one part, and stands behind NaN."""
    import row_top_selection_amd as dt

    g = torch.Generator("cuda").manual_seed(1)
    rows, heads, page, width = 8, 16, 16, 10
    q, cache = make(g, rows, heads, 512, rows * width, page, "bf16")
    table = torch.arange(rows * width, device="cuda", dtype=torch.int32).view(rows, width)
    lens = i32([130, 101, 150, 120, 110, 160, 105, 140])
    bounds = (kw.get("max_shared_len", width * page), kw.get("max_own_len", width * page))
    need, guard = dt.shared_bytes(rows, heads, 512, len(shared), *bounds), 1 << 20
    room = torch.full((guard + need + guard,), 255, dtype=torch.uint8, device="cuda")
    room[guard:guard + need] = 0
    out, lse = dt.attend_shared(q, cache, lens, table, i32(starts), i32(shared), 512, SCALE, workspace=room[guard:guard + need], **kw)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert (room[:guard] == 255).all() and (room[guard + need:] == 255).all()
