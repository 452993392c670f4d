"""Expanded attention behind shared keys: infinite numbers and NaN among one
request's keys are that request's alone, also where its queries stand beside
others' in a tile."""
import math

import numpy as np
import pytest
import torch

from tests.test_serve_attend_gpu import SCALE, close, i32
from tests.test_serve_behind_gpu import definition, inputs

pytestmark = pytest.mark.gpu


def check_others(kind, heads, new, own, shared, bad_rows, bad, clean_requests, **kw):
    """Rows `bad_rows` of the keys and values (a mask) become `bad`; the results of `clean_requests`, which
    see none of them, are the definition's on the tensors as they were."""
    import row_top_selection_amd as dt

    g = torch.Generator("cuda").manual_seed(heads + len(new))
    front = max(s + n for s, n in shared)
    q_starts = np.concatenate([[0], np.cumsum(new)])
    k_starts = np.concatenate([[0], np.cumsum(own)]) + front
    q, k, v, rope = inputs(g, sum(new), front + sum(own), heads, kind)
    lists = (q_starts, k_starts, [s for s, _ in shared], [n for _, n in shared])
    want = definition(q, k, v, rope, *lists)
    size = float((q.float().abs().amax((0, 1)) * torch.cat([k.float().abs().amax((0, 1)), rope.float().abs().amax(0)])).sum() * SCALE)
    for t in (k, v, rope):
        t[bad_rows(front, k_starts)] = bad
    out, lse = dt.attend_expanded_shared(q, k, v, rope, *(i32(x) for x in lists), SCALE, **kw)
    torch.cuda.synchronize()
    pick = np.concatenate([np.arange(q_starts[r], q_starts[r + 1]) for r in clean_requests])
    assert len(pick)
    at = torch.as_tensor(pick)
    close(out[at.cuda()], lse[at.cuda()], tuple(x[at] for x in want), size, 192)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("heads,new,own,shared,kw", [
    (2, [16, 16, 16], [20, 300, 16], [(0, 70)] * 3, {}),                      # in one wave
    (3, [10, 50, 70, 3], [10, 50, 90, 200], [(0, 0)] * 4, {}),                # in several, without shared keys
    (1, [5, 9, 6], [700, 5000, 900], [(0, 3000)] * 3, {}),                    # split by keys
    (8, [1] * 300, [1, 40, 2] * 100, [(0, 33)] * 300, dict(max_keys=0)),      # many short ones
    (1, [1] * 1100, [3] * 1100, [(0, 9), (9, 1)] * 550, dict(max_keys=5000)),  # in packed runs, split
    (160, [3] * 100, [9] * 100, [(0, 40)] * 100, {}),                         # eight waves
], ids=["wave", "waves", "split", "short", "runs", "eight"])
def test_own_keys(kind, bad, heads, new, own, shared, kw):
    def rows(front, k_starts):
        return slice(int(k_starts[1]), int(k_starts[2]))

    check_others(kind, heads, new, own, shared, rows, bad, [0, *range(2, len(new))], **kw)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,requests,kw", [(8, 300, dict(max_keys=0)), (1, 1100, dict(max_keys=5000)), (160, 300, {})])
def test_shared_keys(kind, heads, requests, kw):
    """Runs of three single tokens; every second run's shared keys are bad."""
    shared = [((r // 3) % 2 * 20, 20) for r in range(requests)]

    def rows(front, k_starts):
        return slice(20, 40)

    check_others(kind, heads, [1] * requests, [2] * requests, shared, rows, math.nan,
                 [r for r in range(requests) if r // 3 % 2 == 0], **kw)


def test_last_row_of_a_request():
    """Only the last of a request's values is infinite: all of its rows but the last, in the same tile, may
    be NaN, and the neighbours are not."""
    def rows(front, k_starts):
        return slice(int(k_starts[2]) - 1, int(k_starts[2]))

    check_others("bf16", 4, [30, 30, 30, 30], [30, 30, 30, 30], [(0, 100)] * 4, rows, -math.inf, [0, 2, 3])
