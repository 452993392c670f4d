"""Expanded attention behind shared keys: queries that see nothing of a
neighbour's keys do not slow down the work on these."""
import numpy as np
import pytest

from tests.test_serve_attend_gpu import SCALE, i32
from tests.test_serve_behind_gpu import inputs
from tests.test_serve_wide_time_gpu import times

import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,new,own", [(16, 16, 20000), (16, 1, 2000)])
def test_one_shared_key_less(kind, heads, new, own):
    """Without any shared keys, queries of later requests have seen nothing yet while a tile goes over those of
    the first ones; with one shared key in front all have. The latter is more work, and the former has to take
    no more time than it (and 7%, for what a measurement is off by; looking for references took 14 to 20)."""
    import row_top_selection_amd as dt

    g = torch.Generator("cuda").manual_seed(1)
    requests = 32 // new
    starts = i32(np.arange(requests + 1) * new)
    k_starts = i32(1 + np.arange(requests + 1) * own)
    q, k, v, rope = inputs(g, 32, 1 + requests * own, heads, kind)
    zero, none, one = i32([0] * requests), i32([0] * requests), i32([1] * requests)

    def call(lens):
        return dt.attend_expanded_shared(q, k, v, rope, starts, k_starts, zero, lens, SCALE, max_keys=0)

    without, with_one = times(lambda: call(none), lambda: call(one))
    assert without < 1.07 * with_one, (without, with_one)
