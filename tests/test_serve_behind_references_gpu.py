"""Expanded attention behind shared keys: scores that rise and fall by tens to
hundreds between the shared and the own keys, along them, and from request to
request, so that references are outgrown, found late and far apart."""
import numpy as np
import pytest
import torch

from tests.test_serve_attend_gpu import SCALE, TYPES
from tests.test_serve_behind_gpu import check, inputs

pytestmark = pytest.mark.gpu

WAYS = ["own", "shared", "along", "apart"]


def levels(way, front, k_starts, rng):
    """A level for each key, of -1 to 1."""
    n = int(k_starts[-1])
    at = np.zeros(n)
    own = np.arange(front, n)
    if way == "own":          # every request's own keys above or below the shared ones, by a size of its own
        for a, b in zip(k_starts, k_starts[1:]):
            at[a:b] = rng.uniform(-1, 1)
    elif way == "shared":     # the shared keys rise, and the own ones are as at the beginning
        at[:front] = np.linspace(0, 1, front)
    elif way == "along":      # up and down along each request's own keys, one step for each
        for a, b in zip(k_starts, k_starts[1:]):
            at[a:b] = rng.permutation(np.linspace(-1, 1, b - a)) if b - a > 1 else 1
    else:                     # shared keys far below or above, single own ones far above the others
        at[:front] = rng.choice([-1.0, 1.0])
        at[rng.choice(own, max(len(own) // 40, 1))] = 1
    return at


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("most", [30, 250])
@pytest.mark.parametrize("heads,new,own,shared,kw", [
    (2, [16] * 6, [20, 300, 16, 100, 16, 50], [(0, 130)] * 6, {}),            # several requests a wave
    (3, [5, 60, 2, 90], [5, 60, 200, 90], [(0, 0), (0, 40), (0, 40), (0, 0)], {}),
    (1, [7, 20, 6], [700, 3000, 900], [(0, 2500)] * 3, {}),                   # split by keys
    (8, [1] * 270, [1, 40, 2] * 90, [(0, 33)] * 270, dict(max_keys=0)),       # packed
    (1, [1] * 700, [3] * 700, [(0, 9), (9, 1)] * 350, dict(max_keys=5000)),   # packed and split
    (160, [3] * 90, [9] * 90, [(0, 40)] * 90, {}),                            # eight waves
], ids=["wave", "waves", "split", "packed", "runs", "eight"])
def test_references(kind, way, most, heads, new, own, shared, kw):
    import row_top_selection_amd as dt

    g = torch.Generator("cuda").manual_seed(len(new) + heads)
    rng = np.random.default_rng(len(new) + most)
    front = max(s + n for s, n in shared)
    q_starts = np.concatenate([[0], np.cumsum(new)])
    k_starts = np.concatenate([[0], np.cumsum(own)]) + front
    q, k, v, rope = inputs(g, sum(new), front + sum(own), heads, kind)
    # scores differ by up to `most` either way, by a factor for each query and head
    rope[:, 0] = torch.as_tensor(levels(way, front, k_starts, rng)).to("cuda", TYPES[kind])
    factor = 2 * torch.rand(sum(new), heads, generator=g, device="cuda") - 1
    q[..., 128] = (factor * most / SCALE).to(TYPES[kind])
    check(dt, (q, k, v, rope), q_starts, k_starts, [s for s, _ in shared], [n for _, n in shared], **kw)
