"""Expanded attention behind shared keys: which queries stand together, for more
requests than a workgroup has threads."""
import numpy as np
import pytest
import torch

from tests.test_serve_behind_gpu import check, inputs

pytestmark = pytest.mark.gpu

DEV = "cuda"


def case(rng, requests, most, run):
    """Queries, own keys and shared keys of `requests`, in runs of up to `run` that share, some of them empty."""
    new = rng.integers(0, most + 1, requests)
    new[rng.integers(0, requests, 3)] = most
    own = new + rng.integers(0, 5, requests)
    shared, at = [], 0
    while len(shared) < requests:
        n = int(rng.integers(0, 40))
        shared += [(at, n)] * int(rng.integers(1, run + 1))
        at += n
    return new, own, shared[:requests], at


@pytest.mark.parametrize("heads,requests,most,run", [
    (1, 255, 3, 4), (1, 256, 2, 300), (2, 257, 2, 40), (1, 700, 3, 1), (1, 700, 1, 900), (1, 1400, 2, 90),
    (80, 600, 2, 50), (160, 520, 1, 7),   # eight waves
    (1, 9, 400, 3),
])
def test_runs(heads, requests, most, run):
    import row_top_selection_amd as dt

    rng = np.random.default_rng(requests + most)
    g = torch.Generator(DEV).manual_seed(requests)
    new, own, shared, front = case(rng, requests, most, run)
    q_starts = np.concatenate([[0], np.cumsum(new)])
    k_starts = np.concatenate([[0], np.cumsum(own)]) + front
    tensors = inputs(g, int(new.sum()), front + int(own.sum()), heads, "bf16")
    at = (q_starts, k_starts, [s for s, _ in shared], [n for _, n in shared])
    check(dt, tensors, *at)
    check(dt, tensors, *at, max_keys=100000)


def test_empty_requests_between_runs():
    """Empty requests that share with their neighbours, or do not, at the beginning, the end and in between."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(5)
    new = [0, 0, 3, 0, 200, 0, 0, 40, 0]
    shared = [(0, 9), (4, 4), (0, 50), (7, 7), (0, 50), (0, 50), (1, 1), (0, 50), (3, 3)]
    q_starts = np.concatenate([[0], np.cumsum(new)])
    tensors = inputs(g, sum(new), 50 + sum(new), 3, "fp16")
    check(dt, tensors, q_starts, q_starts + 50, [s for s, _ in shared], [n for _, n in shared])
