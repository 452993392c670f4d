"""Expanded attention behind shared keys, on the GPU against the definition in 64
bits (tests/serve_plain.py)."""
import math

import numpy as np
import pytest
import torch

from tests import serve_plain
from tests.test_serve_attend_gpu import SCALE, TYPES, close, i32

pytestmark = pytest.mark.gpu

DEV = "cuda"


def inputs(g, queries, keys, heads, kind):
    q = torch.randn(queries, heads, 192, generator=g, device=DEV).to(TYPES[kind])
    kv = torch.randn(keys, heads, 256, generator=g, device=DEV).to(TYPES[kind])
    rope = torch.randn(keys, 64, generator=g, device=DEV).to(TYPES[kind])
    return q, kv[..., :128], kv[..., 128:], rope


def definition(q, k, v, rope, q_starts, k_starts, shared_starts, shared_lens, causal=True):
    """Each request by itself, with its shared keys in front of its own; rows of no request are NaN."""
    out = torch.full((q.shape[0], q.shape[1], 128), math.nan, dtype=torch.float64)
    size, lse = out.clone(), torch.full(q.shape[:2], math.nan, dtype=torch.float64)
    for r in range(len(q_starts) - 1):
        a, b = q_starts[r], q_starts[r + 1]
        if a == b:
            continue
        s, n, own = shared_starts[r], shared_lens[r], k_starts[r + 1] - k_starts[r]
        at = torch.cat([torch.arange(s, s + n), torch.arange(k_starts[r], k_starts[r + 1])]).to(DEV)
        x = q[a:b].double().cpu()
        key = torch.cat([k[at].double().cpu(), rope[at].double().cpu()[:, None].expand(-1, q.shape[1], -1)], -1)
        logits = torch.einsum("ihd,jhd->ihj", x, key) * SCALE
        if causal:
            j, i = torch.arange(n + own), torch.arange(b - a)[:, None]
            logits.masked_fill_(((j >= n) & (j - n > i + own - (b - a)))[:, None], -math.inf)
        lse[a:b] = torch.logsumexp(logits, -1)
        w = torch.exp(logits - torch.where(torch.isfinite(lse[a:b]), lse[a:b], 0.0)[..., None])
        value = v[at].double().cpu()
        out[a:b], size[a:b] = torch.einsum("ihj,jhd->ihd", w, value), torch.einsum("ihj,jhd->ihd", w, value.abs())
    return out, lse, size


def check(dt, tensors, q_starts, k_starts, shared_starts, shared_lens, causal=True, **kw):
    q, k, v, rope = tensors
    rows = q.shape[0]
    out, lse = torch.full((rows, q.shape[1], 128), 7.0, device=DEV).to(q.dtype), torch.full((rows, q.shape[1]), 7.0, device=DEV)
    dt.attend_expanded_shared(q, k, v, rope, i32(q_starts), i32(k_starts), i32(shared_starts), i32(shared_lens), SCALE, causal=causal, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    want = definition(q, k, v, rope, q_starts, k_starts, shared_starts, shared_lens, causal)
    real = ~torch.isnan(want[1][:, 0])
    assert (out[~real.to(DEV)] == 7).all() and (lse[~real.to(DEV)] == 7).all()  # rows of no request are left as they were
    size = 0.0
    if len(k):
        size = float((q.float().abs().amax((0, 1)) * torch.cat([k.float().abs().amax((0, 1)), rope.float().abs().amax(0)])).sum() * SCALE)
    pick = real.to(DEV)
    close(out[pick], lse[pick], tuple(x[real] for x in want), size, 192)
    return out, lse


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,new,own,shared", [
    # new tokens of each request, own keys of each, (first shared row, length) of each
    (1, [1], [1], [(0, 0)]),
    (2, [5], [5], [(0, 64)]),
    (3, [5, 9, 1], [5, 9, 1], [(0, 33)] * 3),
    (2, [16] * 20, [16] * 20, [(0, 130)] * 20),                        # several requests a wave
    (2, [1] * 140, [1] * 140, [(3, 70)] * 140),                       # single tokens
    (1, [130, 2, 300], [130, 2, 300], [(0, 257), (0, 257), (5, 20)]),
    (8, [33, 31, 0, 64, 7], [40, 31, 9, 100, 7], [(0, 50), (0, 50), (9, 9), (0, 50), (50, 17)]),
    (4, [20, 30, 10, 5], [0, 3, 10, 100], [(0, 45), (0, 0), (0, 0), (0, 45)]),  # fewer keys than queries
    (2, [10, 10, 10], [10, 10, 10], [(0, 30), (30, 30), (0, 30)]),         # the same keys, apart
    (9, [100, 200], [100, 200], [(0, 1000)] * 2),
])
def test_behind(kind, heads, new, own, shared):
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(heads * len(new))
    front = max(s + n for s, n in shared)
    q_starts = np.concatenate([[0], np.cumsum(new)])
    k_starts = np.concatenate([[0], np.cumsum(own)]) + front
    tensors = inputs(g, sum(new), front + sum(own), heads, kind)
    at = (q_starts, k_starts, [s for s, _ in shared], [n for _, n in shared])
    first = check(dt, tensors, *at)
    check(dt, tensors, *at, causal=False)
    for bound in (0, 100, 5000, 100000):  # how the keys are split, and nothing else
        check(dt, tensors, *at, max_keys=bound)
    again = check(dt, tensors, *at)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_enough_rows_for_eight_waves():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(1)
    rng = np.random.default_rng(1)
    new = rng.integers(1, 300, 60)
    new[7:12] = [1, 2, 0, 31, 33]
    q_starts = np.concatenate([[0], np.cumsum(new)])
    shared = [(0, 200)] * 25 + [(200, 31)] * 20 + [(0, 200)] * 15
    tensors = inputs(g, int(new.sum()), 231 + int(new.sum()), 16, "bf16")
    assert dt.expanded_shared_bytes(16, int(new.sum()), 500) == 0 and new.sum() > 256 * 16
    check(dt, tensors, q_starts, q_starts + 231, [s for s, _ in shared], [n for _, n in shared])


def test_rows_of_no_request_and_keys_that_are_not_there():
    """Starts that leave rows out, shared rows that reach past the keys, negative ones, keys cut off."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(2)
    tensors = inputs(g, 90, 200, 3, "bf16")
    q_starts, k_starts = [10, 30, 31, 75], [100, 120, 121, 165]
    check(dt, tensors, q_starts, k_starts, [0, 0, 40], [60, 60, 50])
    got = dt.attend_expanded_shared(*tensors, i32(q_starts), i32(k_starts), i32([-5, 190, 300]), i32([60, 500, 7]), SCALE)
    want = dt.attend_expanded_shared(*tensors, i32(q_starts), i32(k_starts), i32([0, 190, 0]), i32([60, 10, 0]), SCALE)
    for a, b in zip(got, want):
        assert torch.equal(a[10:75], b[10:75])
    got = dt.attend_expanded_shared(*tensors, i32([0, 20, 500]), i32([150, 170, 10 ** 6]), i32([0, 0]), i32([-3, 10]), SCALE, causal=False)
    want = dt.attend_expanded_shared(*tensors, i32([0, 20, 90]), i32([150, 170, 200]), i32([0, 0]), i32([0, 10]), SCALE, causal=False)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_without_shared_keys_as_attend_expanded():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(3)
    starts, zero = i32([0, 100, 130, 400]), i32([0] * 3)
    tensors = inputs(g, 400, 400, 4, "bf16")
    a, la = dt.attend_expanded(*tensors, starts, starts, 270, SCALE)
    b, lb = dt.attend_expanded_shared(*tensors, starts, starts, zero, zero, SCALE)
    # both are off by half a step of the result, and half a step of each weight
    assert ((a.float() - b.float()).abs() <= 2 ** -7 * (a.float().abs() + tensors[2].float().abs().max())).all()
    assert ((la - lb).abs() <= 1e-5 * (1 + la.abs())).all()


def test_hidden_keys_may_hold_anything():
    """Infinities and NaN in the rows of k, v and k_rope that no query sees: between the shared and the own
    ones, and behind the last."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(4)
    q, k, v, rope = inputs(g, 60, 300, 2, "bf16")
    q_starts, k_starts, s, n = [0, 25, 60], [150, 175, 210], [0, 0], [77, 77]
    want = dt.attend_expanded_shared(q, k, v, rope, i32(q_starts), i32(k_starts), i32(s), i32(n), SCALE)
    for rows in (slice(77, 150), slice(210, 300)):
        for t in (k, v, rope):
            t[rows][::2], t[rows][1::2] = math.nan, math.inf
    got = dt.attend_expanded_shared(q, k, v, rope, i32(q_starts), i32(k_starts), i32(s), i32(n), SCALE)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.isfinite(got[0]).all()


def test_strides_and_workspace():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(5)
    q, k, v, rope = inputs(g, 40, 1600, 2, "fp16")
    at = (i32([0, 15, 40]), i32([1560, 1575, 1600]), i32([0, 0]), i32([1560, 1560]), SCALE)
    want, want_lse = dt.attend_expanded_shared(q, k, v, rope, *at)
    wide_q = torch.zeros(40, 3, 256, device=DEV).half()
    wide_q[:, 1:, 8:200] = q
    wide_r = torch.zeros(1600, 72, device=DEV).half()
    wide_r[:, 8:] = rope
    heads_first = k.transpose(0, 1).contiguous().transpose(0, 1)
    need = dt.expanded_shared_bytes(2, 40, 1600)
    assert need > 0
    work = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    got, lse = dt.attend_expanded_shared(wide_q[:, 1:, 8:200], heads_first, v.contiguous(), wide_r[:, 8:], *at, workspace=work)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    with pytest.raises(dt.DsatopkError) as e:
        dt.attend_expanded_shared(q, k, v, rope, *at, workspace=work[:need - 16])
    assert e.value.status == 6


def test_keys_past_32_bits_of_bytes():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(6)
    big = torch.zeros(40000, 1, 1 << 16, device=DEV, dtype=torch.bfloat16)  # 5.2 GB
    q, k, v, rope = inputs(g, 30, 40000, 1, "bf16")
    big[..., :128], big[..., 128:256] = k, v
    at = (i32([0, 10, 30]), i32([39960, 39970, 39990]), i32([39000, 39000]), i32([900, 900]), SCALE)
    want = dt.attend_expanded_shared(q, k, v, rope, *at)
    got = dt.attend_expanded_shared(q, big[..., :128], big[..., 128:256], rope, *at)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(dt, (q, big[..., :128], big[..., 128:256], rope), [0, 10, 30], [39960, 39970, 39990], [39000] * 2, [900] * 2)


def test_captured_and_replayed():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(7)
    rng = np.random.default_rng(7)
    q, k, v, rope = inputs(g, 300, 2000, 2, "bf16")
    starts, keys, ss, sl = i32([0] * 6), i32([0] * 6), i32([0] * 5), i32([0] * 5)

    def call():
        return dt.attend_expanded_shared(q, k, v, rope, starts, keys, ss, sl, SCALE)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for n in range(4):
        q.copy_(torch.randn(q.shape, generator=g, device=DEV).bfloat16())
        starts.copy_(i32([0, *sorted(rng.integers(0, 300, 4)), 300]))
        keys.copy_(starts + 1500)
        ss.copy_(i32(rng.integers(0, 2, 5) * 700))
        sl.copy_(i32(rng.integers(0, 2, 5) * 400 + 100))
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), n


def test_nothing_to_do():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(8)
    none = i32([])
    q, k, v, rope = inputs(g, 4, 10, 2, "bf16")
    out, lse = dt.attend_expanded_shared(q[:0], k, v, rope, i32([0, 0]), i32([0, 0]), i32([0]), i32([5]), SCALE)
    assert out.shape == (0, 2, 128) and lse.shape == (0, 2)
    dt.attend_expanded_shared(q, k, v, rope, i32([0]), i32([0]), none, none, SCALE)
    # no keys at all
    out, lse = dt.attend_expanded_shared(q, k[:0], v[:0], rope[:0], i32([0, 4]), i32([0, 0]), i32([0]), i32([5]), SCALE)
    assert (out == 0).all() and (lse == -math.inf).all()
