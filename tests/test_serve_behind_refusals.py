"""What expanded attention behind shared keys refuses: the C calls before any
HIP call (fake pointers, no GPU), and the binding before it looks at a pointer."""
import math

import pytest
import torch

import row_top_selection_amd as dt

A16 = 0x10000
A4 = 0x10004
A8 = 0x10008


@pytest.fixture(scope="module")
def lib():
    return dt.lib()


def call(fn, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a)
    a.update(kw)
    return fn(*a.values())


BEHIND = dict(q=A16, q_row=1536, q_head=192, k=A16, k_row=2048, k_head=256, v=A16, v_row=2048, v_head=256, rope=A16,
              rope_row=64, type=0, heads=8, nope=128, rope_dim=64, value=128, scale=0.1, causal=1, qs=A16, ks=A16, ss=A16,
              sl=A16, requests=2, queries=100, keys=20000, longest=20000, out=A16, lse=A16, work=None, bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(requests=-1), 1), (dict(queries=-1), 1), (dict(keys=-1), 1), (dict(longest=-1), 1),
    (dict(queries=(1 << 30) + 1), 1), (dict(keys=(1 << 30) + 1), 1), (dict(heads=0), 1), (dict(heads=1025), 1),
    (dict(nope=64), 1), (dict(rope_dim=128), 1), (dict(value=64), 1), (dict(type=2), 1), (dict(scale=0.0), 1),
    (dict(scale=math.nan), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(rope=None), 1),
    (dict(out=None), 1), (dict(qs=None), 1), (dict(ks=None), 1), (dict(ss=None), 1), (dict(sl=None), 1),
    (dict(k_row=-8), 1), (dict(k_row=1 << 28), 1), (dict(q=A8), 2), (dict(k=A4), 2), (dict(v=A8), 2), (dict(rope=A8), 2),
    (dict(out=A4), 2), (dict(lse=0x10001), 2), (dict(q_head=196), 2), (dict(k_row=2052), 2), (dict(v_head=260), 2),
    (dict(rope_row=68), 2), (dict(), 6), (dict(work=A16, bytes=64), 6), (dict(work=A4, bytes=1 << 40), 2),
])
def test_attend_expanded_shared_refuses(lib, kw, code):
    assert call(lib.dsatopk_attend_expanded_shared, BEHIND, kw) == code


def test_nothing_to_do_is_no_error(lib):
    none = {k: None for k in ("q", "out", "lse", "qs", "ks", "ss", "sl")}
    assert call(lib.dsatopk_attend_expanded_shared, BEHIND, dict(queries=0, **none)) == 0
    assert call(lib.dsatopk_attend_expanded_shared, BEHIND, dict(requests=0, **none)) == 0


def test_expanded_shared_bytes(lib):
    assert dt.expanded_shared_bytes(0, 100, 1000) == 0
    assert dt.expanded_shared_bytes(8, 0, 1000) == 0
    assert dt.expanded_shared_bytes(8, 100, -1) == 0
    assert dt.expanded_shared_bytes(16, 65536, 100000) == 0  # fills the card
    assert dt.expanded_shared_bytes(8, 100, 200) == 0        # too few keys to split
    few = dt.expanded_shared_bytes(1, 300, 20000)
    assert few >= 2 * 300 * 130 * 4 and few % (300 * 130 * 4) == 0


def test_binding_refuses_host_tensors_and_gradients():
    n = torch.zeros(2, dtype=torch.int32)
    q, kv, rope = torch.zeros(4, 2, 192), torch.zeros(4, 2, 128), torch.zeros(4, 64)
    with pytest.raises(ValueError, match="device"):
        dt.attend_expanded_shared(q, kv, kv, rope, n, n, n[:1], n[:1], 0.1)
    with pytest.raises(ValueError, match="gradient"):
        dt.attend_expanded_shared(q.requires_grad_(), kv, kv, rope, n, n, n[:1], n[:1], 0.1)


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    dev = "cuda"
    bf = dict(dtype=torch.bfloat16, device=dev)
    q, kv, rope = torch.zeros(4, 2, 192, **bf), torch.zeros(4, 2, 128, **bf), torch.zeros(4, 64, **bf)
    starts, one = torch.tensor([0, 4], dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)

    def refused(*args, error=ValueError, **kw):
        with pytest.raises(error):
            dt.attend_expanded_shared(*args, **kw)

    refused(q, kv, kv[:3], rope, starts, starts, one, one, 0.1)
    refused(q, kv, kv, rope.half(), starts, starts, one, one, 0.1)
    refused(q[..., :128], kv, kv, rope, starts, starts, one, one, 0.1)
    refused(q, kv, kv, rope, starts, starts[:1], one, one, 0.1)
    refused(q, kv, kv, rope, starts, starts, one[:0], one, 0.1)
    refused(q, kv, kv, rope, starts, starts, one, starts, 0.1)
    refused(q, kv, kv, rope, starts, starts, one.long(), one, 0.1)
    refused(q, kv, kv, rope, starts, starts, one, one.cpu(), 0.1)
    refused(q, kv, kv, rope, starts, starts, one, one, 0.1, out=q)
    refused(q, kv, kv, rope, starts, starts, one, one, -0.1, error=dt.DsatopkError)
    refused(q, kv, kv, rope, starts, starts, one, one, 0.1, max_keys=-1, error=dt.DsatopkError)
    refused(q, kv, kv, rope, starts, starts, one, one, error=TypeError)
    with pytest.raises(ValueError, match="gradient"):
        dt.attend_expanded_shared(q, kv.clone().requires_grad_(), kv, rope, starts, starts, one, one, 0.1)
