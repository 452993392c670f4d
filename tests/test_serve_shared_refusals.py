"""What attention behind shared tokens refuses: the C calls before any HIP
call (fake pointers, no GPU), and the binding before it looks at a pointer."""
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


SHARED = dict(q=A16, q_row=9216, q_head=576, cache=A16, pages=10, page=36864, token=576, ps=64, type=0, heads=16,
              latent=512, rope=64, scale=0.1, lens=A16, table=A16, stride=40, width=40, table_rows=None, starts=A16,
              shared=A16, groups=3, max_shared=2000, max_own=100, rows=40, out=A16, lse=A16, work=None, bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(heads=0), 1), (dict(heads=1025), 1), (dict(latent=128), 1), (dict(rope=32), 1),
    (dict(type=2), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1),
    (dict(ps=48), 1), (dict(ps=1 << 21), 1), (dict(pages=-1), 1), (dict(page=-8), 1), (dict(token=-8), 1),
    (dict(q=None), 1), (dict(cache=None), 1), (dict(out=None), 1), (dict(q_head=-576), 1), (dict(lens=None), 1),
    (dict(table=None), 1), (dict(width=0), 1), (dict(stride=39), 1), (dict(starts=None), 1), (dict(shared=None), 1),
    (dict(groups=0), 1), (dict(groups=-1), 1), (dict(max_shared=-1), 1), (dict(max_own=-1), 1),
    (dict(max_shared=1 << 31), 1), (dict(max_own=(1 << 31) - 64), 1), (dict(rows=1 << 30), 1), (dict(groups=2 ** 31 - 1), 1), (dict(q=A8), 2), (dict(cache=A4), 2),
    (dict(out=A4), 2), (dict(lse=0x10002), 2), (dict(q_row=9220), 2), (dict(token=580), 2), (dict(page=36868), 2),
    (dict(), 6), (dict(work=A16, bytes=100), 6), (dict(work=A4, bytes=1 << 40), 2),
])
def test_attend_shared_refuses(lib, kw, code):
    assert call(lib.dsatopk_attend_shared, SHARED, kw) == code


def test_nothing_to_do_is_no_error(lib):
    none = {k: None for k in ("q", "out", "lse", "lens", "starts", "shared", "table")}
    assert call(lib.dsatopk_attend_shared, SHARED, dict(rows=0, groups=0, **none)) == 0


def test_shared_bytes(lib):
    assert dt.shared_bytes(0, 16, 512, 1, 1000, 10) == 0
    assert dt.shared_bytes(4, 16, 512, 0, 1000, 10) == 0
    assert dt.shared_bytes(4, 16, 512, 1, -1, 10) == 0
    few, many = dt.shared_bytes(4, 16, 512, 1, 100000, 10), dt.shared_bytes(400, 16, 512, 1, 100000, 10)
    assert 0 < few < many and few % 16 == 0
    # a part is the heads of a workgroup; no more of them than the bounds have work for
    assert 0 < dt.shared_bytes(4, 16, 512, 1, 64, 0) < dt.shared_bytes(4, 16, 512, 1, 6400, 0)
    assert dt.shared_bytes(4, 16, 512, 1, 0, 0) > 0
    assert dt.shared_bytes(2 ** 31 - 1, 1024, 512, 2 ** 31 - 1, 2 ** 31 - 65, 2 ** 31 - 65) > 0


def test_binding_refuses_host_tensors_and_gradients():
    n = torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(4, 16, 576, dtype=torch.bfloat16)
    at = (n, torch.zeros(4, 8, dtype=torch.int32), n, n[:3], 512, 0.1)
    with pytest.raises(ValueError, match="device"):
        dt.attend_shared(q, q, *at)
    with pytest.raises(ValueError, match="gradient"):
        dt.attend_shared(q.requires_grad_(), q.detach(), *at)
    with torch.no_grad(), pytest.raises(ValueError, match="device"):
        dt.attend_shared(q, q, *at)


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    dev = "cuda"
    bf = dict(dtype=torch.bfloat16, device=dev)
    q, cache = torch.zeros(4, 16, 576, **bf), torch.zeros(8, 64, 576, **bf)
    lens, table = torch.zeros(4, dtype=torch.int32, device=dev), torch.zeros(4, 8, dtype=torch.int32, device=dev)
    starts = torch.tensor([0, 2, 4], dtype=torch.int32, device=dev)
    shared = torch.zeros(2, dtype=torch.int32, device=dev)

    def refused(*args, error=ValueError, **kw):
        with pytest.raises(error):
            dt.attend_shared(*args, **kw)

    refused(q, cache[..., :512], lens, table, starts, shared, 512, 0.1)
    refused(q, cache.half(), lens, table, starts, shared, 512, 0.1)
    refused(q, cache, lens[:3], table, starts, shared, 512, 0.1)
    refused(q, cache, lens, table[:3], starts, shared, 512, 0.1)
    refused(q, cache, lens, table.long(), starts, shared, 512, 0.1)
    refused(q, cache, lens, table, starts.long(), shared, 512, 0.1)
    refused(q, cache, lens, table, starts, shared[:1], 512, 0.1)
    refused(q, cache, lens, table, starts[:1], shared[:0], 512, 0.1)
    refused(q, cache, lens, table, starts[:0], shared[:0], 512, 0.1)
    refused(q, cache, lens, table, starts.cpu(), shared, 512, 0.1)
    refused(q, cache, lens, table, starts, shared, 512, 0.1, out=torch.zeros(4, 16, 576, **bf))
    refused(q, cache, lens, table, starts, shared, 512, 0.1, lse=torch.zeros(4, 8, device=dev))
    refused(q, cache, lens, table, starts, shared, 448, 0.1, error=dt.DsatopkError)
    refused(q, cache, lens, table, starts, shared, 512, 0.0, error=dt.DsatopkError)
    refused(q, cache, lens, table, starts, shared, 512, 0.1, max_own_len=-1, error=dt.DsatopkError)
    with pytest.raises(TypeError):
        dt.attend_shared(q, cache, lens, table, starts, shared, 512)
    with pytest.raises(ValueError, match="gradient"):
        dt.attend_shared(q, cache.clone().requires_grad_(), lens, table, starts, shared, 512, 0.1)
