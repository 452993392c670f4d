"""What the cache writes refuse: the C calls before any HIP call (fake
pointers, no GPU), and the binding before it looks at a pointer."""
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


LATENT = dict(x=A16, x_row=576, slots=A16, lens=A16, n=4, angles=A16, angle_row=64, positions=100, near=1,
              weight=A16, eps=1e-6, type=0, latent=512, rope=64, cache=A16, pages=10, page=36864, token=576,
              ps=64, out=A16, out_row=576, q=A16, q_row=1536, q_head=192, q_out=A16, qo_row=1536, qo_head=192,
              heads=8, stream=None)

TOKENS_BAD = [
    (dict(n=-1), 1), (dict(n=(1 << 30) + 1), 1), (dict(positions=-1), 1), (dict(rope=32), 1),
    (dict(angle_row=63), 1), (dict(eps=-1e-6), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1),
    (dict(type=2), 1), (dict(type=-1), 1), (dict(pages=-1), 1), (dict(page=-64), 1), (dict(token=-64), 1),
    (dict(ps=0), 1), (dict(ps=48), 1), (dict(ps=1 << 21), 1), (dict(heads=-1), 1), (dict(x=None), 1),
    (dict(slots=None), 1), (dict(lens=None), 1), (dict(angles=None), 1), (dict(cache=None), 1),
    (dict(q=None), 1), (dict(q_out=None), 1), (dict(x_row=-8), 1), (dict(q_row=-8), 1), (dict(qo_head=-8), 1),
    (dict(x=A8), 2), (dict(angles=A8), 2), (dict(angle_row=66), 2), (dict(weight=A4), 2), (dict(cache=A8), 2),
    (dict(q=A8), 2), (dict(q_out=A8), 2), (dict(x_row=580), 2), (dict(page=36868), 2), (dict(token=580), 2),
    (dict(q_row=1540), 2), (dict(q_head=196), 2), (dict(qo_row=1540), 2), (dict(qo_head=196), 2),
]


@pytest.mark.parametrize("kw,code", TOKENS_BAD + [
    (dict(latent=128), 1), (dict(heads=1025), 1), (dict(out=A8), 2), (dict(out_row=580), 2), (dict(out_row=-8), 1)])
def test_append_latent_refuses(lib, kw, code):
    assert call(lib.dsatopk_append_latent, LATENT, kw) == code


INDEX = dict(x=A16, x_row=128, slots=A16, lens=A16, n=4, angles=A16, angle_row=64, positions=100, rope=64, near=0,
             weight=A16, bias=A16, eps=1e-6, type=0, dim=128, cache=A16, to=2, pages=10, page=8192, token=128,
             ps=64, scales=A16, scale_page=64, q=A16, q_row=1024, q_head=128, q_out=A16, qo_row=1024,
             qo_head=128, w=A16, w_row=8, wo=A16, wo_row=8, heads=8, stream=None)


@pytest.mark.parametrize("kw,code", TOKENS_BAD + [
    (dict(dim=96), 1), (dict(heads=129), 1), (dict(to=1), 1), (dict(to=3), 1), (dict(bias=None), 1),
    (dict(weight=None), 1), (dict(scales=None), 1), (dict(w=None), 1), (dict(wo=None), 1),
    (dict(scale_page=-1), 1), (dict(w_row=-1), 1), (dict(wo_row=-1), 1), (dict(bias=A8), 2),
    (dict(scales=0x10002), 2), (dict(w=0x10001), 2), (dict(wo=0x10002), 2), (dict(token=136), 2),
    (dict(page=8200), 2), (dict(qo_head=136), 2)])
def test_append_index_refuses(lib, kw, code):
    assert call(lib.dsatopk_append_index, INDEX, kw) == code


def test_nothing_to_do_is_no_error(lib):
    none = {k: None for k in ("x", "slots", "lens", "cache", "q", "q_out")}
    assert call(lib.dsatopk_append_latent, LATENT, dict(n=0, **none)) == 0
    assert call(lib.dsatopk_append_index, INDEX, dict(n=0, **none)) == 0


I32 = dict(dtype=torch.int32)


def test_binding_refuses_host_tensors_and_gradients():
    x, n = torch.zeros(4, 576, dtype=torch.bfloat16), torch.zeros(4, **I32)
    for fn, last in ((dt.append_latent, 576), (dt.append_index, 128)):
        cache = torch.zeros(2, 16, last, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="device"):
            fn(x[:, :last], cache, n, n, torch.zeros(8, 64))
        with pytest.raises(ValueError, match="gradient"):
            fn(x[:, :last].clone().requires_grad_(), cache, n, n, torch.zeros(8, 64))


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    dev = "cuda"
    bf = dict(dtype=torch.bfloat16, device=dev)
    x, cache, n = torch.zeros(4, 576, **bf), torch.zeros(2, 16, 576, **bf), torch.zeros(4, device=dev, **I32)
    table, q = torch.zeros(8, 64, device=dev), torch.zeros(4, 3, 64, **bf)

    def refused(fn, *args, error=ValueError, **kw):
        with pytest.raises(error):
            fn(*args, **kw)

    f = dt.append_latent
    refused(f, x.float(), cache.float(), n, n, table)
    refused(f, x.to(torch.float8_e4m3fn), cache.to(torch.float8_e4m3fn), n, n, table)
    refused(f, x, cache.half(), n, n, table)
    refused(f, x, cache[..., :512], n, n, table)
    refused(f, x, cache[:1].expand(2, 16, 576), n, n, table)
    refused(f, x, cache, n[:3], n, table)
    refused(f, x, cache, n.long(), n, table)
    refused(f, x, cache, n, n, table.half())
    refused(f, x, cache, n, n, table[:, :32])
    refused(f, x, cache, n, n, table, weight=torch.ones(512, **bf))
    refused(f, x, cache, n, n, table, weight=torch.ones(576, device=dev))
    refused(f, x, cache, n, n, table, q_rope=q[:3])
    refused(f, x, cache, n, n, table, q_rope=q.half())
    refused(f, x, cache, n, n, table, q_rope=q[..., :32])
    refused(f, x, cache, n, n, table, q_rope=q, q_out=q[:, :2])
    refused(f, x, cache, n, n, table, q_out=q)
    refused(f, x, cache, n, n, table, q_rope=q, q_out=q[:, :1].expand(4, 3, 64))
    refused(f, x, cache, n, n, table, out=x.half())
    refused(f, x, cache, n, n, table, out=x[:1].expand(4, 576))
    refused(f, x, cache.cpu(), n, n, table)
    refused(f, x, cache, n, n, table, eps=-1.0, error=dt.DsatopkError)
    refused(f, x[:, :448], torch.zeros(2, 16, 448, **bf), n, n, table, error=dt.DsatopkError)
    refused(f, x, torch.zeros(2, 12, 576, **bf), n, n, table, error=dt.DsatopkError)
    refused(f, x, cache, n, n, table, q_rope=torch.zeros(4, 3, 70, **bf)[..., 6:], error=dt.DsatopkError)

    f, k, iq, w = dt.append_index, x[:, :128], torch.zeros(4, 3, 128, **bf), torch.zeros(4, 3, device=dev)
    keys, eight, scales = torch.zeros(2, 16, 128, **bf), torch.zeros(2, 16, 128, device=dev).to(torch.float8_e4m3fn), torch.zeros(2, 16, device=dev)
    refused(f, k, keys.half(), n, n, table)
    refused(f, k, keys[..., :64], n, n, table)
    refused(f, k, keys, n, n, table, key_scales=scales)
    refused(f, k, eight, n, n, table)
    refused(f, k, eight, n, n, table, key_scales=scales[:1])
    refused(f, k, eight, n, n, table, key_scales=scales.half())
    refused(f, k, eight, n, n, table, key_scales=scales[:1].expand(2, 16)[:, :1].expand(2, 16))
    refused(f, k, keys, n, n, table, weight=torch.ones(128, device=dev))
    refused(f, k, keys, n, n, table, weight=torch.ones(128, device=dev), bias=torch.ones(64, device=dev))
    refused(f, k, keys, n, n, table, q=iq, weights=w)
    refused(f, k, eight, n, n, table, key_scales=scales, q=iq)
    refused(f, k, eight, n, n, table, key_scales=scales, weights=w)
    refused(f, k, eight, n, n, table, key_scales=scales, q=iq, weights=w[:, :2])
    refused(f, k, eight, n, n, table, key_scales=scales, q=iq, weights=w, q_out=iq)
    refused(f, k, eight, n, n, table, key_scales=scales, q=iq, weights=w, weights_out=w.half())
    refused(f, k, keys, n, n, table, q_out=iq)
    refused(f, k, keys, n, n, table, q=iq[..., :64])
    refused(f, x[:, :96], torch.zeros(2, 16, 96, **bf), n, n, table, error=dt.DsatopkError)
