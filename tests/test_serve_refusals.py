"""What the serving operators refuse: the C calls before any HIP call (fake
pointers, no GPU), and the binding before it looks at a pointer."""
import ctypes
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


MAPS = dict(lens=A16, new=A16, n=4, table=A16, stride=8, width=8, ps=64, free=A16, num_free=9,
            tokens=16, starts=A16, slots=A16, rows=A16, row_lens=A16, counts=A16, stream=None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(num_free=-1), dict(tokens=-1), dict(width=-1), dict(stride=7), dict(ps=0),
    dict(ps=48), dict(ps=1 << 21), dict(ps=-64), dict(lens=None), dict(table=None), dict(free=None),
    dict(starts=None), dict(slots=None), dict(rows=None), dict(row_lens=None), dict(counts=None),
])
def test_page_maps_refuses(lib, kw):
    assert call(lib.dsatopk_page_maps, MAPS, kw) == 1


PAGED = dict(q=A16, q_row=8192, q_head=128, w=A16, w_row=64, keys=A16, pages=10, page=8192, token=128,
             scales=A16, scale_page=64, type=0, heads=64, dim=128, lens=A16, table=A16, stride=8,
             width=8, ps=64, table_rows=None, rows=4, out=A16, out_stride=512, columns=512,
             stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(heads=0), 1), (dict(heads=129), 1), (dict(dim=96), 1),
    (dict(type=3), 1), (dict(type=-1), 1), (dict(columns=-1), 1), (dict(columns=(1 << 30) + 1, out_stride=1 << 31), 1),
    (dict(out_stride=511), 1), (dict(q=None), 1), (dict(w=None), 1), (dict(keys=None), 1),
    (dict(lens=None), 1), (dict(out=None), 1), (dict(table=None), 1), (dict(width=0), 1),
    (dict(stride=7), 1), (dict(ps=48), 1), (dict(ps=1 << 21), 1), (dict(pages=-1), 1),
    (dict(q_row=-8), 1), (dict(q=A8), 2), (dict(keys=A4), 2), (dict(q_row=8196), 2),
    (dict(q_head=132), 2), (dict(token=130), 2), (dict(page=8196), 2), (dict(out=0x10002), 2),
    (dict(w=0x10001), 2), (dict(type=2, q_head=136), 2), (dict(type=2, token=8), 2),
])
def test_scores_paged_refuses(lib, kw, code):
    assert call(lib.dsatopk_scores_paged, PAGED, kw) == code


RAGGED = dict(q=A16, q_row=8192, q_head=128, w=A16, w_row=64, keys=A16, n=500, token=128, scales=None,
              type=0, heads=64, dim=128, lens=A16, starts=A16, rows=4, out=A16, out_stride=512,
              columns=500, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(heads=200), 1), (dict(dim=32), 1), (dict(starts=None), 1),
    (dict(n=-1), 1), (dict(lens=None), 1), (dict(columns=513), 1), (dict(q=A8), 2),
    (dict(token=12), 2),
])
def test_scores_ragged_refuses(lib, kw, code):
    assert call(lib.dsatopk_scores_ragged, RAGGED, kw) == code


SELECTED = dict(q=A16, q_row=9216, q_head=576, cache=A16, pages=10, page=36864, token=576, ps=64,
                type=0, heads=16, latent=512, rope=64, scale=0.1, slots=A16, stride=2048, k=2048,
                rows=400, out=A16, lse=A16, work=None, bytes=0, stream=None)

ATTEND_BAD = [
    (dict(rows=-1), 1), (dict(heads=0), 1), (dict(heads=1025), 1), (dict(latent=128), 1),
    (dict(rope=32), 1), (dict(type=2), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=math.inf), 1), (dict(scale=math.nan), 1), (dict(ps=48), 1), (dict(pages=-1), 1),
    (dict(q=None), 1), (dict(cache=None), 1), (dict(out=None), 1), (dict(q_head=-576), 1),
    (dict(q=A8), 2), (dict(cache=A4), 2), (dict(out=A4), 2), (dict(lse=0x10002), 2),
    (dict(q_row=9220), 2), (dict(token=580), 2), (dict(page=36868), 2), (dict(rows=4), 6),
    (dict(rows=4, work=A16, bytes=100), 6), (dict(rows=4, work=A4, bytes=1 << 40), 2),
]


@pytest.mark.parametrize("kw,code", ATTEND_BAD + [
    (dict(k=-1), 1), (dict(stride=2047), 1), (dict(slots=None), 1)])
def test_attend_selected_refuses(lib, kw, code):
    assert call(lib.dsatopk_attend_selected, SELECTED, kw) == code


ATTEND_PAGED = dict(q=A16, q_row=9216, q_head=576, cache=A16, pages=10, page=36864, token=576, ps=64,
                    type=0, heads=16, latent=512, rope=64, scale=0.1, lens=A16, table=A16, stride=40,
                    width=40, table_rows=None, longest=2048, rows=400, out=A16, lse=A16, work=None,
                    bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", ATTEND_BAD + [
    (dict(lens=None), 1), (dict(table=None), 1), (dict(width=0), 1), (dict(stride=39), 1),
    (dict(longest=-1), 1), (dict(longest=1 << 31), 1)])
def test_attend_paged_refuses(lib, kw, code):
    assert call(lib.dsatopk_attend_paged, ATTEND_PAGED, kw) == code


EXPANDED = dict(q=A16, q_row=1536, q_head=192, k=A16, k_row=2048, k_head=256, v=A16, v_row=2048,
                v_head=256, rope=A16, rope_row=64, type=0, heads=8, nope=128, rope_dim=64, value=128,
                scale=0.1, causal=1, qs=A16, ks=A16, requests=2, queries=100, keys=200, longest=60,
                out=A16, lse=A16, work=None, bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(requests=-1), 1), (dict(queries=-1), 1), (dict(keys=-1), 1), (dict(longest=-1), 1),
    (dict(heads=0), 1), (dict(heads=1025), 1), (dict(nope=64), 1), (dict(rope_dim=128), 1),
    (dict(value=64), 1), (dict(type=2), 1), (dict(scale=0.0), 1), (dict(scale=math.nan), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(rope=None), 1), (dict(out=None), 1),
    (dict(qs=None), 1), (dict(ks=None), 1), (dict(k_row=-8), 1), (dict(q=A8), 2), (dict(k=A4), 2),
    (dict(v=A8), 2), (dict(rope=A8), 2), (dict(out=A4), 2), (dict(lse=0x10001), 2),
    (dict(q_head=196), 2), (dict(k_row=2052), 2), (dict(v_head=260), 2), (dict(rope_row=68), 2),
    (dict(k_row=1 << 28), 1), (dict(keys=20000), 6), (dict(keys=20000, work=A16, bytes=64), 6),
    (dict(keys=20000, work=A4, bytes=1 << 40), 2),
])
def test_attend_expanded_refuses(lib, kw, code):
    assert call(lib.dsatopk_attend_expanded, EXPANDED, kw) == code


def test_nothing_to_do_is_no_error(lib):
    none = {k: None for k in ("q", "out", "lse")}
    assert call(lib.dsatopk_scores_paged, PAGED, dict(rows=0, q=None, keys=None, out=None)) == 0
    assert call(lib.dsatopk_scores_ragged, RAGGED, dict(rows=0, q=None, keys=None, out=None)) == 0
    assert call(lib.dsatopk_attend_selected, SELECTED, dict(rows=0, **none)) == 0
    assert call(lib.dsatopk_attend_paged, ATTEND_PAGED, dict(rows=0, **none)) == 0
    assert call(lib.dsatopk_attend_expanded, EXPANDED, dict(queries=0, **none)) == 0
    assert call(lib.dsatopk_attend_expanded, EXPANDED, dict(requests=0, **none)) == 0


def test_attend_bytes(lib):
    assert dt.attend_bytes(0, 16, 512, 2048) == 0
    assert dt.attend_bytes(10 ** 6, 128, 512, 2048) == 0
    few = dt.attend_bytes(1, 16, 512, 131072)
    assert few >= 16 * (512 + 2) * 4 and few % 4 == 0
    assert dt.attend_bytes(1, 16, 512, 64) == 0  # one tile: nothing to split


def test_expanded_bytes(lib):
    assert dt.expanded_bytes(4, 16, 4096, 65536, 1024) == 0  # fills the card
    assert dt.expanded_bytes(2, 8, 100, 200, 60) == 0        # too few keys to split
    assert dt.expanded_bytes(0, 8, 100, 200, 60) == 0
    few = dt.expanded_bytes(2, 1, 300, 10000, 164)
    assert few >= 2 * 300 * 130 * 4 and few % (300 * 130 * 4) == 0


def test_status_string(lib):
    assert b"workspace" in lib.dsatopk_status_string(6)


def test_library_sources_declare_what_they_export(lib):
    for name in dt.EXPORTS:
        assert isinstance(getattr(lib, name), ctypes._CFuncPtr)


# The binding's own checks come before any launch, so they are seen without a
# GPU: host tensors are the first thing it refuses.
I32 = dict(dtype=torch.int32)


def test_binding_refuses_host_tensors():
    lens, table = torch.zeros(4, **I32), torch.zeros(4, 8, **I32)
    q3 = torch.zeros(4, 16, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        dt.page_maps(lens, table, 64, lens, 4)
    with pytest.raises(ValueError, match="device"):
        dt.scores_paged(torch.zeros(4, 64, 128), torch.zeros(4, 64), torch.zeros(8, 64, 128), lens, table)
    with pytest.raises(ValueError, match="device"):
        dt.scores_ragged(torch.zeros(4, 64, 128), torch.zeros(4, 64), torch.zeros(80, 128), lens, lens)
    with pytest.raises(ValueError, match="device"):
        dt.attend_selected(q3, q3, table, 512, 0.1)
    with pytest.raises(ValueError, match="device"):
        dt.attend_paged(q3, q3, lens, table, 512, 0.1)
    with pytest.raises(ValueError, match="device"):
        dt.attend_expanded(torch.zeros(4, 2, 192), *(torch.zeros(4, 2, 128),) * 2, torch.zeros(4, 64), lens, lens, 4, 0.1)


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    dev = "cuda"
    lens, table = torch.zeros(4, device=dev, **I32), torch.zeros(4, 8, device=dev, **I32)
    bf = dict(dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):
        dt.page_maps(lens.long(), table, 64, lens, 4)
    with pytest.raises(ValueError):
        dt.page_maps(lens, table[:3], 64, lens, 4)
    with pytest.raises(ValueError):
        dt.page_maps(lens, table.t(), 64, lens, 4)
    with pytest.raises(ValueError):
        dt.page_maps(lens, table, 64, lens, -1)
    with pytest.raises(dt.DsatopkError):
        dt.page_maps(lens, table, 48, lens, 4)
    q, w, keys = torch.zeros(4, 64, 128, **bf), torch.zeros(4, 64, device=dev), torch.zeros(8, 64, 128, **bf)
    with pytest.raises(ValueError):
        dt.scores_paged(q.float(), w, keys.float(), lens, table)
    with pytest.raises(ValueError):
        dt.scores_paged(q, w.half(), keys, lens, table)
    with pytest.raises(ValueError):
        dt.scores_paged(q, w, keys.half(), lens, table)
    with pytest.raises(ValueError):
        dt.scores_paged(q, w, keys, lens[:3], table)
    with pytest.raises(ValueError):
        dt.scores_paged(q, w, keys, lens, table[:2])
    with pytest.raises(ValueError):
        dt.scores_paged(q, w, keys, lens, table, key_scales=torch.zeros(8, 32, device=dev))
    with pytest.raises(ValueError):
        dt.scores_paged(q, w, keys, lens, table, out=torch.zeros(3, 512, device=dev))
    with pytest.raises(ValueError):
        dt.scores_ragged(q, w, keys[0], lens, None)
    with pytest.raises(dt.DsatopkError):
        dt.scores_paged(torch.zeros(4, 64, 96, **bf), w, torch.zeros(8, 64, 96, **bf), lens, table)
    qa, cache = torch.zeros(4, 16, 576, **bf), torch.zeros(8, 64, 576, **bf)
    with pytest.raises(ValueError):
        dt.attend_selected(qa, cache[..., :512], table, 512, 0.1)
    with pytest.raises(ValueError):
        dt.attend_selected(qa, cache, table.float(), 512, 0.1)
    with pytest.raises(ValueError):
        dt.attend_selected(qa, cache, table, 512, 0.1, out=torch.zeros(4, 16, 576, **bf))
    with pytest.raises(dt.DsatopkError):
        dt.attend_selected(qa, cache, table, 448, 0.1)
    with pytest.raises(dt.DsatopkError):
        dt.attend_paged(qa, cache, lens, table, 512, -0.1)
    with pytest.raises(dt.DsatopkError) as e:
        dt.attend_paged(qa, cache, lens, table, 512, 0.1, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    assert e.value.status == 6
    qe, kv, rope = torch.zeros(4, 2, 192, **bf), torch.zeros(4, 2, 128, **bf), torch.zeros(4, 64, **bf)
    starts = torch.tensor([0, 4], device=dev, **I32)
    with pytest.raises(ValueError):
        dt.attend_expanded(qe, kv, kv[:3], rope, starts, starts, 4, 0.1)
    with pytest.raises(ValueError):
        dt.attend_expanded(qe, kv, kv, rope.half(), starts, starts, 4, 0.1)
    with pytest.raises(ValueError):
        dt.attend_expanded(qe[..., :128], kv, kv, rope, starts, starts, 4, 0.1)
    with pytest.raises(ValueError):
        dt.attend_expanded(qe, kv, kv, rope, starts, starts[:1], 4, 0.1)
