"""Cache writes: arguments that a call has no use for are not looked at."""
import pytest
import torch

import row_top_selection_amd as dt
from tests.test_serve_append_refusals import INDEX, LATENT, call

NONE = dict(x=None, slots=None, lens=None, cache=None)  # without tokens, no pointer is used
QUERIES = dict(heads=0, q=0x10001, q_row=-5, q_head=3, q_out=0x10002, qo_row=-7, qo_head=1)


@pytest.fixture(scope="module")
def lib():
    return dt.lib()


def test_without_tokens(lib):
    assert call(lib.dsatopk_append_latent, LATENT, dict(n=0, **NONE, **QUERIES)) == 0
    assert call(lib.dsatopk_append_latent, LATENT, dict(n=0, **NONE, out=None, out_row=-3)) == 0
    none = dict(w=0x10001, w_row=-1, wo=0x10002, wo_row=-1)
    assert call(lib.dsatopk_append_index, INDEX, dict(n=0, **NONE, **QUERIES, **none)) == 0
    sixteen = dict(to=0, scales=0x10001, scale_page=-9)
    assert call(lib.dsatopk_append_index, INDEX, dict(n=0, **NONE, **none, **sixteen)) == 0
    # and what it has a use for still is
    assert call(lib.dsatopk_append_latent, LATENT, dict(n=0, **NONE, out_row=-3)) == 1
    assert call(lib.dsatopk_append_index, INDEX, dict(n=0, **NONE, w_row=-1)) == 1
    assert call(lib.dsatopk_append_index, INDEX, dict(n=0, **NONE, scale_page=-9)) == 1


@pytest.mark.gpu
def test_with_tokens(lib):
    dev = "cuda"
    x = torch.randn(5, 576, device=dev).bfloat16()
    slots, lens = torch.arange(5, device=dev, dtype=torch.int32), torch.ones(5, device=dev, dtype=torch.int32)
    angles = torch.cat([torch.ones(4, 32, device=dev), torch.zeros(4, 32, device=dev)], 1)
    cache, keys = torch.zeros(2, 16, 576, device=dev).bfloat16(), torch.zeros(2, 16, 128, device=dev).bfloat16()
    tokens = dict(n=5, slots=slots.data_ptr(), lens=lens.data_ptr(), x=x.data_ptr(), x_row=576, angles=angles.data_ptr(), positions=4,
                  weight=None, pages=2, ps=16, stream=torch.cuda.current_stream().cuda_stream)
    assert call(lib.dsatopk_append_latent, LATENT, dict(tokens, cache=cache.data_ptr(), page=16 * 576, out=None, out_row=3, **QUERIES)) == 0
    assert call(lib.dsatopk_append_index, INDEX, dict(tokens, bias=None, cache=keys.data_ptr(), page=16 * 128, to=0, scales=0x10001, scale_page=-9,
                                                      w=0x10001, w_row=-1, wo=0x10002, wo_row=-1, **QUERIES)) == 0
    torch.cuda.synchronize()
    assert torch.equal(cache.view(-1, 576)[:5], x) and torch.equal(keys.view(-1, 128)[:5], x[:, :128])
