"""Cache writes: tensors that are written are refused if their rows share memory,
and taken in any order and with any room between them if they do not."""
import pytest
import torch

from tests import append_plain as plain
from tests.test_serve_append_gpu import TYPES, i32

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_overlapping_rows_are_refused():
    import row_top_selection_amd as dt

    x, n, table = torch.ones(4, 576, device=DEV).bfloat16(), i32([0] * 4), plain.angles(8).to(DEV)
    big = torch.zeros(1 << 20, device=DEV).bfloat16()
    cache, q = big[:2 * 16 * 576].view(2, 16, 576), torch.ones(4, 3, 64, device=DEV).bfloat16()

    def refused(fn, *args, **kw):
        with pytest.raises(ValueError, match="overlap"):
            fn(*args, **kw)

    refused(dt.append_latent, x, big.as_strided((2, 16, 576), (8 * 576, 576, 1)), n, n, table)   # pages
    refused(dt.append_latent, x, big.as_strided((2, 16, 576), (16 * 576, 512, 1)), n, n, table)  # tokens
    refused(dt.append_latent, x, big.as_strided((16, 16, 576), (576, 576, 1)), n, n, table)
    refused(dt.append_latent, x, cache, n, n, table, out=big.as_strided((4, 576), (64, 1)))
    refused(dt.append_latent, x, cache, n, n, table, q_rope=q, q_out=big.as_strided((4, 3, 64), (64, 64, 1)))
    refused(dt.append_latent, x, cache, n, n, table, q_rope=q, q_out=big.as_strided((4, 3, 64), (128, 64, 1)))
    refused(dt.append_latent, x, cache, n, n, table, q_rope=q, q_out=big.as_strided((4, 3, 64), (64, 192, 1)))
    eight, scales = torch.zeros(2, 16, 128, device=DEV).to(TYPES["fp8"]), torch.zeros(64, device=DEV)
    refused(dt.append_index, x[:, :128], eight, n, n, table, key_scales=scales.as_strided((2, 16), (8, 1)))
    iq, w = torch.ones(4, 3, 128, device=DEV).bfloat16(), torch.ones(4, 3, device=DEV)
    refused(dt.append_index, x[:, :128], eight, n, n, table, key_scales=scales[:32].view(2, 16), q=iq, weights=w,
            weights_out=scales.as_strided((4, 3), (2, 1)))


def test_other_orders_and_room_are_taken():
    """Heads before tokens, tokens before pages, rows and planes with room between them, single entries of any stride."""
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(1)
    x, q = torch.randn(4, 576, generator=g, device=DEV).bfloat16(), torch.randn(4, 3, 64, generator=g, device=DEV).bfloat16()
    slots, lens, table = i32([3, 17, 30, 1]), i32([1, 2, 8, 5]), plain.angles(8).to(DEV)
    want_cache = torch.zeros(2, 16, 576, device=DEV).bfloat16()
    want = dt.append_latent(x, want_cache, slots, lens, table, q_rope=q)
    big = torch.zeros(1 << 20, device=DEV).bfloat16()
    for q_out in (torch.zeros(3, 4, 64, device=DEV).bfloat16().transpose(0, 1), big.as_strided((4, 3, 64), (72, 4 * 72, 1)),
                  big.as_strided((4, 3, 64), (4096, 128, 1)), torch.zeros(4, 7, 128, device=DEV).bfloat16()[:, 1::2, 64:]):
        cache = torch.zeros(16, 2, 576, device=DEV).bfloat16().transpose(0, 1)
        got = dt.append_latent(x, cache, slots, lens, table, q_rope=q, q_out=q_out)
        assert got.data_ptr() == q_out.data_ptr() and torch.equal(got, want) and torch.equal(cache, want_cache)
    one = big.as_strided((1, 1, 64), (8, 8, 1))
    assert torch.equal(dt.append_latent(x[:1], want_cache, slots[:1], lens[:1], table, q_rope=q[:1, :1], q_out=one), want[:1, :1])
