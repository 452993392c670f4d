"""What page_maps holds and lets go of."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.as_tensor(np.asarray(v, dtype=np.int32)).cuda()


FIELDS = ("token_starts", "slots", "table_rows", "row_lens", "counts")


def test_outputs_that_are_made_when_asked_for_are_held():
    """Fields of `out` that nobody else holds: all are alive until the call is
    made, so that no two of them are one block."""
    import row_top_selection_amd as dt

    sizes, at = (2, 64, 64, 64, 2), {}

    class Made:
        def __getattr__(self, name):
            t = torch.zeros(sizes[FIELDS.index(name)], dtype=torch.int32, device="cuda")
            at[name] = t.data_ptr()
            return t

    out = Made()
    got = dt.page_maps(i32([40]), i32([[3]]), 64, i32([1]), 64, new_lens=i32([40]), out=out)
    torch.cuda.synchronize()
    assert got is out and len(set(at.values())) == 5


def test_a_field_that_does_not_fit_is_refused():
    import row_top_selection_amd as dt

    args = (i32([40]), i32([[3]]), 64, i32([1]), 64)
    out = dt.page_maps(*args)
    for name in FIELDS:
        with pytest.raises(ValueError, match=name):
            dt.page_maps(*args, out=out._replace(**{name: i32([0] * 9)}))
        with pytest.raises(ValueError, match=name):
            dt.page_maps(*args, out=out._replace(**{name: None}))
    with pytest.raises(AttributeError):
        dt.page_maps(*args, out=out[:3])


def test_outputs_of_a_failed_allocation_are_given_back():
    import row_top_selection_amd as dt

    lens, table, free = i32([4]), i32([[0]]), i32([1])
    dt.page_maps(lens, table, 64, free, 4)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    room = torch.cuda.memory_reserved() + (3 << 30)
    torch.cuda.set_per_process_memory_fraction(room / torch.cuda.get_device_properties(0).total_memory)
    try:
        with pytest.raises(RuntimeError, match="out of memory"):
            dt.page_maps(lens, table, 64, free, 1 << 29)  # outputs of 2 GB: the first fits
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert torch.cuda.memory_allocated() == before
    torch.cuda.empty_cache()


def test_out_of_memory_is_torchs_error():
    import row_top_selection_amd as dt

    lens, table, free = i32([4]), i32([[0]]), i32([1])
    torch.cuda.empty_cache()
    room = torch.cuda.memory_reserved() + (1 << 30)
    torch.cuda.set_per_process_memory_fraction(room / torch.cuda.get_device_properties(0).total_memory)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            dt.page_maps(lens, table, 64, free, 1 << 29)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
