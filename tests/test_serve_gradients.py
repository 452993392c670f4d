"""The serving operators compute no gradients and say so, instead of giving
results without history."""
import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import row_top_selection_amd as dt


def calls(dev):
    """(name, call with the float inputs, those inputs) of every call that takes floats."""
    def t(*shape):
        return torch.zeros(*shape, dtype=torch.bfloat16, device=dev)

    def i32(v):
        return torch.as_tensor(np.asarray(v, dtype=np.int32)).to(dev)

    lens, table, starts = i32([4] * 3), i32([[0]] * 3), i32([0, 3])
    return [
        (lambda q, w, k, s: dt.scores_paged(q, w, k, lens, table, key_scales=s),
         [t(3, 64, 128), t(3, 64).float(), t(2, 16, 128), torch.ones(2, 16, device=dev)]),
        (lambda q, w, k, s, o: dt.scores_ragged(q, w, k, lens, lens, key_scales=s, out=o),
         [t(3, 64, 128), t(3, 64).float(), t(40, 128), torch.ones(40, device=dev), torch.zeros(3, 40, device=dev)]),
        (lambda q, c, o, l: dt.attend_selected(q, c, i32([[0]] * 3), 512, 0.1, out=o, lse=l),
         [t(3, 16, 576), t(2, 16, 576), t(3, 16, 512), torch.zeros(3, 16, device=dev)]),
        (lambda q, c: dt.attend_paged(q, c, lens, table, 512, 0.1), [t(3, 16, 576), t(2, 16, 576)]),
        (lambda q, k, v, r: dt.attend_expanded(q, k, v, r, starts, starts, 3, 0.1),
         [t(3, 2, 192), t(3, 2, 128), t(3, 2, 128), t(3, 64)]),
    ]


# The refusal comes before any look at where a tensor lies: the CPU shows it.
# There is always a first tensor, a host tensor, that is refused next.
@pytest.mark.parametrize("n", range(5))
def test_a_first_input_that_requires_gradients_is_refused(n):
    call, inputs = calls("cpu")[n]
    inputs[0] = inputs[0].requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        call(*inputs)
    with torch.no_grad(), pytest.raises(ValueError, match="device"):
        call(*inputs)
    with torch.inference_mode(), pytest.raises(ValueError, match="device"):
        call(*inputs)
    with pytest.raises(ValueError, match="device"):
        call(inputs[0].detach(), *inputs[1:])


@pytest.mark.parametrize("n", range(5))
def test_a_first_input_with_a_tangent_is_refused(n):
    call, inputs = calls("cpu")[n]
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(inputs[0], torch.ones_like(inputs[0]))
        with pytest.raises(ValueError, match="gradient"):
            call(dual, *inputs[1:])
        with torch.no_grad(), pytest.raises(ValueError, match="gradient"):
            call(dual, *inputs[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("n", range(5))
def test_every_input_that_requires_gradients_is_refused(n):
    call, inputs = calls("cuda")[n]
    call(*inputs)
    for i, x in enumerate(inputs):
        some = list(inputs)
        some[i] = x.clone().requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            call(*some)
        with torch.no_grad():
            got = call(*some)
        assert not any(t.requires_grad for t in (got if isinstance(got, tuple) else (got,)) if t is not some[i])
        some[i] = x.clone() * torch.ones((), device="cuda", dtype=x.dtype, requires_grad=True)  # not a leaf
        with pytest.raises(ValueError, match="gradient"):
            call(*some)
