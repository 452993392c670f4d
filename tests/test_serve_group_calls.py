"""The cache writes and the attention behind shared tokens or keys: gradients are
refused, a given stream's memory is taken, and two calls go on at once."""
import threading

import numpy as np
import pytest
import torch

import row_top_selection_amd as dt

SCALE = 192 ** -0.5


def calls(dev):
    """(call with the float inputs, those inputs) of every call."""
    def t(*shape):
        return torch.zeros(*shape, dtype=torch.bfloat16, device=dev)

    def f(*shape):
        return torch.ones(*shape, device=dev)

    def i32(v):
        return torch.as_tensor(np.asarray(v, dtype=np.int32)).to(dev)

    lens, table, starts, one = i32([4] * 3), i32([[0]] * 3), i32([0, 3]), i32([1])
    return [
        (lambda x, c, a, w, q, o, p: dt.append_latent(x, c, lens, lens, a, weight=w, q_rope=q, q_out=o, out=p),
         [t(3, 576), t(2, 16, 576), f(8, 64), f(512), t(3, 2, 64), t(3, 2, 64), t(3, 576)]),
        (lambda x, c, a, w, b, q: dt.append_index(x, c, lens, lens, a, weight=w, bias=b, q=q),
         [t(3, 128), t(2, 16, 128), f(8, 64), f(128), f(128), t(3, 2, 128)]),
        (lambda q, c, o, l: dt.attend_shared(q, c, lens, table, starts, one, 512, SCALE, out=o, lse=l),
         [t(3, 16, 576), t(2, 16, 576), t(3, 16, 512), f(3, 16)]),
        (lambda q, k, v, r, o, l: dt.attend_expanded_shared(q, k, v, r, starts, starts, one, one, SCALE, out=o, lse=l),
         [t(3, 2, 192), t(4, 2, 128), t(4, 2, 128), t(4, 64), t(3, 2, 128), f(3, 2)]),
    ]


@pytest.mark.parametrize("n", range(4))
def test_a_first_input_that_requires_gradients_is_refused(n):
    call, inputs = calls("cpu")[n]
    inputs[0].requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        call(*inputs)
    with torch.no_grad(), pytest.raises(ValueError, match="device"):
        call(*inputs)


@pytest.mark.gpu
@pytest.mark.parametrize("n", range(4))
def test_every_input_that_requires_gradients_is_refused(n):
    call, inputs = calls("cuda")[n]
    call(*inputs)
    for i in range(len(inputs)):
        with pytest.raises(ValueError, match="gradient"):
            call(*inputs[:i], inputs[i].detach().clone().requires_grad_(), *inputs[i + 1:])
        with torch.no_grad():
            call(*inputs[:i], inputs[i].detach().clone().requires_grad_(), *inputs[i + 1:])
    torch.cuda.synchronize()


def big(g):
    """(call, bytes of its workspace) of the two that take one."""
    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    def i32(v):
        return torch.as_tensor(np.asarray(v, dtype=np.int32)).cuda()

    q, cache = randn(24, 16, 576), randn(64, 64, 576)
    table = torch.randint(0, 64, (24, 32), generator=g, device="cuda").to(torch.int32)
    lens, starts, shared = i32(np.arange(24) * 7 + 1500), i32([0, 15, 24]), i32([1400, 1999])
    p, k, v, rope = randn(300, 4, 192), randn(9000, 4, 128), randn(9000, 4, 128), randn(9000, 64)
    qs, ks, first, front = i32([0, 120, 300]), i32([8000, 8120, 8300]), i32([0, 0]), i32([8000, 8000])
    return [(lambda **kw: dt.attend_shared(q, cache, lens, table, starts, shared, 512, SCALE, **kw),
             dt.shared_bytes(24, 16, 512, 2, 32 * 64, 32 * 64)),
            (lambda **kw: dt.attend_expanded_shared(p, k, v, rope, qs, ks, first, front, SCALE, **kw),
             dt.expanded_shared_bytes(4, 300, 9000))]


@pytest.mark.gpu
@pytest.mark.parametrize("n", range(2))
@pytest.mark.parametrize("by_handle", [False, True])
def test_memory_is_of_the_given_stream(n, by_handle):
    from tests.test_serve_streams_gpu import owner, segments

    call, room = big(torch.Generator("cuda").manual_seed(1))[n]
    want = call()
    before, side = torch.cuda.current_stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    theirs = sum(segments(side).values())
    side.wait_stream(before)
    out = call(stream=side.cuda_stream if by_handle else side)
    assert torch.cuda.current_stream() == before
    torch.cuda.synchronize()
    assert room > 0 and all(owner(t) == side.cuda_stream for t in out)
    assert sum(segments(side).values()) - theirs >= room
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
@pytest.mark.parametrize("n", range(2))
def test_two_calls_at_once(n):
    """Two threads on streams of their own, each with workspaces that its calls allocate."""
    call, _ = big(torch.Generator("cuda").manual_seed(2))[n]
    want = call()
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = call()
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    wrong.append(got)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
