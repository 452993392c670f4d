"""Serving operators on a stream that is given to the call, while the current
stream is another: whose memory a call takes, and its results."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
SCALE = 192 ** -0.5


def i32(v):
    return torch.as_tensor(np.asarray(v, dtype=np.int32)).to(DEV)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def selected(g):
    import row_top_selection_amd as dt

    q, cache = randn(g, 8, 128, 576), randn(g, 64, 64, 576)
    slots = torch.randint(0, 64 * 64, (8, 2048), generator=g, device=DEV).to(torch.int32)
    return lambda **kw: dt.attend_selected(q, cache, slots, 512, SCALE, **kw), dt.attend_bytes(8, 128, 512, 2048)


def paged(g):
    import row_top_selection_amd as dt

    q, cache = randn(g, 8, 128, 576), randn(g, 64, 64, 576)
    table = torch.randint(0, 64, (8, 2048), generator=g, device=DEV).to(torch.int32)
    lens = i32([4000, 1, 70, 0, 3000, 2500, 9, 3333])
    return (lambda **kw: dt.attend_paged(q, cache, lens, table, 512, SCALE, **kw),
            dt.attend_bytes(8, 128, 512, 2048 * 64))


def expanded(g):
    import row_top_selection_amd as dt

    q, k, v, rope = randn(g, 256, 4, 192), randn(g, 20000, 4, 128), randn(g, 20000, 4, 128), randn(g, 20000, 64)
    qs, ks = i32([0, 256]), i32([0, 20000])
    return (lambda **kw: dt.attend_expanded(q, k, v, rope, qs, ks, 256, SCALE, **kw),
            dt.expanded_bytes(1, 4, 256, 20000, 256))


def scores(g):
    import row_top_selection_amd as dt

    q, w, keys = randn(g, 70, 64, 128), torch.rand(70, 64, generator=g, device=DEV), randn(g, 5000, 128)
    lens, starts = i32([5000] * 70), i32([0] * 70)  # all columns: others would not be written
    return lambda **kw: dt.scores_ragged(q, w, keys, lens, starts, **kw), 0


def scores_of_pages(g):
    import row_top_selection_amd as dt

    q, w, keys = randn(g, 9, 64, 128), torch.rand(9, 64, generator=g, device=DEV), randn(g, 40, 64, 128)
    table, lens = i32(np.arange(9 * 32).reshape(9, 32) % 40), i32([2048] * 9)
    return lambda **kw: dt.scores_paged(q, w, keys, lens, table, **kw), 0


def maps(g):
    import row_top_selection_amd as dt

    lens, free, table = i32(np.arange(1, 300)), i32(np.arange(5000)), i32(np.zeros((299, 20)))
    return lambda **kw: tuple(dt.page_maps(lens, table, 16, free, 299 * 150, new_lens=lens, **kw)), 0


CALLS = [selected, paged, expanded, scores, scores_of_pages, maps]


def as_tuple(out):
    return out if isinstance(out, tuple) else (out,)


def segments(stream):
    """{address: bytes} of the allocator's segments for a stream."""
    return {s["address"]: s["total_size"] for s in torch.cuda.memory_snapshot() if s["stream"] == stream.cuda_stream}


def owner(t):
    """The stream whose memory holds t."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("by_handle", [False, True])
@pytest.mark.parametrize("what", CALLS)
def test_memory_is_of_the_given_stream(what, by_handle):
    call, room = what(torch.Generator(DEV).manual_seed(1))
    before = torch.cuda.current_stream()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    mine, theirs = segments(before), sum(segments(side).values())
    if what in (selected, paged):
        assert room > 20 << 20  # more than any segment has left
    side.wait_stream(before)
    out = as_tuple(call(stream=side.cuda_stream if by_handle else side))
    assert torch.cuda.current_stream() == before
    torch.cuda.synchronize()
    assert all(owner(t) == side.cuda_stream for t in out)
    assert sum(segments(side).values()) - theirs >= room
    if what in (selected, paged):
        assert segments(before) == mine


def test_the_current_stream_is_back_after_a_refusal():
    import row_top_selection_amd as dt

    g = torch.Generator(DEV).manual_seed(2)
    side, before = torch.cuda.Stream(), torch.cuda.current_stream()
    q, cache = randn(g, 4, 16, 576), randn(g, 4, 64, 576)
    with pytest.raises(dt.DsatopkError):
        dt.attend_selected(q, cache, i32(np.zeros((4, 8))), 448, SCALE, stream=side)
    assert torch.cuda.current_stream() == before
    with pytest.raises(ValueError):
        dt.attend_selected(q, cache, i32(np.zeros((3, 8))), 512, SCALE, stream=side)
    assert torch.cuda.current_stream() == before
    with pytest.raises(AttributeError):
        dt.attend_selected(q, cache, i32(np.zeros((4, 8))), 512, SCALE, stream="side")
    assert torch.cuda.current_stream() == before


@pytest.mark.parametrize("what", CALLS)
def test_results_on_a_given_stream(what):
    """The current stream allocates and fills blocks of the workspace's and
    the results' sizes while the given one may still be at work."""
    call, room = what(torch.Generator(DEV).manual_seed(3))
    want = [t.clone() for t in as_tuple(call())]
    sizes = [room] * (room > 0) + [t.numel() * t.element_size() for t in want]
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    for _ in range(4):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(3):  # in front of the call's kernels, so that they end late
                torch.mm(busy, busy)
        got = as_tuple(call(stream=side))
        fill = [torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xFF) for n in sizes for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del fill, got  # read on the current stream, dropped at once
        torch.cuda.synchronize()


def test_the_current_stream_given_by_name_in_a_capture():
    call, room = selected(torch.Generator(DEV).manual_seed(4))
    want = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(stream=torch.cuda.current_stream())
    for _ in range(3):
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_two_threads_with_streams_of_their_own():
    calls = [what(torch.Generator(DEV).manual_seed(5)) [0] for what in (selected, expanded)]
    want = [[t.clone() for t in call()] for call in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(call, right):
        side = torch.cuda.Stream()
        for n in range(40):
            if n % 2:
                got = call(stream=side)
            else:
                with torch.cuda.stream(side):
                    got = call()
            side.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, right)):
                wrong.append(n)

    threads = [threading.Thread(target=work, args=(c, w)) for c, w in zip(calls, want) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("what", CALLS)
def test_the_default_stream_given_while_another_is_current(what):
    call, _ = what(torch.Generator(DEV).manual_seed(6))
    want = [t.clone() for t in as_tuple(call())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for stream in (0, torch.cuda.default_stream()):
            got = as_tuple(call(stream=stream))
            assert torch.cuda.current_stream() == side
            assert all(owner(t) == 0 for t in got)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
