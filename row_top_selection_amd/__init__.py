"""Python binding of ``libdsatopk.so`` (the C ABI in ``include/dsatopk.h``).

Argument marshalling only: every step of the selection runs in the HIP
kernels of the library. Tensors are torch CUDA (HIP) tensors; torch is used
for device memory and the current stream. If the library has not been
built, every call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
from pathlib import Path
from typing import NamedTuple

LIB_PATH = Path(__file__).resolve().parent / "libdsatopk.so"

MAX_K = 2048
MAX_SEQ_LEN = 131072

STATUS = {
    0: "DSATOPK_OK",
    1: "DSATOPK_ERR_INVALID_ARG",
    2: "DSATOPK_ERR_ALIGNMENT",
    3: "DSATOPK_ERR_PLAN_TOO_SMALL",
    4: "DSATOPK_ERR_HIP",
    5: "DSATOPK_ERR_TOO_LARGE",
    6: "DSATOPK_ERR_WORKSPACE_TOO_SMALL",
}

NOALLOC_MAX_ROWS = 262144

EXPORTS = ("dsatopk_status_string", "dsatopk_plan_bytes", "dsatopk_plan", "dsatopk_plan_error",
           "dsatopk_paged", "dsatopk_paged_packed", "dsatopk_ragged", "dsatopk_paged_noalloc",
           "dsatopk_page_maps", "dsatopk_scores_paged", "dsatopk_scores_ragged",
           "dsatopk_attend_bytes", "dsatopk_attend_selected", "dsatopk_attend_paged",
           "dsatopk_attend_expanded")


class DsatopkError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({_lib().dsatopk_status_string(status).decode()})")


_handle = None


def _lib():
    """The loaded library with argument types set (raises if not built)."""
    global _handle
    if _handle is None:
        if not LIB_PATH.exists():
            raise ImportError(f"{LIB_PATH} is not built: run row_top_selection_amd.build.build()")
        # torch's HIP runtime first: it carries the soname this library
        # links against, so the library binds to it. Loaded the other way
        # round, the process would hold a second HIP runtime, which knows
        # none of torch's streams.
        import torch  # noqa: F401

        lib = ctypes.CDLL(str(LIB_PATH))
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        lib.dsatopk_status_string.argtypes = [ctypes.c_int]
        lib.dsatopk_status_string.restype = ctypes.c_char_p
        lib.dsatopk_plan_bytes.argtypes = [i32]
        lib.dsatopk_plan_bytes.restype = sz
        lib.dsatopk_plan.argtypes = [P, P, i32, i32, P, sz, P]
        lib.dsatopk_plan.restype = ctypes.c_int
        lib.dsatopk_plan_error.argtypes = [P, sz, P, P]
        lib.dsatopk_plan_error.restype = ctypes.c_int
        lib.dsatopk_paged.argtypes = [P, i64, P, P, P, i64, i32, i32, i32, P, sz, P, P]
        lib.dsatopk_paged.restype = ctypes.c_int
        lib.dsatopk_paged_packed.argtypes = [P, i64, P, P, P, i64, i32, P, P, i32, i32, P, sz,
                                             P, P, P]
        lib.dsatopk_paged_packed.restype = ctypes.c_int
        lib.dsatopk_ragged.argtypes = [P, i64, P, P, P, i32, i32, P, sz, P, P]
        lib.dsatopk_ragged.restype = ctypes.c_int
        lib.dsatopk_paged_noalloc.argtypes = [P, i64, P, P, P, i64, i32, i32, i32, P, P]
        lib.dsatopk_paged_noalloc.restype = ctypes.c_int
        lib.dsatopk_page_maps.argtypes = [P, P, i32, P, i64, i32, i32, P, i32, i32, P, P, P, P, P,
                                          P]
        lib.dsatopk_page_maps.restype = ctypes.c_int
        lib.dsatopk_scores_paged.argtypes = [P, i64, i64, P, i64, P, i64, i64, i64, P, i64, i32,
                                             i32, i32, P, P, i64, i32, i32, P, i32, P, i64, i64, P]
        lib.dsatopk_scores_paged.restype = ctypes.c_int
        lib.dsatopk_scores_ragged.argtypes = [P, i64, i64, P, i64, P, i64, i64, P, i32, i32, i32,
                                              P, P, i32, P, i64, i64, P]
        lib.dsatopk_scores_ragged.restype = ctypes.c_int
        f32 = ctypes.c_float
        lib.dsatopk_attend_bytes.argtypes = [i32, i32, i32, i64]
        lib.dsatopk_attend_bytes.restype = sz
        lib.dsatopk_attend_selected.argtypes = [P, i64, i64, P, i64, i64, i64, i32, i32, i32, i32,
                                                i32, f32, P, i64, i32, i32, P, P, P, sz, P]
        lib.dsatopk_attend_selected.restype = ctypes.c_int
        lib.dsatopk_attend_paged.argtypes = [P, i64, i64, P, i64, i64, i64, i32, i32, i32, i32,
                                             i32, f32, P, P, i64, i32, P, i64, i32, P, P, P, sz, P]
        lib.dsatopk_attend_paged.restype = ctypes.c_int
        lib.dsatopk_attend_expanded.argtypes = [P, i64, i64, P, i64, i64, P, i64, i64, P, i64, i32,
                                                i32, i32, i32, i32, f32, i32, P, P, i32, i32, i32,
                                                i32, P, P, P]
        lib.dsatopk_attend_expanded.restype = ctypes.c_int
        _handle = lib
    return _handle


def lib():
    """Raw ctypes handle of libdsatopk.so."""
    return _lib()


def _stream(stream):
    import torch

    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on(t, like, name):
    """t must be a device tensor on like's device."""
    if not t.is_cuda or t.device != like.device:
        raise ValueError(f"{name} must be a device tensor on {like.device}")
    return t


def _vec_i32(t, n, name, like=None):
    import torch

    if t is None:
        return None
    if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 vector of length {n}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if like is not None:
        _on(t, like, name)
    return t


def _scores(scores):
    import torch

    if scores.dtype != torch.float32 or scores.dim() != 2 or scores.stride(1) != 1:
        raise ValueError("scores must be a 2-D float32 tensor with contiguous columns")
    if not scores.is_cuda:
        raise ValueError("scores must be a device tensor")
    return scores


def _out(out, rows, k, like, name="out"):
    import torch

    if out is None:
        return torch.empty((rows, k), dtype=torch.int32, device=like.device)
    if out.dtype != torch.int32 or tuple(out.shape) != (rows, k) or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape ({rows}, {k})")
    return _on(out, like, name)


def _plan_arg(plan, like):
    """(pointer, bytes) of a plan tensor on like's device, or (None, 0)."""
    import torch

    if plan is None:
        return None, 0
    if plan.dtype != torch.uint8 or not plan.is_contiguous():
        raise ValueError("plan must be a contiguous uint8 tensor from plan()")
    _on(plan, like, "plan")
    return plan.data_ptr(), plan.numel()


def plan_bytes(num_rows: int) -> int:
    return int(_lib().dsatopk_plan_bytes(int(num_rows)))


def plan(seq_lens, k: int, row_starts=None, out=None, stream=None):
    """Build a plan (uint8 device tensor) from ``seq_lens`` / ``row_starts``."""
    import torch

    n = int(seq_lens.shape[0])
    _vec_i32(seq_lens, n, "seq_lens")
    _vec_i32(row_starts, n, "row_starts", seq_lens)
    nbytes = plan_bytes(n)
    if out is None:
        out = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=seq_lens.device)
    else:
        _plan_arg(out, seq_lens)
    st = _lib().dsatopk_plan(_ptr(seq_lens), _ptr(row_starts), n, int(k), _ptr(out), out.numel(),
                             _stream(stream))
    if st != 0:
        raise DsatopkError(st, "dsatopk_plan")
    return out


def plan_error(plan, stream=None) -> int:
    """The plan's error word (synchronizes the stream): 1 if a split row's
    wait gave up in a transform call since the plan was built, else 0."""
    err = ctypes.c_int32(0)
    st = _lib().dsatopk_plan_error(_ptr(plan), plan.numel(), ctypes.byref(err), _stream(stream))
    if st != 0:
        raise DsatopkError(st, "dsatopk_plan_error")
    return int(err.value)


def paged(scores, seq_lens, page_table, page_size: int, k: int, row_starts=None, plan=None,
          out=None, stream=None, table_rows=None, table_starts=None, out_raw=None):
    """PAGED top-k: int32 ``[rows, k]`` of page-table-mapped positions.

    Packed rows (``dsatopk_paged_packed``): ``table_rows`` picks each row's
    page-table row, ``table_starts`` its table position of window position
    0; ``out_raw`` (int32 ``[rows, k]``, or True to allocate one) also
    receives the window positions, slot for slot. Returns ``out``, or
    ``(out, out_raw)`` when ``out_raw`` is given."""
    import torch

    scores = _scores(scores)
    rows = int(scores.shape[0])
    _vec_i32(seq_lens, rows, "seq_lens", scores)
    _vec_i32(row_starts, rows, "row_starts", scores)
    _vec_i32(table_rows, rows, "table_rows", scores)
    _vec_i32(table_starts, rows, "table_starts", scores)
    packed = table_rows is not None or table_starts is not None or out_raw is not None
    if page_table.dtype != torch.int32:
        raise ValueError("page_table must be int32")
    if page_table.dim() != 2 or page_table.stride(1) != 1:
        raise ValueError("page_table must be [table rows, width] with contiguous columns")
    _on(page_table, scores, "page_table")
    if table_rows is None and page_table.shape[0] != rows:
        raise ValueError("page_table must have one row per score row without table_rows")
    out = _out(out, rows, int(k), scores)
    if out_raw is True:
        out_raw = _out(None, rows, int(k), scores, "out_raw")
    elif out_raw is not None:
        out_raw = _out(out_raw, rows, int(k), scores, "out_raw")
    plan_ptr, plan_n = _plan_arg(plan, scores)
    if not packed:
        st = _lib().dsatopk_paged(
            _ptr(scores), scores.stride(0), _ptr(seq_lens), _ptr(row_starts), _ptr(page_table),
            page_table.stride(0), int(page_size), rows, int(k), plan_ptr, plan_n, _ptr(out),
            _stream(stream))
        if st != 0:
            raise DsatopkError(st, "dsatopk_paged")
        return out
    st = _lib().dsatopk_paged_packed(
        _ptr(scores), scores.stride(0), _ptr(seq_lens), _ptr(row_starts), _ptr(page_table),
        page_table.stride(0), int(page_size), _ptr(table_rows), _ptr(table_starts), rows,
        int(k), plan_ptr, plan_n, _ptr(out), _ptr(out_raw), _stream(stream))
    if st != 0:
        raise DsatopkError(st, "dsatopk_paged_packed")
    return out if out_raw is None else (out, out_raw)


def ragged(scores, seq_lens, out_offsets, k: int, row_starts=None, plan=None, out=None,
           stream=None):
    """RAGGED top-k: int32 ``[rows, k]`` of position + out_offsets[row]."""
    scores = _scores(scores)
    rows = int(scores.shape[0])
    _vec_i32(seq_lens, rows, "seq_lens", scores)
    _vec_i32(row_starts, rows, "row_starts", scores)
    _vec_i32(out_offsets, rows, "out_offsets", scores)
    out = _out(out, rows, int(k), scores)
    plan_ptr, plan_n = _plan_arg(plan, scores)
    st = _lib().dsatopk_ragged(
        _ptr(scores), scores.stride(0), _ptr(seq_lens), _ptr(row_starts), _ptr(out_offsets),
        rows, int(k), plan_ptr, plan_n, _ptr(out), _stream(stream))
    if st != 0:
        raise DsatopkError(st, "dsatopk_ragged")
    return out


def paged_noalloc(scores, seq_lens, page_table, page_size: int, k: int, row_starts=None,
                  out=None, stream=None):
    """PAGED top-k through ``dsatopk_paged_noalloc`` (the plan lives in the
    library's static device memory; nothing is allocated except ``out`` when
    it is not given)."""
    import torch

    scores = _scores(scores)
    rows = int(scores.shape[0])
    _vec_i32(seq_lens, rows, "seq_lens", scores)
    _vec_i32(row_starts, rows, "row_starts", scores)
    if page_table.dtype != torch.int32:
        raise ValueError("page_table must be int32")
    if page_table.dim() != 2 or page_table.stride(1) != 1 or page_table.shape[0] != rows:
        raise ValueError("page_table must be [rows, width] with contiguous columns")
    _on(page_table, scores, "page_table")
    out = _out(out, rows, int(k), scores)
    st = _lib().dsatopk_paged_noalloc(
        _ptr(scores), scores.stride(0), _ptr(seq_lens), _ptr(row_starts), _ptr(page_table),
        page_table.stride(0), int(page_size), rows, int(k), _ptr(out), _stream(stream))
    if st != 0:
        raise DsatopkError(st, "dsatopk_paged_noalloc")
    return out


class PageMaps(NamedTuple):
    """What ``page_maps`` writes beside the page table."""

    token_starts: "torch.Tensor"  # int32 [requests + 1]
    slots: "torch.Tensor"         # int32 [num_tokens], -1: none
    table_rows: "torch.Tensor"    # int32 [num_tokens]
    row_lens: "torch.Tensor"      # int32 [num_tokens]
    counts: "torch.Tensor"        # int32 [2]: tokens, pages opened


def _table(page_table, like, name="page_table"):
    import torch

    if page_table.dtype != torch.int32:
        raise ValueError(f"{name} must be int32")
    if page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError(f"{name} must be [rows, width] with contiguous columns")
    if not page_table.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if like is not None:
        _on(page_table, like, name)
    return page_table


def _row_stride(t):
    """Elements between t's rows (at least a row: what one row's stride says does not matter)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _stride(t, dim):
    """t's stride; 0 where one entry makes it meaningless."""
    return t.stride(dim) if t.shape[dim] > 1 else 0


def page_maps(seq_lens, page_table, page_size: int, free_pages, num_tokens: int, new_lens=None,
              out=None, stream=None):
    """The pages, slots and top-k row arguments of a serving step.

    Requests of ``seq_lens`` tokens after the step, ``new_lens`` of them new
    (None: one each), take the pages that they lack from ``free_pages``:
    these are written into ``page_table`` in place. Returns ``PageMaps``,
    whose ``slots``, ``table_rows`` and ``row_lens`` have ``num_tokens`` rows
    (empty ones behind the step's tokens). ``out``: a ``PageMaps`` to write
    into."""
    import torch

    n, t = int(seq_lens.shape[0]), int(num_tokens)
    _vec_i32(seq_lens, n, "seq_lens")
    _vec_i32(new_lens, n, "new_lens", seq_lens)
    _table(page_table, seq_lens)
    if page_table.shape[0] != n:
        raise ValueError("page_table must have one row per request")
    _vec_i32(free_pages, int(free_pages.shape[0]), "free_pages", seq_lens)
    if t < 0:
        raise ValueError("num_tokens must not be negative")
    if out is None:
        sizes = (n + 1, t, t, t, 2)
        # one allocation, its parts at 16-byte boundaries
        whole = torch.empty(sum((s + 3) // 4 * 4 for s in sizes), dtype=torch.int32,
                            device=seq_lens.device)
        parts, at = [], 0
        for s in sizes:
            parts.append(whole[at:at + s])
            at += (s + 3) // 4 * 4
        out = PageMaps(*parts)
    else:
        for name, size in zip(PageMaps._fields, (n + 1, t, t, t, 2)):
            _vec_i32(getattr(out, name), size, name, seq_lens)
    st = _lib().dsatopk_page_maps(
        _ptr(seq_lens), _ptr(new_lens), n, _ptr(page_table), _row_stride(page_table),
        page_table.shape[1], int(page_size), _ptr(free_pages), free_pages.shape[0], t,
        *(_ptr(getattr(out, name)) for name in ("token_starts", "slots", "table_rows", "row_lens",
                                                "counts")), _stream(stream))
    if st != 0:
        raise DsatopkError(st, "dsatopk_page_maps")
    return out


def _element_type(t, name, fp8=False):
    """The library's number for t's element type."""
    import torch

    types = {torch.bfloat16: 0, torch.float16: 1}
    if fp8:
        types[torch.float8_e4m3fn] = 2
    if t.dtype not in types:
        raise ValueError(f"{name} must be one of {', '.join(str(d) for d in types)}")
    return types[t.dtype]


def _tensor(t, dims, like, name):
    """A device tensor of ``dims`` dimensions with a contiguous last one."""
    if t.dim() != dims or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must have {dims} dimensions, the last one contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if like is not None:
        _on(t, like, name)
    return t


def _score_args(q, weights, keys, key_scales, key_dims):
    import torch

    _tensor(q, 3, None, "q")
    rows, heads, dim = q.shape
    _tensor(weights, 2, q, "weights")
    if weights.dtype != torch.float32 or tuple(weights.shape) != (rows, heads):
        raise ValueError(f"weights must be float32 of shape ({rows}, {heads})")
    _tensor(keys, key_dims, q, "keys")
    kind = _element_type(q, "q", fp8=True)
    if keys.dtype != q.dtype or keys.shape[-1] != dim:
        raise ValueError("keys must have q's type and head dimension")
    if key_scales is not None:
        _tensor(key_scales, key_dims - 1, q, "key_scales")
        if key_scales.dtype != torch.float32 or key_scales.shape != keys.shape[:-1]:
            raise ValueError("key_scales must be float32, one per key")
    return kind, int(rows), int(heads), int(dim)


def _score_out(out, rows, columns, like):
    import torch

    if out is None:
        # a top-k's score buffer: row stride a multiple of 4
        return torch.empty((rows, max(4, (columns + 3) // 4 * 4)), dtype=torch.float32,
                           device=like.device)
    _tensor(out, 2, like, "out")
    if out.dtype != torch.float32 or out.shape[0] != rows:
        raise ValueError(f"out must be float32 with {rows} rows")
    return out


def scores_paged(q, weights, keys, seq_lens, page_table, key_scales=None, table_rows=None,
                 out=None, stream=None):
    """Indexer scores over a paged key cache, as ``paged`` reads them.

    ``q`` [rows, heads, dim] and ``keys`` [pages, page_size, dim] in
    bfloat16, float16 or float8_e4m3fn, ``weights`` float32 [rows, heads],
    ``key_scales`` float32 [pages, page_size] or None. Column j < seq_len of
    row b of ``out`` gets key_scale[j] * sum_h weights[b, h] * max(0, q[b, h]
    . key[j]); other columns are not written. Returns ``out`` (allocated with
    a column per table position when None)."""
    kind, rows, heads, dim = _score_args(q, weights, keys, key_scales, 3)
    _vec_i32(seq_lens, rows, "seq_lens", q)
    _vec_i32(table_rows, rows, "table_rows", q)
    _table(page_table, q)
    if table_rows is None and page_table.shape[0] != rows:
        raise ValueError("page_table must have one row per query row without table_rows")
    page_size = int(keys.shape[1])
    out = _score_out(out, rows, page_table.shape[1] * page_size, q)
    st = _lib().dsatopk_scores_paged(
        _ptr(q), _stride(q, 0), _stride(q, 1), _ptr(weights), _stride(weights, 0), _ptr(keys),
        keys.shape[0], _stride(keys, 0), _stride(keys, 1), _ptr(key_scales),
        0 if key_scales is None else _stride(key_scales, 0), kind, heads, dim, _ptr(seq_lens),
        _ptr(page_table), _row_stride(page_table), page_table.shape[1], page_size,
        _ptr(table_rows), rows, _ptr(out), _row_stride(out), out.shape[1], _stream(stream))
    if st != 0:
        raise DsatopkError(st, "dsatopk_scores_paged")
    return out


def scores_ragged(q, weights, keys, seq_lens, row_starts, key_scales=None, out=None,
                  stream=None):
    """Indexer scores over flattened keys [tokens, dim], as ``ragged`` reads
    them: row b's window is columns row_starts[b] .. row_starts[b] +
    seq_lens[b] - 1 of ``out``; other columns are not written. Arguments as
    for ``scores_paged``, ``key_scales`` float32 [tokens]."""
    kind, rows, heads, dim = _score_args(q, weights, keys, key_scales, 2)
    _vec_i32(seq_lens, rows, "seq_lens", q)
    _vec_i32(row_starts, rows, "row_starts", q)
    if row_starts is None:
        raise ValueError("row_starts is required")
    out = _score_out(out, rows, keys.shape[0], q)
    st = _lib().dsatopk_scores_ragged(
        _ptr(q), _stride(q, 0), _stride(q, 1), _ptr(weights), _stride(weights, 0), _ptr(keys),
        keys.shape[0], _stride(keys, 0), _ptr(key_scales), kind, heads, dim, _ptr(seq_lens),
        _ptr(row_starts), rows, _ptr(out), _row_stride(out), out.shape[1], _stream(stream))
    if st != 0:
        raise DsatopkError(st, "dsatopk_scores_ragged")
    return out


def _attend_out(out, lse, q, shape):
    """Attention's results: out (q's type) of ``shape``, lse (float32) of its first two."""
    import torch

    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
    elif out.dtype != q.dtype or tuple(out.shape) != shape or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {q.dtype} tensor of shape {shape}")
    else:
        _on(out, q, "out")
    if lse is None:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=q.device)
    elif lse.dtype != torch.float32 or tuple(lse.shape) != shape[:2] or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {shape[:2]}")
    else:
        _on(lse, q, "lse")
    return out, lse


def _attend_args(q, cache, latent_dim, out, lse, workspace, max_tokens):
    import torch

    _tensor(q, 3, None, "q")
    _tensor(cache, 3, q, "cache")
    rows, heads, dim = q.shape
    kind = _element_type(q, "q")
    if cache.dtype != q.dtype or cache.shape[-1] != dim:
        raise ValueError("cache must have q's type and last dimension")
    out, lse = _attend_out(out, lse, q, (rows, heads, int(latent_dim)))
    if workspace is None:
        need = attend_bytes(rows, heads, latent_dim, max_tokens)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    else:
        _on(workspace, q, "workspace")
    head = (_ptr(q), _stride(q, 0), _stride(q, 1), _ptr(cache), cache.shape[0], _stride(cache, 0),
            _stride(cache, 1), cache.shape[1], kind, heads, int(latent_dim), dim - int(latent_dim))
    tail = (_ptr(out), _ptr(lse), _ptr(workspace), 0 if workspace is None else workspace.numel())
    return out, lse, rows, head, tail


def attend_bytes(num_rows: int, num_heads: int, latent_dim: int, max_tokens: int) -> int:
    """Workspace bytes of ``attend_selected`` (max_tokens: k) and
    ``attend_paged`` (max_tokens: max_seq_len)."""
    return int(_lib().dsatopk_attend_bytes(int(num_rows), int(num_heads), int(latent_dim),
                                           int(max_tokens)))


def attend_selected(q, cache, slots, latent_dim: int, scale: float, out=None, lse=None,
                    workspace=None, stream=None):
    """Absorbed latent attention over selected cache slots.

    ``q`` [rows, heads, latent_dim + 64] and ``cache`` [pages, page_size,
    latent_dim + 64] in bfloat16 or float16; ``slots`` int32 [rows, k] as
    ``paged`` returns them (-1: none). Returns ``(out, lse)``: q's type
    [rows, heads, latent_dim], and float32 [rows, heads]. ``workspace``: uint8
    of ``attend_bytes(rows, heads, latent_dim, k)`` (allocated when None)."""
    import torch

    _tensor(slots, 2, q, "slots")
    if slots.dtype != torch.int32 or slots.shape[0] != q.shape[0]:
        raise ValueError("slots must be int32 with one row per query row")
    k = int(slots.shape[1])
    out, lse, rows, head, tail = _attend_args(q, cache, latent_dim, out, lse, workspace, k)
    st = _lib().dsatopk_attend_selected(*head, float(scale), _ptr(slots), _row_stride(slots), k,
                                        rows, *tail, _stream(stream))
    if st != 0:
        raise DsatopkError(st, "dsatopk_attend_selected")
    return out, lse


def attend_paged(q, cache, seq_lens, page_table, latent_dim: int, scale: float, table_rows=None,
                 max_seq_len=None, out=None, lse=None, workspace=None, stream=None):
    """Absorbed latent attention over the first ``seq_lens`` positions of each
    row's page table. Arguments as for ``attend_selected`` and ``paged``;
    ``max_seq_len`` bounds ``seq_lens`` (the table's width when None) and
    sets how rows are split."""
    _tensor(q, 3, None, "q")
    n = int(q.shape[0])
    _vec_i32(seq_lens, n, "seq_lens", q)
    _vec_i32(table_rows, n, "table_rows", q)
    _table(page_table, q)
    if table_rows is None and page_table.shape[0] != n:
        raise ValueError("page_table must have one row per query row without table_rows")
    _tensor(cache, 3, q, "cache")
    if max_seq_len is None:
        max_seq_len = page_table.shape[1] * cache.shape[1]
    out, lse, rows, head, tail = _attend_args(q, cache, latent_dim, out, lse, workspace,
                                              int(max_seq_len))
    st = _lib().dsatopk_attend_paged(*head, float(scale), _ptr(seq_lens), _ptr(page_table),
                                     _row_stride(page_table), page_table.shape[1],
                                     _ptr(table_rows), int(max_seq_len), rows, *tail,
                                     _stream(stream))
    if st != 0:
        raise DsatopkError(st, "dsatopk_attend_paged")
    return out, lse


def attend_expanded(q, k, v, k_rope, q_starts, k_starts, max_queries: int, scale: float,
                    causal: bool = True, out=None, lse=None, stream=None):
    """Expanded latent attention over a ragged batch of prompts.

    ``q`` [queries, heads, 192], ``k`` and ``v`` [keys, heads, 128] and
    ``k_rope`` [keys, 64] in bfloat16 or float16 (k and v may be parts of one
    tensor); ``q_starts`` and ``k_starts`` int32 [requests + 1];
    ``max_queries`` bounds a request's queries, which are its last tokens.
    Returns ``(out, lse)``: q's type [queries, heads, 128], and float32
    [queries, heads]."""
    _tensor(q, 3, None, "q")
    queries, heads, dim = q.shape
    kind = _element_type(q, "q")
    for name, t, dims in (("k", k, 3), ("v", v, 3), ("k_rope", k_rope, 2)):
        _tensor(t, dims, q, name)
        if t.dtype != q.dtype or t.shape[0] != k.shape[0] or (dims == 3 and t.shape[1] != heads):
            raise ValueError(f"{name} must have q's type, k's rows and q's heads")
    if dim != k.shape[2] + k_rope.shape[1]:
        raise ValueError("q's last dimension must be k's and k_rope's together")
    n = int(q_starts.shape[0]) - 1
    if n < 0:
        raise ValueError("q_starts must have an entry more than there are requests")
    _vec_i32(q_starts, n + 1, "q_starts", q)
    _vec_i32(k_starts, n + 1, "k_starts", q)
    out, lse = _attend_out(out, lse, q, (queries, heads, int(v.shape[2])))
    st = _lib().dsatopk_attend_expanded(
        _ptr(q), _stride(q, 0), _stride(q, 1), _ptr(k), _stride(k, 0), _stride(k, 1), _ptr(v),
        _stride(v, 0), _stride(v, 1), _ptr(k_rope), _stride(k_rope, 0), kind, heads, k.shape[2],
        k_rope.shape[1], v.shape[2], float(scale), int(bool(causal)), _ptr(q_starts),
        _ptr(k_starts), n, queries, k.shape[0], int(max_queries), _ptr(out), _ptr(lse),
        _stream(stream))
    if st != 0:
        raise DsatopkError(st, "dsatopk_attend_expanded")
    return out, lse
