"""Python binding of the operators declared in include/kda_attn.h: causal attention
over prompts, attention of drafted tokens over a paged cache, the store of keys
and values into that cache, and its block tables and slots.

Argument marshalling only, as in ``ops`` and ``ssm_ops``: tensors are checked for
dtype, shape and device, their pointers and strides and the current HIP stream
go to the library, and there is no fallback.  ``stream=`` is as there.

A serving step with ``lens`` tokens of each request in the cache and T new ones:

    slots, new_lens, head = attn.assign_pages(lens, table, free_pages, head, page_size=64, tokens_per_seq=T)
    attn.store(k, v, k_cache, v_cache, slots)                      # k, v of the new tokens
    out, _ = attn.decode(q, k_cache, v_cache, table, lens)          # q [N, T, H, D]
"""
from __future__ import annotations

import ctypes

from .ops import _check, _ptr, load_library
from .ssm_ops import _batch, _check_tensor, _gpu, _launch, _like, _new, _offsets, _row_stride

_i32, _i64, _f32, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p

__all__ = ["AssignProblem", "DecodeProblem", "KvCache", "PrefillProblem", "StoreProblem", "assign_pages", "call_raw",
           "decode", "decode_workspace_size", "prefill", "store"]


class PrefillProblem(ctypes.Structure):
    """Mirror of ``kda_attn_problem``."""

    _fields_ = [("num_seqs", _i32), ("total_tokens", _i64), ("num_heads", _i32), ("num_kv_heads", _i32),
                ("head_dim", _i32), ("scale", _f32), ("cu_seqlens_int64", _i32), ("q_stride", _i64),
                ("k_stride", _i64), ("v_stride", _i64), ("out_stride", _i64)]


class KvCache(ctypes.Structure):
    """Mirror of ``kda_kv_cache``."""

    _fields_ = [("num_kv_heads", _i32), ("head_dim", _i32), ("dtype", _i32), ("page_size", _i32),
                ("num_pages", _i64), ("page_stride", _i64), ("token_stride", _i64)]


class DecodeProblem(ctypes.Structure):
    """Mirror of ``kda_attn_decode_problem``."""

    _fields_ = [("num_seqs", _i32), ("tokens_per_seq", _i32), ("num_heads", _i32), ("scale", _f32),
                ("table_rows", _i64), ("table_width", _i32), ("tree_per_seq", _i32), ("q_stride", _i64),
                ("out_stride", _i64), ("cache", KvCache)]


class StoreProblem(ctypes.Structure):
    """Mirror of ``kda_kv_store_problem``."""

    _fields_ = [("tokens", _i64), ("k_stride", _i64), ("v_stride", _i64), ("cache", KvCache)]


class AssignProblem(ctypes.Structure):
    """Mirror of ``kda_kv_assign_problem``."""

    _fields_ = [("num_seqs", _i32), ("total_tokens", _i64), ("page_size", _i32), ("table_width", _i32),
                ("table_rows", _i64), ("num_free", _i64), ("cu_seqlens_int64", _i32)]


# entry point: its problem, and how many pointers follow (with a byte count
# for the decode's workspace); the *_validate functions take no stream
_SIGNATURES = {
    "kda_attn_validate": (PrefillProblem, [_P] * 6),
    "kda_attn_prefill": (PrefillProblem, [_P] * 7),
    "kda_attn_decode_workspace_size": (DecodeProblem, [ctypes.POINTER(ctypes.c_size_t)]),
    "kda_attn_decode_validate": (DecodeProblem, [_P] * 12 + [ctypes.c_size_t]),
    "kda_attn_decode": (DecodeProblem, [_P] * 12 + [ctypes.c_size_t, _P]),
    "kda_kv_store_validate": (StoreProblem, [_P] * 7),
    "kda_kv_store": (StoreProblem, [_P] * 8),
    "kda_kv_assign_validate": (AssignProblem, [_P] * 9),
    "kda_kv_assign": (AssignProblem, [_P] * 10),
}
_ready = {}


def _fn(name: str):
    f = _ready.get(name)
    if f is None:
        f = getattr(load_library(), name)
        problem, rest = _SIGNATURES[name]
        f.argtypes = [ctypes.POINTER(problem)] + rest
        f.restype = ctypes.c_int
        _ready[name] = f
    return f


def call_raw(name: str, problem, *args) -> int:
    """Call an entry point of include/kda_attn.h with raw integer pointers
    (0 for NULL), in the header's order; returns the status."""
    return _fn(name)(ctypes.byref(problem), *args)


def decode_workspace_size(problem: DecodeProblem) -> int:
    n = ctypes.c_size_t(0)
    _check(_fn("kda_attn_decode_workspace_size")(ctypes.byref(problem), ctypes.byref(n)),
           "kda_attn_decode_workspace_size")
    return int(n.value)


def _rows(name: str, t, dtype, shape, dev):
    """``_check_tensor`` of a tensor whose rows may be strided, with the usual
    answer first: these calls take a good part of a small operator's time."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev:
        _check_tensor(name, t, dtype, shape, dev, False)


def _packed(name: str, t, dtype, shape, dev):
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _check_tensor(name, t, dtype, shape, dev)


def _stride(name: str, t, lead: int, shape) -> int:
    """``_row_stride``, the usual answers first."""
    if t.is_contiguous():
        return 0
    st = t.stride()
    if st[-1] == 1 and st[-2] == shape[-1] and shape[0] > 1:
        if lead == 1 and st[0] > 0:
            return st[0]
        if lead == 2 and st[1] > 0 and st[0] == shape[1] * st[1]:
            return st[1]
    return _row_stride(name, t, lead)


def _scale(scale, D: int) -> float:
    return D ** -0.5 if scale is None else float(scale)


def _lse(lse, wanted: bool, like, shape, dev, stream, mine):
    """The tensor that takes the logarithms, or None."""
    import torch

    if lse is not None:
        _check_tensor("lse", lse, torch.float32, shape, dev)
    elif wanted:
        lse = _new(like, stream, shape, torch.float32)
        mine.append(lse)
    return lse


def prefill(q, k, v, *, cu_seqlens=None, scale=None, out=None, return_lse: bool = False, lse=None, stream=None):
    """Causal attention over prompts.

    q: bf16 [T, H, D] (packed, with cu_seqlens int32 or int64 [N + 1]) or
    [B, T, H, D]; k, v: bf16 likewise with a number of heads that divides H, each
    shared by that many neighbouring query heads.  D is 64 or 128; rows may be strided
    (columns of one projection's row).  scale: of the scores, D ** -0.5 by
    default.  Rows behind cu_seqlens[N] are left as they are.  Returns (out,
    lse): lse, fp32 q.shape[:-1], is the logarithm of each row's sum of
    exponentials, None without return_lse or a tensor to take it."""
    import torch

    dev = _gpu(q, stream)
    bf = torch.bfloat16
    lead, N, T = _batch(q, 2, cu_seqlens, "[T, H, D] or [B, T, H, D]")
    shape = q.shape
    H, D = shape[lead:]
    if k.dim() != lead + 2:
        raise ValueError("k and v must be q.shape[:-2] + (KV, D)")
    KV = k.shape[lead]
    _rows("q", q, bf, shape, dev)
    _rows("k", k, bf, kv_shape := shape[:lead] + (KV, D), dev)
    _rows("v", v, bf, kv_shape, dev)
    cu64 = _offsets(cu_seqlens, dev)
    mine = []
    if out is None:
        out = _like(q, stream)
        mine.append(out)
    else:
        _rows("out", out, bf, shape, dev)
    lse = _lse(lse, return_lse, q, shape[:-1], dev, stream, mine)
    p = PrefillProblem(N, T, H, KV, D, _scale(scale, D), cu64, _stride("q", q, lead, shape), _stride("k", k, lead, kv_shape),
                       _stride("v", v, lead, kv_shape), _stride("out", out, lead, shape))
    _launch("kda_attn_prefill", dev, stream, p,
            [q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(cu_seqlens), out.data_ptr(), _ptr(lse)], mine, call_raw)
    return out, lse


def _strides(name: str, c, shape):
    """Elements between a cache's pages and between a page's tokens (0, 0: packed)."""
    page, token, head, one = c.stride()
    P, size, KV, D = shape
    if (D > 1 and one != 1) or (KV > 1 and head != D):
        raise ValueError(f"{name}: the last 2 dimensions must be contiguous")
    if (P > 1 and page <= 0) or (size > 1 and token <= 0):
        raise ValueError(f"{name}: pages and tokens must have positive strides")
    return (page if P > 1 else 0), (token if size > 1 else 0)


def _cache(k_cache, v_cache, k_scale, v_scale, dev) -> KvCache:
    import torch

    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("k_cache and v_cache must be [pages, page_size, KV, D]")
    P, size, KV, D = shape
    kind = k_cache.dtype
    if kind is torch.bfloat16:
        if k_scale is not None or v_scale is not None:
            raise ValueError(f"{'v_scale' if k_scale is None else 'k_scale'} is for a float8_e4m3fn cache")
    elif kind is torch.float8_e4m3fn:
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is None:
                raise ValueError(f"an 8-bit cache needs {name}")
            _packed(name, s, torch.float32, (KV,), dev)
    else:
        raise TypeError(f"k_cache must be bfloat16 or float8_e4m3fn, got {kind}")
    if k_cache.device != dev:
        raise ValueError(f"k_cache is on {k_cache.device}, expected {dev}")
    _rows("v_cache", v_cache, kind, shape, dev)
    page = token = 0
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        page, token = _strides("k_cache", k_cache, shape)
        if (page, token) != _strides("v_cache", v_cache, shape):
            raise ValueError("k_cache and v_cache must have the same strides")
    return KvCache(KV, D, kind is not torch.bfloat16, size, P, page, token)


def _table(table, rows, N, dev):
    import torch

    shape = table.shape
    if len(shape) != 2:
        raise ValueError("table must be [rows, pages of a row]")
    _packed("table", table, torch.int32, shape, dev)
    if rows is not None:
        _packed("rows", rows, torch.int32, (N,), dev)
    return shape


def decode(q, k_cache, v_cache, table, lens, *, rows=None, tree=None, scale=None, k_scale=None, v_scale=None, out=None,
           return_lse: bool = False, lse=None, workspace=None, stream=None):
    """Attention of T tokens (1 to 64) of each of N requests over a paged cache
    that holds their keys and values already, at the positions lens[n] + (0..T - 1).

    q: bf16 [N, T, H, D] (rows may be strided); k_cache, v_cache: bf16 or e4m3
    [pages, page_size, KV, D], KV dividing H, pages of 16 to 1024 tokens (a power of two;
    pages and tokens may be strided, as halves of one buffer are); k_scale, v_scale: fp32 [KV],
    positive, for e4m3.  table: int32 [R, W], a row of pages per request;
    rows: int32 [N], the requests' rows (None: row n), entries outside [0, R) mark
    empty slots (zero outputs).  lens: int32 [N], the tokens ahead of these.
    tree: int64 [N, T] or [T]: bit j of a token's word says that it sees the
    request's token j (itself included); None is a chain (j <= i).  All see
    the positions below lens[n]; a token that sees nothing gives zeros.
    workspace: a buffer of ``decode_workspace_size`` bytes; when None one is taken
    from torch's allocator if contexts are cut into parts.  Returns (out, lse) as
    ``prefill``; ``out=q`` overwrites q."""
    import torch

    dev = _gpu(q, stream)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [N, T, H, D]")
    N, T, H, D = shape
    _rows("q", q, torch.bfloat16, shape, dev)
    cache = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    if cache.head_dim != D:
        raise ValueError(f"k_cache has heads of {cache.head_dim}, q of {D}")
    R, W = _table(table, rows, N, dev)
    _packed("lens", lens, torch.int32, (N,), dev)
    if tree is not None:
        _packed("tree", tree, torch.int64, (T,) if tree.dim() == 1 else (N, T), dev)
    mine = []
    if out is None:
        out = _like(q, stream)
        mine.append(out)
    else:
        _rows("out", out, torch.bfloat16, shape, dev)
    lse = _lse(lse, return_lse, q, shape[:-1], dev, stream, mine)
    p = DecodeProblem(N, T, H, _scale(scale, D), R, W, int(tree is not None and tree.dim() == 2),
                      _stride("q", q, 2, shape), _stride("out", out, 2, shape), cache)
    if workspace is None:
        need = decode_workspace_size(p)
        if need:
            workspace = _new(q, stream, (need,), torch.uint8)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}")
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _launch("kda_attn_decode", dev, stream, p,
            [q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), _ptr(rows), lens.data_ptr(), _ptr(tree),
             _ptr(k_scale), _ptr(v_scale), out.data_ptr(), _ptr(lse), _ptr(workspace), size], mine, call_raw)
    return out, lse


def store(k, v, k_cache, v_cache, slots, *, k_scale=None, v_scale=None, stream=None):
    """Keys and values of T tokens into a paged cache, in place.

    k, v: bf16 [T, KV, D] (rows may be strided); the caches and scales as for
    ``decode``; slots: int64 [T], page * page_size + place in the page, distinct; a
    slot outside the cache (-1) stores nothing.  An e4m3 cache takes x / scale,
    at most 448 in magnitude, rounded to nearest even."""
    import torch

    dev = _gpu(k, stream)
    shape = k.shape
    if len(shape) != 3:
        raise ValueError("k and v must be [T, KV, D]")
    T = shape[0]
    cache = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    _rows("k", k, torch.bfloat16, (T, cache.num_kv_heads, cache.head_dim), dev)
    _rows("v", v, torch.bfloat16, shape, dev)
    _packed("slots", slots, torch.int64, (T,), dev)
    p = StoreProblem(T, _stride("k", k, 1, shape), _stride("v", v, 1, shape), cache)
    _launch("kda_kv_store", dev, stream, p,
            [k.data_ptr(), v.data_ptr(), slots.data_ptr(), _ptr(k_scale), _ptr(v_scale), k_cache.data_ptr(),
             v_cache.data_ptr()], (), call_raw)


def assign_pages(lens, table, free_pages, free_head, *, page_size: int, rows=None, cu_seqlens=None, total_tokens=None,
                 tokens_per_seq: int = 1, slots=None, lens_out=None, head_out=None, stream=None):
    """Pages and slots of requests' new tokens, on the device.

    lens: int32 [N], the tokens that each request has in its pages.  New ones:
    tokens_per_seq for each, or those of a packed batch, cu_seqlens int32 or int64
    [N + 1], whose row count is total_tokens (or that of ``slots``).  table: int32
    [R, W], the requests' rows of pages, updated in place; rows: int32 [N] (None: row n),
    entries outside [0, R) mark empty slots of the batch.  free_pages: int32 [F]
    and free_head: int32 [1], the first of them that is free: pages that the new tokens
    open come from there on, in the order of the requests.  Returns (slots int64
    [tokens], lens_out, head_out), which are for ``store`` and for the next step;
    tokens without a page (an empty slot, a table that is too narrow, no free page:
    head_out is past F then) and rows behind cu_seqlens[N] have the slot -1."""
    import torch

    dev = _gpu(lens, stream)
    i32 = torch.int32
    shape = lens.shape
    if len(shape) != 1:
        raise ValueError("lens must be [N]")
    N = shape[0]
    _packed("lens", lens, i32, shape, dev)
    R, W = _table(table, rows, N, dev)
    F = free_pages.numel()
    _packed("free_pages", free_pages, i32, (F,), dev)
    _packed("free_head", free_head, i32, (1,), dev)
    cu64 = _offsets(cu_seqlens, dev)
    if cu_seqlens is None:
        if total_tokens is not None or tokens_per_seq < 0:
            raise ValueError("total_tokens is for packed batches" if total_tokens is not None
                             else "tokens_per_seq must not be negative")
        T = N * tokens_per_seq
    else:
        if cu_seqlens.numel() != N + 1:
            raise ValueError(f"cu_seqlens must have {N + 1} entries")
        if total_tokens is None and slots is None:
            raise ValueError("a packed batch needs total_tokens or slots")
        T = slots.numel() if total_tokens is None else total_tokens
    mine = []

    if slots is None:
        slots = _new(lens, stream, (T,), torch.int64)
        mine.append(slots)
    else:
        _packed("slots", slots, torch.int64, (T,), dev)
    if lens_out is None:
        lens_out = _like(lens, stream)
        mine.append(lens_out)
    else:
        _packed("lens_out", lens_out, i32, shape, dev)
    if head_out is None:
        head_out = _like(free_head, stream)
        mine.append(head_out)
    else:
        _packed("head_out", head_out, i32, (1,), dev)
    p = AssignProblem(N, T, page_size, W, R, F, cu64)
    _launch("kda_kv_assign", dev, stream, p,
            [lens.data_ptr(), _ptr(rows), _ptr(cu_seqlens), table.data_ptr(), free_pages.data_ptr(), free_head.data_ptr(),
             slots.data_ptr(), lens_out.data_ptr(), head_out.data_ptr()], mine, call_raw)
    return slots, lens_out, head_out
