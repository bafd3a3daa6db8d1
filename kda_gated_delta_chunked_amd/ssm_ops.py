"""Python binding of the operators declared in include/kda_ssm.h: the short
causal convolution, the selective state space scan (prompts and state-pool
decode) and the residual RMS norm with its 8-bit output.

Argument marshalling only, as in ``ops``: tensors are checked for dtype, shape
and device, their pointers and row strides and the current HIP stream go to
the library, and there is no fallback.

With ``stream=`` a call runs on that stream instead: the caller sees to it that
its inputs are ready there and are kept until the stream is done with them, and
that it is before the results are used on another stream.  Results and
workspaces that the call allocates are the stream's own from the start.
"""
from __future__ import annotations

import ctypes

from .ops import STATE_DTYPES, _check, _check_stream, _ptr, load_library

_i32, _i64, _f32, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p

ACTIVATIONS = {"none": 0, "silu": 1}
SPLIT_TOKENS = 128  # KDA_SSM_SPLIT_TOKENS


class ConvProblem(ctypes.Structure):
    """Mirror of ``kda_conv_problem``."""

    _fields_ = [("num_seqs", _i32), ("total_tokens", _i64), ("dim", _i32), ("width", _i32),
                ("activation", _i32), ("cu_seqlens_int64", _i32), ("x_stride", _i64), ("out_stride", _i64)]


class ConvDecodeProblem(ctypes.Structure):
    """Mirror of ``kda_conv_decode_problem``."""

    _fields_ = [("num_seqs", _i32), ("tokens_per_seq", _i32), ("dim", _i32), ("width", _i32),
                ("activation", _i32), ("pool_size", _i64), ("x_stride", _i64), ("out_stride", _i64)]


class SsmProblem(ctypes.Structure):
    """Mirror of ``kda_ssm_problem``."""

    _fields_ = [("num_seqs", _i32), ("total_tokens", _i64), ("num_heads", _i32), ("num_groups", _i32),
                ("head_dim", _i32), ("d_state", _i32), ("dt_softplus", _i32), ("state_dtype", _i32),
                ("cu_seqlens_int64", _i32), ("piece_tokens", _i32), ("packed", _i32), ("x_stride", _i64), ("b_stride", _i64),
                ("c_stride", _i64), ("z_stride", _i64), ("out_stride", _i64)]


class SsmDecodeProblem(ctypes.Structure):
    """Mirror of ``kda_ssm_decode_problem``."""

    _fields_ = [("num_seqs", _i32), ("tokens_per_seq", _i32), ("num_heads", _i32), ("num_groups", _i32),
                ("head_dim", _i32), ("d_state", _i32), ("dt_softplus", _i32), ("state_dtype", _i32),
                ("pool_size", _i64), ("x_stride", _i64), ("b_stride", _i64), ("c_stride", _i64),
                ("z_stride", _i64), ("out_stride", _i64)]


class NormProblem(ctypes.Structure):
    """Mirror of ``kda_norm_problem``."""

    _fields_ = [("rows", _i64), ("dim", _i32), ("eps", _f32), ("out_dtype", _i32), ("scale_group", _i32),
                ("x_stride", _i64)]


# entry point: its problem, and how many pointers follow (with a byte count
# for the scan's workspace); the *_validate functions take no stream
_SIGNATURES = {
    "kda_conv_validate": (ConvProblem, [_P] * 7),
    "kda_conv_prefill": (ConvProblem, [_P] * 8),
    "kda_conv_decode_validate": (ConvDecodeProblem, [_P] * 6),
    "kda_conv_decode": (ConvDecodeProblem, [_P] * 7),
    "kda_ssm_plan": (SsmProblem, [ctypes.POINTER(_i32)]),
    "kda_ssm_prefill_workspace_size": (SsmProblem, [ctypes.POINTER(ctypes.c_size_t)]),
    "kda_ssm_validate": (SsmProblem, [_P] * 13 + [ctypes.c_size_t]),
    "kda_ssm_prefill": (SsmProblem, [_P] * 13 + [ctypes.c_size_t, _P]),
    "kda_ssm_decode_validate": (SsmDecodeProblem, [_P] * 11),
    "kda_ssm_decode": (SsmDecodeProblem, [_P] * 12),
    "kda_add_rmsnorm_validate": (NormProblem, [_P] * 6),
    "kda_add_rmsnorm": (NormProblem, [_P] * 7),
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
    """Call an entry point of include/kda_ssm.h with raw integer pointers
    (0 for NULL), in the header's order; returns the status."""
    return _fn(name)(ctypes.byref(problem), *args)


def ssm_workspace_size(problem: SsmProblem) -> int:
    n = ctypes.c_size_t(0)
    _check(_fn("kda_ssm_prefill_workspace_size")(ctypes.byref(problem), ctypes.byref(n)),
           "kda_ssm_prefill_workspace_size")
    return int(n.value)


def ssm_plan(problem: SsmProblem) -> int:
    """The piece length kda_ssm_prefill takes for this problem (0: no split)."""
    n = _i32(0)
    _check(_fn("kda_ssm_plan")(ctypes.byref(problem), ctypes.byref(n)), "kda_ssm_plan")
    return int(n.value)


def _row_stride(name: str, t, lead: int) -> int:
    """Elements between a tensor's rows: `lead` leading dimensions count rows
    with one stride, the others are packed.  0 stands for packed rows."""
    if t.is_contiguous():
        return 0
    shape, stride = t.shape, t.stride()
    want = 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if shape[i] != 1 and stride[i] != want:
            raise ValueError(f"{name}: the last {t.dim() - lead} dimensions must be contiguous")
        want *= shape[i]
    step = span = 0
    for i in range(lead - 1, -1, -1):
        if shape[i] == 1:
            continue
        if span and stride[i] != span:
            raise ValueError(f"{name}: rows must have one stride")
        if not span:
            step = stride[i]
            if step <= 0:
                raise ValueError(f"{name}: rows must have a positive stride")
            span = step
        span *= shape[i]
    return step


def _check_tensor(name: str, t, dtype, shape, dev, contiguous: bool = True):
    """dtype, device, shape and packing of a tensor (None passes)."""
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _gpu(t, stream):
    if not t.is_cuda:
        raise ValueError("libkda runs on the GPU: tensors must be on a cuda (HIP) device")
    dev = t.device
    if stream is not None:
        _check_stream(stream, dev)
    return dev


def _like(x, stream, dtype=None):
    """A packed tensor of x's shape (about 1 us cheaper than one from a shape)."""
    import torch

    if stream is None:
        return torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)
    with torch.cuda.stream(stream):
        return torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)


def _new(x, stream, shape, dtype):
    import torch

    if stream is None:
        return x.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return x.new_empty(shape, dtype=dtype)


def _launch(name: str, dev, stream, problem, args, mine=(), call=call_raw):
    """Enqueue on `stream` (None: the current one).  Buffers of the binding's own
    come out of that stream's part of torch's allocator: from the current stream's
    a block could be one that work queued there still uses.  Results (`mine`) are
    read on the current stream next, and freed there: the allocator is told, so
    that a later call on `stream` does not get them early."""
    import torch

    current = torch._C._cuda_getCurrentRawStream(dev.index)
    raw = current if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev.index:
        status = call(name, problem, *args, raw)
    else:
        with torch.cuda.device(dev):
            status = call(name, problem, *args, raw)
    if raw != current:
        here = torch.cuda.current_stream(dev)
        for t in mine:
            t.record_stream(here)
    if status:
        _check(status, name)


def _activation(name) -> int:
    kind = ACTIVATIONS.get(name)
    if kind is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}")
    return kind


def _offsets(cu_seqlens, dev):
    import torch

    if cu_seqlens is None:
        return 0
    if cu_seqlens.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"cu_seqlens must be int32 or int64, got {cu_seqlens.dtype}")
    if cu_seqlens.device != dev or not cu_seqlens.is_contiguous() or cu_seqlens.dim() != 1 \
            or cu_seqlens.numel() < 2:
        raise ValueError(f"cu_seqlens must be contiguous [N + 1] on {dev}")
    return int(cu_seqlens.dtype == torch.int64)


def _batch(x, inner: int, cu_seqlens, what: str):
    """(leading dimensions, sequences, tokens) of a packed [T, ...] or fixed
    [B, T, ...] input with `inner` dimensions per token."""
    shape = x.shape
    if len(shape) == inner + 2:
        if cu_seqlens is not None:
            raise ValueError("cu_seqlens is for packed inputs")
        return 2, shape[0], shape[0] * shape[1]
    if len(shape) != inner + 1:
        raise ValueError(f"x must be {what}")
    return 1, 1 if cu_seqlens is None else cu_seqlens.numel() - 1, shape[0]


def conv_prefill(x, weight, bias=None, *, cu_seqlens=None, initial_state=None, final_state=None,
                 output_final_state: bool = True, activation: str = "silu", out=None, stream=None):
    """Short causal convolution over prompts, depthwise.

    x: bf16 [T, D] (packed, with cu_seqlens int32 or int64 [N + 1]) or
    [B, T, D], rows may be strided (columns of a wider row).  weight: bf16
    [D, W], W = 2..4; bias: bf16 [D] or None.  initial_state: bf16
    [N, W - 1, D], the rows ahead of each sequence, oldest first (None:
    zeros).  activation: "silu" or "none".  Returns (out, final_state);
    final_state is the last W - 1 rows of each sequence, its state included,
    and None with output_final_state=False.  final_state=initial_state updates
    in place; out must not be x.  (For ``prefill``, whose q, k and v are packed: a
    call for each one's columns of a projection's row gives packed results.)"""
    import torch

    dev = _gpu(x, stream)
    bf = torch.bfloat16
    lead, N, T = _batch(x, 1, cu_seqlens, "[T, D] or [B, T, D]")
    shape = x.shape
    D, W = shape[-1], weight.shape[-1]
    state = (N, W - 1, D)
    _check_tensor("x", x, bf, shape, dev, False)
    _check_tensor("weight", weight, bf, (D, W), dev)
    _check_tensor("bias", bias, bf, (D,), dev)
    _check_tensor("initial_state", initial_state, bf, state, dev)
    _check_tensor("final_state", final_state, bf, state, dev)
    _check_tensor("out", out, bf, shape, dev, False)
    cu64 = _offsets(cu_seqlens, dev)
    mine = []
    if out is None:
        out = _like(x, stream)
        mine.append(out)
    if final_state is None and output_final_state:
        final_state = _new(x, stream, state, bf)
        mine.append(final_state)
    p = ConvProblem(N, T, D, W, _activation(activation), cu64, _row_stride("x", x, lead),
                    _row_stride("out", out, lead))
    _launch("kda_conv_prefill", dev, stream, p,
            [_ptr(x), _ptr(weight), _ptr(bias), _ptr(cu_seqlens), _ptr(initial_state), _ptr(out),
             _ptr(final_state)], mine)
    return out, final_state


def conv_decode(x, weight, bias, state_pool, state_indices, *, activation: str = "silu", out=None, stream=None):
    """Short causal convolution for T tokens of each of N requests.

    x: bf16 [N, T, D] (rows may be strided); state_pool: bf16 [P, W - 1, D],
    updated in place; state_indices: int32 [N], entries outside [0, P) mark
    empty slots (zero outputs, no state touched).  Returns out (``out=x``
    overwrites x)."""
    import torch

    dev = _gpu(x, stream)
    bf = torch.bfloat16
    if x.dim() != 3 or state_pool.dim() != 3:
        raise ValueError("x must be [N, T, D] and state_pool [P, W - 1, D]")
    shape, size = x.shape, state_pool.shape[0]
    N, T, D = shape
    W = weight.shape[-1]
    _check_tensor("x", x, bf, shape, dev, False)
    _check_tensor("weight", weight, bf, (D, W), dev)
    _check_tensor("bias", bias, bf, (D,), dev)
    _check_tensor("state_pool", state_pool, bf, (size, W - 1, D), dev)
    _check_tensor("state_indices", state_indices, torch.int32, (N,), dev)
    _check_tensor("out", out, bf, shape, dev, False)
    mine = []
    if out is None:
        out = _like(x, stream)
        mine.append(out)
    p = ConvDecodeProblem(N, T, D, W, _activation(activation), size,
                          _row_stride("x", x, 2), _row_stride("out", out, 2))
    _launch("kda_conv_decode", dev, stream, p,
            [_ptr(x), _ptr(weight), _ptr(bias), _ptr(state_pool), _ptr(state_indices), _ptr(out)], mine)
    return out


def _ssm_tokens(x, dt, A, B, C, D, z, dt_bias, out, lead, stream):
    """Checks what the scan's two forms share; returns (H, G, P, N)."""
    import torch

    dev = _gpu(x, stream)
    bf, f32 = torch.bfloat16, torch.float32
    shape = x.shape
    tok, (H, P) = shape[:lead], shape[lead:]
    if B.dim() != lead + 2:
        raise ValueError("B and C must be x.shape[:-2] + (G, N)")
    G, N = B.shape[lead:]
    _check_tensor("x", x, bf, shape, dev, False)
    _check_tensor("dt", dt, f32, tok + (H,), dev)
    _check_tensor("A", A, f32, (H,), dev)
    _check_tensor("B", B, bf, tok + (G, N), dev, False)
    _check_tensor("C", C, bf, B.shape, dev, False)
    _check_tensor("D", D, f32, (H,), dev)
    _check_tensor("z", z, bf, shape, dev, False)
    _check_tensor("dt_bias", dt_bias, f32, (H,), dev)
    _check_tensor("out", out, bf, shape, dev, False)
    return H, G, P, N


def _state_dtype(dtype) -> int:
    import torch

    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("states must be float32 or bfloat16")
    return STATE_DTYPES["bf16" if dtype == torch.bfloat16 else "fp32"]


def ssm_prefill(x, dt, A, B, C, *, D=None, z=None, dt_bias=None, dt_softplus: bool = False, cu_seqlens=None,
                initial_state=None, final_state=None, output_final_state: bool = True, out=None,
                state_dtype=None, workspace=None, piece_tokens: int = 0, stream=None):
    """Selective state space scan over prompts, one decay per head.

    x (and the gate z): bf16 [T, H, P] (packed, with cu_seqlens int32 or int64
    [N + 1]) or [B, T, H, P]; B, C: bf16 [T, G, S] likewise, G dividing H; rows
    may be strided (columns of one wider row).  P and S are 64 or 128.  dt:
    fp32 [T, H], plus dt_bias [H], through softplus with dt_softplus.  A: fp32
    [H], negative.  D: fp32 [H], the skip term, or None.  States: fp32 or bf16
    [N, H, S, P] (initial_state None: zeros); final_state=initial_state
    updates in place.  workspace: a buffer of ``ssm_workspace_size`` bytes; when
    None one is taken from torch's allocator if the scan runs in pieces.
    Returns (out, final_state); final_state is None with
    output_final_state=False."""
    import torch

    lead, N, T = _batch(x, 2, cu_seqlens, "[T, H, P] or [B, T, H, P]")
    H, G, P, S = _ssm_tokens(x, dt, A, B, C, D, z, dt_bias, out, lead, stream)
    dev = x.device
    if state_dtype is None:
        given = initial_state if initial_state is not None else final_state
        state_dtype = torch.float32 if given is None else given.dtype
    kind = _state_dtype(state_dtype)
    shape = (N, H, S, P)
    _check_tensor("initial_state", initial_state, state_dtype, shape, dev)
    _check_tensor("final_state", final_state, state_dtype, shape, dev)
    cu64 = _offsets(cu_seqlens, dev)
    mine = []
    if out is None:
        out = _like(x, stream)
        mine.append(out)
    if final_state is None and output_final_state:
        final_state = _new(x, stream, shape, state_dtype)
        mine.append(final_state)
    p = SsmProblem(N, T, H, G, P, S, int(dt_softplus), kind, cu64, int(piece_tokens),
                   int(cu_seqlens is not None), _row_stride("x", x, lead),
                   _row_stride("B", B, lead), _row_stride("C", C, lead),
                   0 if z is None else _row_stride("z", z, lead), _row_stride("out", out, lead))
    if workspace is None:
        # (short sequences are never split unless asked for: not worth a call)
        need = ssm_workspace_size(p) if piece_tokens or T > SPLIT_TOKENS * N else 0
        if need:
            workspace = _new(x, stream, (need,), torch.uint8)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}")
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _launch("kda_ssm_prefill", dev, stream, p,
            [_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(cu_seqlens),
             _ptr(initial_state), _ptr(out), _ptr(final_state), _ptr(workspace), size], mine)
    return out, final_state


def ssm_decode(x, dt, A, B, C, state_pool, state_indices, *, D=None, z=None, dt_bias=None,
               dt_softplus: bool = False, out=None, stream=None):
    """Selective state space scan for T tokens of each of N requests.

    x (and z): bf16 [N, T, H, P]; B, C: bf16 [N, T, G, S]; dt: fp32 [N, T, H];
    state_pool: fp32 or bf16 [pool, H, S, P], updated in place; state_indices:
    int32 [N], entries outside the pool mark empty slots (zero outputs, no
    state touched).  The rest as for ssm_prefill.  Returns out (``out=x``
    overwrites x)."""
    import torch

    if x.dim() != 4:
        raise ValueError("x must be [N, T, H, P]")
    H, G, P, S = _ssm_tokens(x, dt, A, B, C, D, z, dt_bias, out, 2, stream)
    dev = x.device
    N, T = x.shape[:2]
    kind = _state_dtype(state_pool.dtype)
    if state_pool.dim() != 4:
        raise ValueError(f"state_pool must be [pool, {H}, {S}, {P}]")
    size = state_pool.shape[0]
    _check_tensor("state_pool", state_pool, state_pool.dtype, (size, H, S, P), dev)
    _check_tensor("state_indices", state_indices, torch.int32, (N,), dev)
    mine = []
    if out is None:
        out = _like(x, stream)
        mine.append(out)
    p = SsmDecodeProblem(N, T, H, G, P, S, int(dt_softplus), kind, size,
                         _row_stride("x", x, 2), _row_stride("B", B, 2), _row_stride("C", C, 2),
                         0 if z is None else _row_stride("z", z, 2), _row_stride("out", out, 2))
    _launch("kda_ssm_decode", dev, stream, p,
            [_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(state_pool),
             _ptr(state_indices), _ptr(out)], mine)
    return out


def add_rmsnorm(x, weight, *, residual=None, eps: float = 1e-6, out_dtype=None, scale_group: int = 0, out=None,
                scales=None, residual_out=None, stream=None):
    """RMS norm over the last dimension, of x or of x + residual.

    x: bf16 [..., D] (rows may be strided), residual: bf16 like x or None,
    weight: bf16 [D].  out_dtype: torch.bfloat16 (default) or
    torch.float8_e4m3fn, then with an fp32 scale per row (scale_group=0) or per
    128 columns (scale_group=128).  residual_out: None allocates bf16(x +
    residual), False leaves it out, a tensor (``residual`` itself for an
    update in place) takes it.  Returns (out, residual_out or None, scales or
    None); scales are [..., 1] or [..., ceil(D / 128)]."""
    import torch

    dev = _gpu(x, stream)
    bf = torch.bfloat16
    shape = x.shape
    D = shape[-1]
    if out_dtype is None:
        out_dtype = bf if out is None else out.dtype
    if out_dtype not in (bf, torch.float8_e4m3fn):
        raise TypeError("out_dtype must be bfloat16 or float8_e4m3fn")
    fp8 = out_dtype != bf
    if residual is None and residual_out is not None and residual_out is not False:
        raise ValueError("residual_out needs a residual")
    if not fp8 and (scales is not None or scale_group):
        raise ValueError("scales are for a float8_e4m3fn output")
    groups = shape[:-1] + ((D + 127) // 128 if scale_group else 1,) if fp8 else None
    mine = []
    if residual is None or residual_out is False:
        residual_out = None
    elif residual_out is None:
        residual_out = _like(x, stream)
        mine.append(residual_out)
    if out is None:
        out = _like(x, stream, out_dtype)
        mine.append(out)
    if fp8 and scales is None:
        scales = _new(x, stream, groups, torch.float32)
        mine.append(scales)
    _check_tensor("x", x, bf, shape, dev, False)
    _check_tensor("residual", residual, bf, shape, dev)
    _check_tensor("weight", weight, bf, (D,), dev)
    _check_tensor("out", out, out_dtype, shape, dev)
    _check_tensor("scales", scales, torch.float32, groups, dev)
    _check_tensor("residual_out", residual_out, bf, shape, dev)
    p = NormProblem(x.numel() // D if D else 0, D, float(eps), int(fp8), int(scale_group),
                    _row_stride("x", x, x.dim() - 1))
    _launch("kda_add_rmsnorm", dev, stream, p,
            [_ptr(x), _ptr(residual), _ptr(weight), _ptr(out), _ptr(scales), _ptr(residual_out)], mine)
    return out, residual_out, scales
