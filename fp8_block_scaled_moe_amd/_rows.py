"""Binding of include/moe_rows.h: the routed-expert step for any number of
tokens, as separate calls.

Argument checks and marshalling only. Every call allocates its outputs (and
all but the norm a workspace where one is needed) from torch's caching
allocator and launches on the current stream of the tensors' device, or on
`stream` when one is given; it never synchronises, so it can be captured into
a graph. With `stream`, as under torch.cuda.stream, the outputs are that
stream's: its work has to be behind what wrote the inputs, and whoever reads the
outputs on another stream waits for it and records them there. The inputs are
recorded on it by the call.
"""

from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from ._capi import DTYPE_BF16, DTYPE_F32, MoeDecodeError, OK, _FP8, _need, lib

QUANT = {None: 0, "fp8": 1, "fp8_p2": 2, "mxfp8": 3}
SUMS = {"fp32": 0, "fp8": 1}
ROWS_MAX_D = 16384
ROWS_MAX_TOKENS = 1048576
_I32_MAX = 2**31 - 1  # sizes are 32-bit integers in the C ABI

_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_U8 = (torch.uint8, torch.float8_e8m0fnu)
_vp, _i32, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float


class NormArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("D", _i32), ("k", _i32), ("R", _i32), ("eps", _f32), ("quant", _i32),
                ("residual", _vp), ("delta", _vp), ("y", _vp), ("pos", _vp), ("weights", _vp), ("gamma", _vp),
                ("residual_out", _vp), ("out", _vp), ("q", _vp), ("scale", _vp)]


class RouteArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("E", _i32), ("k", _i32), ("logits_dtype", _i32), ("local_begin", _i32),
                ("local_experts", _i32), ("routed_scale", _f32), ("logits", _vp), ("bias", _vp), ("ids", _vp),
                ("weights", _vp), ("offsets", _vp), ("rows", _vp), ("pos", _vp), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t)]


class GroupedArgs(ctypes.Structure):
    _fields_ = [("R", _i32), ("X", _i32), ("E", _i32), ("N", _i32), ("K", _i32), ("quant", _i32),
                ("limit", _f32), ("x", _vp), ("x_scale", _vp), ("rows", _vp),
                ("offsets", _vp), ("w", _vp), ("w_scale", _vp), ("out", _vp), ("out_scale", _vp), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t), ("sums", _i32)]


class RoutedRows(NamedTuple):
    """ids, weights and pos are [T, top_k]; offsets [local experts + 1]; rows
    [T * top_k], of which the first offsets[-1] are written."""
    ids: torch.Tensor
    weights: torch.Tensor
    offsets: torch.Tensor
    rows: torch.Tensor
    pos: torch.Tensor


def _arg(t, name, dtypes, dev, shape, align=16) -> int:
    """The tensor's address, after the checks of _need (repeated there for
    its message)."""
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and t.device == dev
            and t.is_contiguous()):
        p = t.data_ptr()
        if p % align == 0:
            return p
    _need(t, name, dtypes, dev, align=align, shape=shape)
    return t.data_ptr()


def _on_gpu(dev: torch.device) -> None:
    if dev.type != "cuda":
        raise ValueError(f"the tensors must be on a GPU, got {dev}")


@contextlib.contextmanager
def _place(dev, stream, inputs):
    """Makes dev, and stream if one is given, current; `inputs` are recorded on
    that stream, so that their memory is not handed out anew before it is
    through with them."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(stream, device=dev)
            if stream.device != dev:
                raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
            with torch.cuda.stream(stream):
                yield
            for t in inputs:
                if t is not None:
                    t.record_stream(stream)


class _Here:
    """No change of device or stream."""

    def __enter__(self):
        return None

    def __exit__(self, *_):
        return False


_here = _Here()


def _where(dev, stream, *inputs):
    _on_gpu(dev)
    return _here if stream is None and dev.index == torch.cuda.current_device() else _place(dev, stream, inputs)


# The current stream's handle without an object around it, where this torch
# has it (1.8 us less per call, of some 13).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(name, args, dev) -> None:
    rc = getattr(lib(), name)(ctypes.byref(args), _raw_stream(dev.index))
    if rc != OK:
        raise MoeDecodeError(rc, name)


def add_rmsnorm_quant(residual: Optional[torch.Tensor], gamma: Optional[torch.Tensor], eps: float = 1e-5, *,
                      delta: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                      pos: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                      quant: Optional[str] = "fp8", want_residual: bool = True, want_out: bool = True,
                      inplace: bool = False, stream=None):
    """(residual_out, out, q, scale) of h = residual + delta + sum_j
    weights[t, j] y[pos[t, j]] and its RMSNorm (include/moe_rows.h).

    residual, delta [T, D] BF16; y [R, D] BF16 with pos [T, k] int32 and
    weights [T, k] FP32 (route_rows); gamma [D] BF16, None for no
    normalisation. Any of residual, delta and the routed rows may be absent,
    not all. quant: "fp8" (q [T, D] uint8 codes, scale [T, D/128] FP32),
    "fp8_p2" (power-of-two scales), "mxfp8" (scale [T, D/32] E8M0 bytes) or
    None (q and scale None). residual_out and out are BF16, None when not
    wanted. inplace: residual_out is `residual` itself, updated."""
    if quant not in QUANT:
        raise ValueError(f"quant must be one of {list(QUANT)}, got {quant!r}")
    like = residual if residual is not None else delta
    if like is not None:
        if not isinstance(like, torch.Tensor) or like.dim() != 2:
            raise ValueError("residual and delta must be [T, D] tensors")
        T, D = like.shape
    elif y is not None and pos is not None:
        like = y
        if not isinstance(y, torch.Tensor) or y.dim() != 2 or not isinstance(pos, torch.Tensor) or pos.dim() != 2:
            raise ValueError("y must be [R, D] and pos [T, k]")
        T, D = pos.shape[0], y.shape[1]
    else:
        raise ValueError("at least one of residual, delta and routed rows (y, pos, weights) is needed")
    if inplace and (residual is None or not want_residual):
        raise ValueError("inplace needs a residual to update")
    if T > ROWS_MAX_TOKENS:
        raise ValueError(f"at most {ROWS_MAX_TOKENS} tokens, got {T}")
    dev = like.device
    rp = None if residual is None else _arg(residual, "residual", _BF16, dev, (T, D))
    dp = None if delta is None else _arg(delta, "delta", _BF16, dev, (T, D))
    gp = None if gamma is None else _arg(gamma, "gamma", _BF16, dev, (D,))
    yp = pp = wp = None
    k = R = 0
    if y is not None or pos is not None or weights is not None:
        if not isinstance(y, torch.Tensor) or y.dim() != 2 or not isinstance(pos, torch.Tensor) or pos.dim() != 2:
            raise ValueError("routed rows need y [R, D], pos [T, k] and weights [T, k]")
        R, k = y.shape[0], pos.shape[1]
        if R > _I32_MAX:
            raise ValueError(f"y has {R} rows, at most 2^31 - 1 are supported")
        yp = _arg(y, "y", _BF16, dev, (R, D))
        pp = _arg(pos, "pos", _I32, dev, (T, k), 4)
        wp = _arg(weights, "weights", _F32, dev, (T, k), 4)
        if k == 0 or (R == 0 and T > 0):
            raise ValueError("routed rows must not be empty")
    unit = 8 if quant is None else 32 if quant == "mxfp8" else 128
    if D % unit or not 0 < D <= ROWS_MAX_D or k > 32:
        raise ValueError(f"D must be a multiple of {unit} up to {ROWS_MAX_D} and top_k at most 32, got D={D}, k={k}")
    if not (want_residual or want_out or quant is not None):
        raise ValueError("no output is wanted")
    with _where(dev, stream, residual, gamma, delta, y, pos, weights):
        if like.shape == (T, D):
            new = lambda dtype: torch.empty_like(like, dtype=dtype)  # noqa: E731
        else:
            new = lambda dtype: like.new_empty((T, D), dtype=dtype)  # noqa: E731
        res = (residual if inplace else new(torch.bfloat16)) if want_residual else None
        out = new(torch.bfloat16) if want_out else None
        q = scale = None
        if quant is not None:
            q = new(torch.uint8)
            scale = (like.new_empty((T, D // 32), dtype=torch.uint8) if quant == "mxfp8"
                     else like.new_empty((T, D // 128), dtype=torch.float32))
        if T:
            _call("moe_add_rmsnorm_quant",
                  NormArgs(T, D, k, R, eps, QUANT[quant], rp, dp, yp, pp, wp, gp, None if res is None else res.data_ptr(),
                           None if out is None else out.data_ptr(), None if q is None else q.data_ptr(),
                           None if scale is None else scale.data_ptr()), dev)
    return res, out, q, scale


def route_rows(logits: torch.Tensor, bias: torch.Tensor, *, top_k: int, routed_scale: float, local_begin: int = 0,
               local_experts: Optional[int] = None, stream=None) -> RoutedRows:
    """Biased sigmoid top-k of logits [T, E] (FP32 or BF16) with bias [E]
    FP32, and the tokens grouped by expert (include/moe_rows.h)."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a [T, E] tensor")
    T, E = logits.shape
    if T > ROWS_MAX_TOKENS:
        raise ValueError(f"at most {ROWS_MAX_TOKENS} tokens, got {T}")
    dev = logits.device
    lp = _arg(logits, "logits", (torch.float32, torch.bfloat16), dev, (T, E), 2 if logits.dtype == torch.bfloat16 else 4)
    bp = _arg(bias, "bias", _F32, dev, (E,), 4)
    El = E - local_begin if local_experts is None else local_experts
    if not 1 <= E <= 1024 or not 1 <= top_k <= min(E, 32):
        raise ValueError(f"1 <= E <= 1024 and 1 <= top_k <= min(E, 32) are needed, got E={E}, top_k={top_k}")
    if not (local_begin >= 0 and El >= 1 and local_begin + El <= E):
        raise ValueError(f"local experts [{local_begin}, {local_begin + El}) must lie in [0, {E})")
    with _where(dev, stream, logits, bias):
        ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        pos, weights = torch.empty_like(ids), torch.empty_like(ids, dtype=torch.float32)
        offsets, rows = ids.new_empty(El + 1), ids.new_empty(T * top_k)
        need = lib().moe_route_rows_workspace(T, El)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _call("moe_route_rows",
              RouteArgs(T, E, top_k, DTYPE_BF16 if logits.dtype == torch.bfloat16 else DTYPE_F32, local_begin, El,
                        routed_scale, lp, bp, ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(),
                        pos.data_ptr(), None if ws is None else ws.data_ptr(), need), dev)
    return RoutedRows(ids, weights, offsets, rows, pos)


def _grouped(x, x_scale, w, w_scale, offsets, rows):
    """Checks shared by the grouped products: (dev, R, X, E, N, K, quant and
    the addresses in GroupedArgs order)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be an [X, K] tensor")
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must be an [E, N, K] tensor")
    X, K = x.shape
    E, N, dev = w.shape[0], w.shape[1], x.device
    if K < 128 or K % 128 or N < 128 or N % 128 or not 1 <= E <= 1024:
        raise ValueError(f"K and N must be multiples of 128 and 1 <= E <= 1024, got E={E}, N={N}, K={K}")
    if not isinstance(x_scale, torch.Tensor):
        raise ValueError("x_scale must be a tensor")
    if rows is not None and (not isinstance(rows, torch.Tensor) or rows.dim() != 1):
        raise ValueError("rows must be an [R] tensor")
    if max(X, N, K, 0 if rows is None else rows.shape[0]) > _I32_MAX:
        raise ValueError("rows and columns are limited to 2^31 - 1")
    mx = x_scale.dtype != torch.float32
    xp = _arg(x, "x", _FP8, dev, (X, K))
    sp = _arg(x_scale, "x_scale", _U8 if mx else _F32, dev, (X, K // 32 if mx else K // 128), 4)
    wp = _arg(w, "w", _FP8, dev, (E, N, K))
    wsp = _arg(w_scale, "w_scale", _F32, dev, (E, N // 128, K // 128), 4)
    op = _arg(offsets, "offsets", _I32, dev, (E + 1,), 4)
    rp, R = None, X
    if rows is not None:
        R = rows.shape[0]
        rp = _arg(rows, "rows", _I32, dev, (R,), 4)
        if R and not X:
            raise ValueError("x has no rows to gather")
    return dev, R, (R, X, E, N, K, QUANT["mxfp8" if mx else "fp8"]), (xp, sp, rp, op, wp, wsp)


def grouped_gemm(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, offsets: torch.Tensor,
                 *, rows: Optional[torch.Tensor] = None, sums: str = "fp32", stream=None) -> torch.Tensor:
    """[R, N] BF16 product of every expert with its own rows (include/moe_rows.h):
    grouped row i of expert e (offsets[e] <= i < offsets[e + 1]) is
    x[rows[i]] (x[i] without rows) times w[e]^T.

    x [X, K] e4m3 codes (uint8 or float8_e4m3fn) with x_scale [X, K/128] FP32
    or, for MXFP8, [X, K/32] E8M0 bytes (uint8 or float8_e8m0fnu); w [E, N, K]
    e4m3 with w_scale [E, N/128, K/128] FP32. Rows from offsets[E] on are left
    unwritten. sums: "fp32", or "fp8" for the faster and coarser ones of the
    FP8 matrix instruction."""
    if sums not in SUMS:
        raise ValueError(f"sums must be one of {list(SUMS)}, got {sums!r}")
    dev, R, sizes, ptrs = _grouped(x, x_scale, w, w_scale, offsets, rows)
    with _where(dev, stream, x, x_scale, w, w_scale, offsets, rows):
        out = torch.empty((R, sizes[3]), dtype=torch.bfloat16, device=dev)
        if R:
            need = lib().moe_grouped_gemm_workspace(R, *sizes[2:5])
            ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
            _call("moe_grouped_gemm", GroupedArgs(*sizes, 0.0, *ptrs, out.data_ptr(), None,
                                                  None if ws is None else ws.data_ptr(), need, SUMS[sums]), dev)
    return out


def grouped_swiglu(x: torch.Tensor, x_scale: torch.Tensor, w13: torch.Tensor, w13_scale: torch.Tensor,
                   offsets: torch.Tensor, *, limit: float, rows: Optional[torch.Tensor] = None, stream=None):
    """(h [R, I] e4m3 codes uint8, h_scale [R, I/128] FP32): the clamped
    SwiGLU of every expert's up and gate products with its own rows, in 8 bits
    (include/moe_rows.h). w13 [E, 2I, K], rows 0..I-1 up, I..2I-1 gate; the
    other arguments as grouped_gemm's."""
    dev, R, sizes, ptrs = _grouped(x, x_scale, w13, w13_scale, offsets, rows)
    if sizes[3] % 256:
        raise ValueError(f"w13 must hold 2I rows with I a multiple of 128, got {sizes[3]}")
    if not limit > 0:
        raise ValueError(f"limit must be positive, got {limit}")
    I = sizes[3] // 2
    with _where(dev, stream, x, x_scale, w13, w13_scale, offsets, rows):
        h = torch.empty((R, I), dtype=torch.uint8, device=dev)
        scale = torch.empty((R, I // 128), dtype=torch.float32, device=dev)
        if R:
            need = lib().moe_grouped_swiglu_workspace(R, *sizes[2:5])
            ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
            _call("moe_grouped_swiglu", GroupedArgs(*sizes, limit, *ptrs, h.data_ptr(), scale.data_ptr(),
                                                    None if ws is None else ws.data_ptr(), need), dev)
    return h, scale
