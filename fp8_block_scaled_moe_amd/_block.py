"""Binding of include/moe_block.h: what stands around the routed experts in a
layer, for any number of tokens.

Argument checks and marshalling only, in the manner of _rows.py: outputs and
workspaces come from torch's caching allocator, calls launch on the current
stream of the tensors' device, or on `stream` when one is given, and never
synchronise, so they can be captured into a graph.
"""

from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional

import torch

from ._capi import DTYPE_BF16, DTYPE_F32, lib
from ._rows import (QUANT, ROWS_MAX_D, ROWS_MAX_TOKENS, NormArgs, RouteArgs, RoutedRows, _BF16, _F32, _I32, _I32_MAX, _arg,
                    _call, _where)

ACTS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "sigmoid": 5}
SCORES = {"sigmoid": 0, "softmax": 1}
GATE_NONE, GATE_ROW, GATE_COLUMN, GATE_FULL = range(4)
DENSE_MAX_DIM = 1048576
DENSE_MAX_STRIDE = 2**23  # of rows of x, w and the residual, in values
ROUTE_MAX_GROUPS = 64

_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
_FLOATS = (torch.float32, torch.bfloat16)
_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class DenseArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("N", _i32), ("K", _i32), ("act", _i32), ("out_dtype", _i32), ("bias_dtype", _i32),
                ("residual_dtype", _i32), ("ldx", _i64), ("ldw", _i64), ("ldr", _i64), ("x", _vp), ("w", _vp), ("bias", _vp),
                ("residual", _vp), ("out", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class RouteScoredArgs(ctypes.Structure):
    _fields_ = [("route", RouteArgs), ("scores", _i32), ("groups", _i32), ("top_groups", _i32), ("group_best", _i32),
                ("renormalise", _i32)]


class JoinArgs(ctypes.Structure):
    _fields_ = [("norm", NormArgs), ("post_eps", _f32), ("residual_scale", _f32), ("gamma_offset", _f32), ("gate_kind", _i32),
                ("gate_dtype", _i32), ("post_gamma", _vp), ("gate", _vp)]


def _matrix(t, name, dtypes, dev, shape, unit):
    """(address, row stride) of a matrix whose rows are contiguous, `unit`
    values between row starts and 2 * unit (BF16) bytes their alignment."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and t.device == dev and t.is_contiguous():
        p = t.data_ptr()  # the usual case, without what the others are told
        if p % 16 == 0:
            return p, shape[1]
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    rows, columns = shape
    ld, step = t.stride()
    if columns > 1 and step != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if rows > 1 and (ld < columns or ld % unit):
        raise ValueError(f"the rows of {name} must not overlap and lie a multiple of {unit} values apart, got {ld}")
    if rows > 1 and ld >= DENSE_MAX_STRIDE:
        raise ValueError(f"the rows of {name} must lie less than 2^23 values apart, got {ld}")
    p = t.data_ptr()
    align = 16 if unit > 1 else t.element_size()
    if p % align:
        raise ValueError(f"{name} must start on a {align}-byte boundary")
    return p, ld if rows > 1 else columns


@functools.lru_cache(maxsize=4096)
def _dense_workspace(T, N, K) -> int:
    return lib().moe_dense_gemm_workspace(T, N, K)


def dense_gemm(x: torch.Tensor, w: torch.Tensor, *, bias: Optional[torch.Tensor] = None, act: Optional[str] = None,
               residual: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """[T, N] = act(x w^T + bias) + residual (include/moe_block.h).

    x [T, K] and w [N, K] BF16 (K a multiple of 8), bias [N] and residual
    [T, N] BF16 or FP32; rows of x, w and residual contiguous, those of x and
    w a multiple of 8 values apart (columns of a wider matrix will do). act:
    "relu", "silu", "gelu", "gelu_tanh", "sigmoid" or None. Sums, bias,
    activation and residual in FP32, rounded once to out_dtype (BF16 or FP32:
    a router's logits)."""
    if act not in ACTS:
        raise ValueError(f"act must be one of {list(ACTS)}, got {act!r}")
    if out_dtype not in _DTYPES:
        raise ValueError(f"out_dtype must be torch.bfloat16 or torch.float32, got {out_dtype}")
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("x must be a [T, K] and w an [N, K] tensor")
    T, K = x.shape
    N, dev = w.shape[0], x.device
    if T > ROWS_MAX_TOKENS:
        raise ValueError(f"at most {ROWS_MAX_TOKENS} rows, got {T}")
    if K % 8 or not 8 <= K <= DENSE_MAX_DIM or not 1 <= N <= DENSE_MAX_DIM:
        raise ValueError(f"K must be a multiple of 8, N and K at most {DENSE_MAX_DIM}, got N={N}, K={K}")
    xp, ldx = _matrix(x, "x", _BF16, dev, (T, K), 8)
    wp, ldw = _matrix(w, "w", _BF16, dev, (N, K), 8)
    bp = rp = None
    bias_dtype = residual_dtype = 0
    ldr = N
    if bias is not None:
        bp = _arg(bias, "bias", _FLOATS, dev, (N,), 2 if getattr(bias, "dtype", None) == torch.bfloat16 else 4)
        bias_dtype = _DTYPES[bias.dtype]
    if residual is not None:
        rp, ldr = _matrix(residual, "residual", _FLOATS, dev, (T, N), 1)
        residual_dtype = _DTYPES[residual.dtype]
    with _where(dev, stream, x, w, bias, residual):
        out = torch.empty((T, N), dtype=out_dtype, device=dev)
        if T:
            need = _dense_workspace(T, N, K)
            ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
            _call("moe_dense_gemm",
                  DenseArgs(T, N, K, ACTS[act], _DTYPES[out_dtype], bias_dtype, residual_dtype, ldx, ldw, ldr, xp, wp, bp, rp,
                            out.data_ptr(), None if ws is None else ws.data_ptr(), need), dev)
    return out


def route_rows_scored(logits: torch.Tensor, bias: Optional[torch.Tensor] = None, *, top_k: int, routed_scale: float = 1.0,
                      scores: str = "sigmoid", groups: int = 1, top_groups: Optional[int] = None, group_best: Optional[int] = None,
                      renormalise: bool = True, local_begin: int = 0, local_experts: Optional[int] = None,
                      stream=None) -> RoutedRows:
    """Top-k of logits [T, E] (FP32 or BF16) by sigmoid or softmax scores plus
    bias [E] FP32 (or None), and the tokens grouped by expert as route_rows
    gives them (include/moe_block.h).

    Of `groups` equal runs of experts the top_groups (None: all) with the
    largest values take part: a group's value is its largest key (group_best =
    1) or the sum of its two largest (2; None: 2 where a group has two experts).
    Weights are the picked scores, without the bias, over their sum
    (renormalise) or as they are, times routed_scale."""
    if scores not in SCORES:
        raise ValueError(f"scores must be one of {list(SCORES)}, got {scores!r}")
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a [T, E] tensor")
    T, E = logits.shape
    if T > ROWS_MAX_TOKENS:
        raise ValueError(f"at most {ROWS_MAX_TOKENS} tokens, got {T}")
    dev = logits.device
    bf16 = logits.dtype == torch.bfloat16
    lp = _arg(logits, "logits", _FLOATS, dev, (T, E), 2 if bf16 else 4)
    bp = None if bias is None else _arg(bias, "bias", _F32, dev, (E,), 4)
    El = E - local_begin if local_experts is None else local_experts
    if not 1 <= E <= 1024 or not 1 <= top_k <= min(E, 32):
        raise ValueError(f"1 <= E <= 1024 and 1 <= top_k <= min(E, 32) are needed, got E={E}, top_k={top_k}")
    if not (local_begin >= 0 and El >= 1 and local_begin + El <= E):
        raise ValueError(f"local experts [{local_begin}, {local_begin + El}) must lie in [0, {E})")
    if not 1 <= groups <= ROUTE_MAX_GROUPS or E % groups:
        raise ValueError(f"groups must be a divisor of E up to {ROUTE_MAX_GROUPS}, got E={E}, groups={groups}")
    size = E // groups
    top = groups if top_groups is None else top_groups
    best = min(size, 2) if group_best is None else group_best
    if not 1 <= top <= groups or best not in (1, 2) or best > size:
        raise ValueError(f"1 <= top_groups <= groups and group_best 1 or 2, at most a group's experts, are needed, got "
                         f"top_groups={top}, groups={groups}, group_best={best}")
    if top_k > top * size:
        raise ValueError(f"top_k {top_k} picks do not fit {top} groups of {size} experts")
    if not math.isfinite(routed_scale):
        raise ValueError(f"routed_scale must be finite, got {routed_scale}")
    with _where(dev, stream, logits, bias):
        ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        pos, weights = torch.empty_like(ids), torch.empty_like(ids, dtype=torch.float32)
        offsets, rows = ids.new_empty(El + 1), ids.new_empty(T * top_k)
        need = lib().moe_route_rows_workspace(T, El)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _call("moe_route_rows_scored",
              RouteScoredArgs(RouteArgs(T, E, top_k, DTYPE_BF16 if bf16 else DTYPE_F32, local_begin, El, routed_scale, lp, bp,
                                        ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), pos.data_ptr(),
                                        None if ws is None else ws.data_ptr(), need),
                              SCORES[scores], groups, top, best, 1 if renormalise else 0), dev)
    return RoutedRows(ids, weights, offsets, rows, pos)


def join_rmsnorm_quant(residual: Optional[torch.Tensor], gamma: Optional[torch.Tensor], eps: float = 1e-5, *,
                       delta: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                       pos: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                       post_gamma: Optional[torch.Tensor] = None, post_eps: Optional[float] = None,
                       gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0, gamma_offset: float = 0.0,
                       quant: Optional[str] = "fp8", want_residual: bool = True, want_out: bool = True, inplace: bool = False,
                       stream=None):
    """(residual_out, out, q, scale) of h = residual_scale residual + gate n
    and its RMSNorm, where n is the block's output b = delta + sum_j weights[t,
    j] y[pos[t, j]], normalised with post_gamma (include/moe_block.h).

    residual, delta, y, pos, weights, gamma, quant, want_residual, want_out and
    inplace as in add_rmsnorm_quant; delta and the routed rows (y, pos, weights)
    may not both be absent. post_gamma [D] BF16, None for b as it is, with
    post_eps (None: eps). gate: [T] or [T, 1] FP32 or BF16 (one value for a
    token), [D] or [1, D] BF16 (for a column), [T, D] BF16, or None; where T is
    D, [T, 1] or [1, D] says which. gamma_offset is added to gamma and post_gamma (1.0 where they hold the distance from one)."""
    if quant not in QUANT:
        raise ValueError(f"quant must be one of {list(QUANT)}, got {quant!r}")
    routed = y is not None or pos is not None or weights is not None
    if routed and (not isinstance(y, torch.Tensor) or y.dim() != 2 or not isinstance(pos, torch.Tensor) or pos.dim() != 2):
        raise ValueError("routed rows need y [R, D], pos [T, k] and weights [T, k]")
    like = delta if delta is not None else y
    if like is None:
        raise ValueError("a block's output is needed: delta or routed rows (y, pos, weights)")
    if not isinstance(like, torch.Tensor) or like.dim() != 2:
        raise ValueError("delta must be a [T, D] tensor")
    T, D = pos.shape[0] if delta is None else delta.shape[0], like.shape[1]
    if inplace and (residual is None or not want_residual):
        raise ValueError("inplace needs a residual to update")
    if T > ROWS_MAX_TOKENS:
        raise ValueError(f"at most {ROWS_MAX_TOKENS} tokens, got {T}")
    dev = like.device
    dp = None if delta is None else _arg(delta, "delta", _BF16, dev, (T, D))
    rp = None if residual is None else _arg(residual, "residual", _BF16, dev, (T, D))
    gp = None if gamma is None else _arg(gamma, "gamma", _BF16, dev, (D,))
    op = None if post_gamma is None else _arg(post_gamma, "post_gamma", _BF16, dev, (D,))
    yp = pp = wp = up = None
    k = R = gate_dtype = 0
    if routed:
        R, k = y.shape[0], pos.shape[1]
        if R > _I32_MAX:
            raise ValueError(f"y has {R} rows, at most 2^31 - 1 are supported")
        yp = _arg(y, "y", _BF16, dev, (R, D))
        pp = _arg(pos, "pos", _I32, dev, (T, k), 4)
        wp = _arg(weights, "weights", _F32, dev, (T, k), 4)
        if k == 0 or (R == 0 and T > 0):
            raise ValueError("routed rows must not be empty")
    kind = GATE_NONE
    if gate is not None:
        shape = tuple(gate.shape) if isinstance(gate, torch.Tensor) else None
        if shape == (T, D):
            kind = GATE_FULL
        elif shape in ((D,), (1, D)):
            kind = GATE_COLUMN
        elif shape in ((T,), (T, 1)):
            kind = GATE_ROW
        else:
            raise ValueError(f"gate must be a tensor [T], [T, 1], [D], [1, D] or [T, D] with T={T}, D={D}, got {shape}")
        if shape == (T,) and T == D:
            raise ValueError("a gate of T = D values is given as [T, 1] or [1, D]")
        bf16 = gate.dtype == torch.bfloat16
        up = _arg(gate, "gate", _FLOATS if kind == GATE_ROW else _BF16, dev, shape, 16 if kind != GATE_ROW else 2 if bf16 else 4)
        gate_dtype = _DTYPES[gate.dtype]
    unit = 8 if quant is None else 32 if quant == "mxfp8" else 128
    if D % unit or not 0 < D <= ROWS_MAX_D or k > 32:
        raise ValueError(f"D must be a multiple of {unit} up to {ROWS_MAX_D} and top_k at most 32, got D={D}, k={k}")
    if not (want_residual or want_out or quant is not None):
        raise ValueError("no output is wanted")
    if not (math.isfinite(residual_scale) and math.isfinite(gamma_offset)):
        raise ValueError("residual_scale and gamma_offset must be finite")
    with _where(dev, stream, residual, gamma, delta, y, pos, weights, post_gamma, gate):
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
            _call("moe_join_rmsnorm_quant",
                  JoinArgs(NormArgs(T, D, k, R, eps, QUANT[quant], rp, dp, yp, pp, wp, gp, None if res is None else res.data_ptr(),
                                    None if out is None else out.data_ptr(), None if q is None else q.data_ptr(),
                                    None if scale is None else scale.data_ptr()),
                           eps if post_eps is None else post_eps, residual_scale, gamma_offset, kind, gate_dtype, op, up), dev)
    return res, out, q, scale
