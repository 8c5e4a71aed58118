"""The operators over any number of tokens (include/moe_rows.h) in float64
NumPy.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Routing and quantisation are the layer's (moe.route, moe.quantize_blocks) and
the boundary's (boundary.mxfp8_quantize); this file has the grouping of the
routes by expert and the sum + RMSNorm row.
"""

from __future__ import annotations

from typing import Tuple

import numpy as np

from .boundary import mxfp8_quantize
from .codecs import f32
from .moe import quantize_blocks


def group_routes(ids, local_begin: int, local_experts: int) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """The routes ids [T, k] grouped by local expert, tokens ascending inside
    an expert: (offsets [local_experts + 1], rows: the token of each grouped
    row, pos [T, k]: the grouped row of each pick, -1 where the expert is not
    local)."""
    ids = np.asarray(ids)
    T, k = ids.shape
    offsets, rows, pos = [0], [], np.full((T, k), -1, np.int64)
    for e in range(local_begin, local_begin + local_experts):
        for t, j in np.argwhere(ids == e):
            pos[t, j] = len(rows)
            rows.append(t)
        offsets.append(len(rows))
    return np.array(offsets), np.array(rows, np.int64), pos


def sum_rows(residual, delta, y, pos, weights) -> np.ndarray:
    """h = residual + delta + sum_j weights[t, j] * y[pos[t, j]] in float64,
    rounded once to binary32. Any of the three parts may be None; a position
    outside y adds nothing."""
    h = 0.0
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    if delta is not None:
        h = h + np.asarray(delta, np.float64)
    if y is not None:
        y, pos = np.asarray(y, np.float64), np.asarray(pos)
        inside = (pos >= 0) & (pos < y.shape[0])
        w = np.where(inside, np.asarray(weights, np.float64), 0.0)
        h = h + (w[..., None] * y[np.where(inside, pos, 0)]).sum(axis=1)
    return f32(h)


def norm_rows(h, gamma, eps: float) -> np.ndarray:
    """v = (h * rstd) * gamma with rstd = binary32(1 / sqrt(mean(h^2) + eps))
    and both products rounded to binary32."""
    h = np.asarray(h, np.float64)
    rstd = f32(1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + float(f32(eps))))
    return f32(f32(h * rstd) * np.asarray(gamma, np.float64))


def quantize_rows(v, quant: str):
    """(codes, scales) of binary32 rows: "fp8", "fp8_p2" or "mxfp8"."""
    if quant == "mxfp8":
        return mxfp8_quantize(v)
    return quantize_blocks(v, ue8m0=quant == "fp8_p2", reciprocal=True)
