"""The operators around the routed experts (include/moe_block.h) in float64
NumPy.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The grouping of the routes, the row sum and the quantisation are rows.py's;
this file has the dense product, the scored routing and the join of a block's
output with the residual.
"""

from __future__ import annotations

import math

import numpy as np

from .codecs import f32
from .rows import sum_rows

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(v, act):
    v = np.asarray(v, np.float64)
    with np.errstate(over="ignore"):
        if act == "relu":
            return np.maximum(v, 0.0)
        if act == "silu":
            return v / (1.0 + np.exp(-v))
        if act == "sigmoid":
            return 1.0 / (1.0 + np.exp(-v))
        if act == "gelu":
            return 0.5 * v * (1.0 + _erf(v / math.sqrt(2.0)))
        if act == "gelu_tanh":
            return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v**3)))
    return v


def dense(x, w, bias=None, act=None, residual=None):
    """(out, before): act(x w^T + bias) + residual in float64, and x w^T + bias."""
    v = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        v = v + np.asarray(bias, np.float64)
    out = activation(v, act)
    return out if residual is None else out + np.asarray(residual, np.float64), v


def scores(logits, kind: str) -> np.ndarray:
    """Scores rounded to binary32 from float64; a softmax row of minus infinities has scores of 0."""
    z = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return f32(1.0 / (1.0 + np.exp(-z)))
        top = z.max(axis=1, keepdims=True)
        e = np.exp(z - np.where(np.isneginf(top), 0.0, top))
        total = e.sum(axis=1, keepdims=True)
        return f32(e / np.where(total == 0.0, 1.0, total))


def route_scored(logits, bias, top_k: int, routed_scale: float, *, kind: str = "sigmoid", groups: int = 1, top_groups: int = 1,
                 group_best: int = 1, renormalise: bool = True):
    """(ids, weights, keys) of every token, one expert at a time."""
    s = scores(logits, kind)
    key = s if bias is None else f32(s + f32(bias)[None, :])
    T, E = s.shape
    size = E // groups
    ids, weights = np.empty((T, top_k), np.int32), np.empty((T, top_k))
    scale = float(f32(routed_scale))
    for t in range(T):
        value = []
        for g in range(groups):
            best = sorted(key[t, g * size:(g + 1) * size], reverse=True)[:group_best]
            value.append(float(f32(sum(best))))
        inside = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
        may = [e for e in range(E) if e // size in inside]
        picked = sorted(may, key=lambda e: (-key[t, e], e))[:top_k]
        total = 0.0
        for e in picked:
            total = float(f32(total + s[t, e]))
        ids[t] = picked
        if not renormalise:
            weights[t] = f32(s[t, picked] * scale)
        elif total == 0.0:
            weights[t] = 0.0
        else:
            weights[t] = f32(f32(s[t, picked] / total) * scale)
    return ids, weights, key


def _rstd(h, eps):
    return f32(1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + float(f32(eps))))


def join_rows(residual, delta, y, pos, weights, *, gamma, eps, post_gamma=None, post_eps=None, gate=None, residual_scale=1.0,
              gamma_offset=0.0):
    """(h, v): the residual row and its normalised form, binary32 values; gate
    broadcasts against [T, D]. Both norms are binary32 steps; the residual row is
    rounded once, from products that float64 holds exactly."""
    n = b = np.asarray(sum_rows(None, delta, y, pos, weights), np.float64)
    plus = lambda g: f32(np.asarray(g, np.float64) + float(f32(gamma_offset)))  # noqa: E731
    if post_gamma is not None:
        n = f32(f32(b * _rstd(b, eps if post_eps is None else post_eps)) * plus(post_gamma))
    h = n * (1.0 if gate is None else np.asarray(gate, np.float64))
    if residual is not None:
        h = h + np.asarray(residual, np.float64) * float(f32(residual_scale))
    h = np.asarray(f32(h), np.float64)
    return h, h if gamma is None else f32(f32(h * _rstd(h, eps)) * plus(gamma))
