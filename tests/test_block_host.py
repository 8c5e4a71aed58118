"""Host checks of the calls around the experts (include/moe_block.h): the
header as C, the ctypes mirrors of its structs, argument errors of the C ABI
(returned before any device work) and of the Python binding; the oracle's
pieces against brute force and closed forms."""

import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import fp8_block_scaled_moe_amd as pkg
from fp8_block_scaled_moe_amd import _block, _capi, _rows
from oracle import block as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, SMALL = _capi.ERR_INVALID_ARG, _capi.ERR_UNSUPPORTED, _capi.ERR_SCRATCH_TOO_SMALL
P = 0x10000  # never dereferenced: every case fails validation or is empty
BF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_capi.LIB_PATH):
        from fp8_block_scaled_moe_amd import build
        build.build()
    return pkg.lib()


@pytest.mark.parametrize("c,mirror", [("moe_dense_args", _block.DenseArgs), ("moe_route_scored_args", _block.RouteScoredArgs),
                                      ("moe_join_args", _block.JoinArgs)])
def test_struct_layout_matches_c(tmp_path, c, mirror):
    fields = [f for f, _ in mirror._fields_]
    body = "\n".join(f'  printf("%zu\\n", offsetof({c}, {f}));' for f in fields)
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"moe_block.h\"\n"
                   f"int main(void) {{\n  printf(\"%zu\\n\", sizeof({c}));\n{body}\n  return 0;\n}}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    out = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert out[0] == ctypes.sizeof(mirror)
    assert out[1:] == [getattr(mirror, f).offset for f in fields]


def fill(cls, base, over):
    a = cls()
    for f, v in {**base, **over}.items():
        setattr(a, f, v)
    return ctypes.byref(a)


DENSE = dict(T=3, N=40, K=64, act=0, out_dtype=1, bias_dtype=0, residual_dtype=1, ldx=64, ldw=64, ldr=40, x=P, w=P, out=P)


@pytest.mark.parametrize("over,code", [
    (dict(T=0, x=None, w=None, out=None), 0),               # an empty call
    (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(N=-8), INVALID),
    (dict(T=1048577), UNSUPPORTED), (dict(N=1048577), UNSUPPORTED), (dict(K=1048584, ldx=1048584, ldw=1048584), UNSUPPORTED),
    (dict(K=60), UNSUPPORTED), (dict(act=-1), UNSUPPORTED), (dict(act=6), UNSUPPORTED), (dict(out_dtype=2), UNSUPPORTED),
    (dict(bias=P, bias_dtype=2), UNSUPPORTED), (dict(residual=P, residual_dtype=-1), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(out=None), INVALID),
    (dict(x=P + 8), INVALID), (dict(w=P + 8), INVALID), (dict(out=P + 8), INVALID), (dict(bias=P + 2), INVALID),
    (dict(bias=P + 1, bias_dtype=1), INVALID), (dict(residual=P + 1), INVALID), (dict(residual=P + 2, residual_dtype=0), INVALID),
    (dict(ldx=56), INVALID), (dict(ldx=68), INVALID), (dict(ldw=56), INVALID), (dict(ldw=65), INVALID), (dict(residual=P, ldr=39), INVALID),
    (dict(ldx=-64), INVALID), (dict(ldx=2**23), UNSUPPORTED), (dict(ldw=2**23), UNSUPPORTED), (dict(residual=P, ldr=2**23), UNSUPPORTED), (dict(workspace=P + 8), INVALID),
])
def test_dense_argument_errors(L, over, code):
    assert L.moe_dense_gemm(fill(_block.DenseArgs, DENSE, over), None) == code


ROUTE = dict(T=100, E=64, k=4, logits_dtype=0, local_begin=0, local_experts=64, routed_scale=1.0, logits=P, bias=P, ids=P,
             weights=P, offsets=P, rows=P, pos=P, workspace=P, workspace_bytes=1 << 20)
SCORED = dict(scores=0, groups=8, top_groups=4, group_best=2, renormalise=1)


def scored(route=(), **over):
    r = _rows.RouteArgs()
    for f, v in {**ROUTE, **dict(route)}.items():
        setattr(r, f, v)
    return fill(_block.RouteScoredArgs, dict(SCORED, route=r), over)


@pytest.mark.parametrize("route,over,code", [
    (dict(T=-1), {}, INVALID), (dict(E=1025), {}, UNSUPPORTED), (dict(k=33), {}, UNSUPPORTED), (dict(logits=None), {}, INVALID),
    (dict(bias=P + 2), {}, INVALID), (dict(workspace=None), {}, INVALID), (dict(workspace_bytes=255), {}, SMALL),
    (dict(offsets=None), {}, INVALID), (dict(local_begin=1), {}, INVALID), (dict(routed_scale=float("inf")), {}, INVALID),
    ({}, dict(scores=2), UNSUPPORTED), ({}, dict(scores=-1), UNSUPPORTED),
    ({}, dict(groups=0), INVALID), ({}, dict(groups=7), UNSUPPORTED), (dict(E=260, local_experts=260), dict(groups=65), UNSUPPORTED),
    ({}, dict(top_groups=0), INVALID), ({}, dict(top_groups=9), INVALID), ({}, dict(group_best=0), INVALID),
    ({}, dict(group_best=3), INVALID), (dict(k=1), dict(groups=64, group_best=2), INVALID),
    (dict(k=9), dict(top_groups=1), INVALID), ({}, dict(renormalise=2), INVALID), ({}, dict(renormalise=-1), INVALID),
])
def test_scored_argument_errors(L, route, over, code):
    assert L.moe_route_rows_scored(scored(route, **over), None) == code


NORM = dict(T=2, D=256, k=0, R=0, eps=1e-5, quant=1, residual=P, delta=P, gamma=P, residual_out=P, out=P, q=P, scale=P)
JOIN = dict(post_eps=1e-5, residual_scale=1.0, gamma_offset=0.0, gate_kind=0, gate_dtype=1, post_gamma=P)


def join(norm=(), **over):
    n = _rows.NormArgs()
    for f, v in {**NORM, **dict(norm)}.items():
        setattr(n, f, v)
    return fill(_block.JoinArgs, dict(JOIN, norm=n), over)


@pytest.mark.parametrize("norm,over,code", [
    (dict(T=0, D=-1), {}, 0),                               # an empty call, whatever the rest
    (dict(T=-1), {}, INVALID), (dict(D=192), {}, UNSUPPORTED), (dict(quant=4), {}, UNSUPPORTED), (dict(q=None), {}, INVALID),
    (dict(eps=float("nan")), {}, INVALID), (dict(delta=None), {}, INVALID), (dict(delta=P + 8), {}, INVALID),
    (dict(k=33, y=P, pos=P, weights=P, R=4), {}, UNSUPPORTED), (dict(k=1), {}, INVALID),
    ({}, dict(post_eps=-1.0), INVALID), ({}, dict(post_eps=float("nan")), INVALID), ({}, dict(post_eps=float("inf")), INVALID),
    ({}, dict(residual_scale=float("inf")), INVALID), ({}, dict(residual_scale=float("nan")), INVALID),
    ({}, dict(gamma_offset=float("nan")), INVALID), ({}, dict(post_gamma=P + 8), INVALID),
    ({}, dict(gate_kind=4, gate=P), UNSUPPORTED), ({}, dict(gate_kind=-1, gate=P), UNSUPPORTED),
    ({}, dict(gate_kind=2, gate=P, gate_dtype=0), UNSUPPORTED), ({}, dict(gate_kind=3, gate=P, gate_dtype=0), UNSUPPORTED),
    ({}, dict(gate_kind=1, gate=P, gate_dtype=2), UNSUPPORTED), ({}, dict(gate=P), INVALID), ({}, dict(gate_kind=1), INVALID),
    ({}, dict(gate_kind=3, gate=P + 8), INVALID), ({}, dict(gate_kind=1, gate=P + 2, gate_dtype=0), INVALID),
    ({}, dict(gate_kind=1, gate=P + 1, gate_dtype=1), INVALID),
])
def test_join_argument_errors(L, norm, over, code):
    assert L.moe_join_rmsnorm_quant(join(norm, **over), None) == code


def test_null_argument_blocks(L):
    for f in (L.moe_dense_gemm, L.moe_route_rows_scored, L.moe_join_rmsnorm_quant):
        assert f(None, None) == INVALID


def test_dense_workspace(L):
    """Nothing for empty and for impossible sizes, whole FP32 outputs otherwise."""
    f = L.moe_dense_gemm_workspace
    assert f(0, 256, 4096) == f(-1, 256, 4096) == f(4, 0, 4096) == f(4, 256, 0) == f(4, -1, 64) == 0
    for T in (1, 3, 17, 64, 100, 509, 5000, 1048576):
        for N, K in ((1, 8), (256, 7168), (896, 3584), (4096, 7168), (1048576, 64), (8, 1048576)):
            need = f(T, N, K)
            assert need % (T * ((N + 7) // 8 * 8) * 4) == 0 and need <= 8 * T * ((N + 7) // 8 * 8) * 4
    assert f(8192, 7168, 7168) == 0
    need = f(256, 4096, 7168)  # K split over workgroups
    assert need
    over = dict(T=256, N=4096, K=7168, ldx=7168, ldw=7168, workspace=P)
    assert L.moe_dense_gemm(fill(_block.DenseArgs, DENSE, dict(over, workspace_bytes=need - 1)), None) == SMALL


# ---- the binding: shapes, types and layouts are checked before the device -----------------------


def dense_args(T=3, N=24, K=64):
    return dict(x=torch.zeros(T, K, dtype=BF), w=torch.zeros(N, K, dtype=BF), bias=torch.zeros(N), residual=torch.zeros(T, N, dtype=BF))


BAD_DENSE = {
    "x 1-D": dict(x=torch.zeros(64, dtype=BF)),
    "x dtype": dict(x=torch.zeros(3, 64)),
    "x fp16": dict(x=torch.zeros(3, 64, dtype=torch.float16)),
    "x columns apart": dict(x=torch.zeros(3, 128, dtype=BF)[:, ::2]),
    "x transposed": dict(x=torch.zeros(64, 3, dtype=BF).t()),
    "x odd stride": dict(x=torch.zeros(3, 68, dtype=BF)[:, :64]),
    "x overlapping rows": dict(x=torch.zeros(1, 64, dtype=BF).expand(3, 64)),
    "x misaligned": dict(x=torch.zeros(3, 72, dtype=BF)[:, 4:68]),
    "w width": dict(w=torch.zeros(24, 56, dtype=BF)),
    "w 3-D": dict(w=torch.zeros(1, 24, 64, dtype=BF)),
    "w transposed": dict(w=torch.zeros(64, 24, dtype=BF).t()),
    "no columns": dict(w=torch.zeros(0, 64, dtype=BF), bias=None, residual=None),
    "K odd": dict(x=torch.zeros(3, 60, dtype=BF), w=torch.zeros(24, 60, dtype=BF)),
    "K zero": dict(x=torch.zeros(3, 0, dtype=BF), w=torch.zeros(24, 0, dtype=BF)),
    "bias shape": dict(bias=torch.zeros(23)),
    "bias dtype": dict(bias=torch.zeros(24).double()),
    "bias strided": dict(bias=torch.zeros(48)[::2]),
    "bias a number": dict(bias=1.0),
    "residual shape": dict(residual=torch.zeros(3, 25, dtype=BF)),
    "residual dtype": dict(residual=torch.zeros(3, 24, dtype=torch.float16)),
    "residual transposed": dict(residual=torch.zeros(24, 3, dtype=BF).t()),
    "residual broadcast": dict(residual=torch.zeros(1, 24, dtype=BF).expand(3, 24)),
    "act": dict(act="tanh"),
    "out_dtype": dict(out_dtype=torch.float16),
}


@pytest.mark.parametrize("what", sorted(BAD_DENSE))
def test_dense_binding_refuses(what):
    with pytest.raises(ValueError) as e:
        pkg.dense_gemm(**{**dense_args(), **BAD_DENSE[what]})
    assert "on a GPU" not in str(e.value)


@pytest.mark.parametrize("args,kw", [
    ((torch.zeros(8),), dict(top_k=2)),
    ((torch.zeros(2, 8).double(),), dict(top_k=2)),
    ((torch.zeros(2, 8), torch.zeros(7)), dict(top_k=2)),
    ((torch.zeros(2, 8), torch.zeros(8, dtype=BF)), dict(top_k=2)),
    ((torch.zeros(2, 8),), dict(top_k=0)),
    ((torch.zeros(2, 8),), dict(top_k=9)),
    ((torch.zeros(2, 1025),), dict(top_k=2)),
    ((torch.zeros(2, 16)[:, ::2],), dict(top_k=2)),
    ((torch.zeros(2, 8),), dict(top_k=2, scores="relu")),
    ((torch.zeros(2, 8),), dict(top_k=2, groups=0)),
    ((torch.zeros(2, 8),), dict(top_k=2, groups=3)),
    ((torch.zeros(2, 260),), dict(top_k=2, groups=130)),
    ((torch.zeros(2, 8),), dict(top_k=2, groups=4, top_groups=0)),
    ((torch.zeros(2, 8),), dict(top_k=2, groups=4, top_groups=5)),
    ((torch.zeros(2, 8),), dict(top_k=2, groups=4, group_best=3)),
    ((torch.zeros(2, 8),), dict(top_k=2, groups=8, group_best=2)),
    ((torch.zeros(2, 8),), dict(top_k=3, groups=4, top_groups=1)),
    ((torch.zeros(2, 8),), dict(top_k=2, local_begin=4, local_experts=5)),
    ((torch.zeros(2, 8),), dict(top_k=2, routed_scale=float("nan"))),
])
def test_scored_binding_refuses(args, kw):
    with pytest.raises(ValueError) as e:
        pkg.route_rows_scored(*args, **kw)
    assert "on a GPU" not in str(e.value)


def join_args(T=3, D=256, k=2, R=6):
    return dict(residual=torch.zeros(T, D, dtype=BF), gamma=torch.zeros(D, dtype=BF), delta=torch.zeros(T, D, dtype=BF),
                y=torch.zeros(R, D, dtype=BF), pos=torch.zeros(T, k, dtype=torch.int32), weights=torch.zeros(T, k),
                post_gamma=torch.zeros(D, dtype=BF), gate=torch.zeros(T, 1))


BAD_JOIN = {
    "residual shape": dict(residual=torch.zeros(2, 256, dtype=BF)),
    "residual dtype": dict(residual=torch.zeros(3, 256)),
    "delta 1-D": dict(delta=torch.zeros(256, dtype=BF)),
    "delta strided": dict(delta=torch.zeros(3, 512, dtype=BF)[:, ::2]),
    "no block output": dict(delta=None, y=None, pos=None, weights=None),
    "y missing": dict(y=None),
    "weights missing": dict(weights=None),
    "pos tokens": dict(pos=torch.zeros(2, 2, dtype=torch.int32)),
    "post_gamma length": dict(post_gamma=torch.zeros(128, dtype=BF)),
    "post_gamma dtype": dict(post_gamma=torch.zeros(256)),
    "gate shape": dict(gate=torch.zeros(3, 2)),
    "gate a number": dict(gate=0.5),
    "gate dtype": dict(gate=torch.zeros(3, 1).double()),
    "gate full in FP32": dict(gate=torch.zeros(3, 256)),
    "gate column in FP32": dict(gate=torch.zeros(256)),
    "gate strided": dict(gate=torch.zeros(3, 2)[:, :1]),
    "residual_scale": dict(residual_scale=float("inf")),
    "gamma_offset": dict(gamma_offset=float("nan")),
    "quant name": dict(quant="fp4"),
    "nothing wanted": dict(quant=None, want_out=False, want_residual=False),
    "in place without residual": dict(residual=None, inplace=True),
}


@pytest.mark.parametrize("what", sorted(BAD_JOIN))
def test_join_binding_refuses(what):
    with pytest.raises(ValueError) as e:
        pkg.join_rmsnorm_quant(**{**join_args(), **BAD_JOIN[what]})
    assert "on a GPU" not in str(e.value)


def test_join_binding_refuses_an_ambiguous_gate():
    with pytest.raises(ValueError, match=r"\[T, 1\] or \[1, D\]"):
        pkg.join_rmsnorm_quant(None, None, delta=torch.zeros(8, 8, dtype=BF), gate=torch.zeros(8, dtype=BF), quant=None)


def test_binding_needs_a_gpu():
    with pytest.raises(ValueError, match="on a GPU"):
        pkg.dense_gemm(**dense_args())
    with pytest.raises(ValueError, match="on a GPU"):
        pkg.route_rows_scored(torch.zeros(2, 8), top_k=2)
    with pytest.raises(ValueError, match="on a GPU"):
        pkg.join_rmsnorm_quant(**join_args())


def test_sizes_past_the_limits_are_refused():
    """Views of one row: nothing is allocated."""
    far = torch.zeros(2**23 + 8, dtype=BF).as_strided((2, 8), (2**23, 1))
    with pytest.raises(ValueError, match="2\\^23"):
        pkg.dense_gemm(torch.zeros(1, 8, dtype=BF), far)
    many = 2**32 + 1
    with pytest.raises(ValueError, match="rows"):
        pkg.dense_gemm(torch.zeros(1, 8, dtype=BF).expand(many, 8), torch.zeros(1, 8, dtype=BF))
    with pytest.raises(ValueError, match="tokens"):
        pkg.route_rows_scored(torch.zeros(1, 8).expand(many, 8), top_k=2)
    with pytest.raises(ValueError, match="tokens"):
        pkg.join_rmsnorm_quant(None, None, delta=torch.zeros(1, 8, dtype=BF).expand(many, 8), quant=None)


# ---- the oracle's pieces ------------------------------------------------------------------------


def test_activations_closed_forms():
    v = np.array([-1e30, -30.0, -1.0, 0.0, 1.0, 30.0])
    assert np.array_equal(ref.activation(v, "relu"), np.maximum(v, 0))
    for act in ("silu", "gelu", "gelu_tanh"):
        got = ref.activation(v, act)
        assert got[3] == 0.0 and got[0] == 0.0 and abs(got[5] - 30.0) < 1e-9 and got[1] <= 0.0
    assert abs(ref.activation(1.0, "silu") - 1.0 / (1.0 + math.exp(-1.0))) < 1e-15
    assert abs(ref.activation(1.0, "gelu") - 0.8413447460685429) < 1e-12
    assert abs(ref.activation(1.0, "gelu_tanh") - 0.8411919906082768) < 1e-12
    assert ref.activation(0.0, "sigmoid") == 0.5


def test_route_scored_brute_force():
    """An expert is picked exactly if its group is among the best and fewer
    than k others of such groups beat it."""
    rng = np.random.default_rng(0)
    for _ in range(60):
        groups, size = int(rng.integers(1, 5)), int(rng.integers(1, 5))
        top, E = int(rng.integers(1, groups + 1)), groups * size
        k, best = int(rng.integers(1, top * size + 1)), int(rng.integers(1, min(size, 2) + 1))
        z, bias = np.round(rng.standard_normal((3, E)) * 2), np.round(rng.standard_normal(E)) * 0.25
        kind = ("sigmoid", "softmax")[int(rng.integers(2))]
        ids, w, key = ref.route_scored(z, bias, k, 1.5, kind=kind, groups=groups, top_groups=top, group_best=best)
        for t in range(3):
            value = [np.float32(np.sort(key[t, g * size:(g + 1) * size])[::-1][:best].sum()) for g in range(groups)]
            inside = [sum(value[h] > value[g] or (value[h] == value[g] and h < g) for h in range(groups)) < top for g in range(groups)]
            beaten = [sum(inside[f // size] and (key[t, f] > key[t, e] or (key[t, f] == key[t, e] and f < e)) for f in range(E))
                      for e in range(E)]
            want = {e for e in range(E) if inside[e // size] and beaten[e] < k}
            assert set(ids[t]) == want and [beaten[e] for e in ids[t]] == list(range(k))
        np.testing.assert_allclose(w.sum(axis=1), 1.5, rtol=1e-6)


def test_join_reduces_to_the_norm():
    """Without a second norm, gate and scale it is rows.py's sum and norm."""
    from oracle import rows

    rng = np.random.default_rng(1)
    r, d, g = (rng.standard_normal(s) for s in ((4, 64), (4, 64), (64,)))
    r, d, g = (np.asarray(torch.from_numpy(v).to(BF).double()) for v in (r, d, g))
    h, v = ref.join_rows(r, d, None, None, None, gamma=g, eps=1e-5)
    assert np.array_equal(h, rows.sum_rows(r, d, None, None, None)) and np.array_equal(v, rows.norm_rows(h, g, 1e-5))
    h, v = ref.join_rows(None, d, None, None, None, gamma=None, eps=1e-5, post_gamma=g, gate=0.5)
    np.testing.assert_allclose(h, 0.5 * rows.norm_rows(d, g, 1e-5), rtol=2.0**-22)
    assert np.array_equal(v, h)
