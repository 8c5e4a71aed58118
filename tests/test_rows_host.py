"""Host checks of the calls over any number of tokens (include/moe_rows.h):
the header as C, the ctypes mirrors of its structs, argument errors of the C
ABI (returned before any device work) and of the Python binding."""

import ctypes
import os
import subprocess

import pytest
import torch

import fp8_block_scaled_moe_amd as pkg
from fp8_block_scaled_moe_amd import _capi, _rows

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, SMALL = _capi.ERR_INVALID_ARG, _capi.ERR_UNSUPPORTED, _capi.ERR_SCRATCH_TOO_SMALL
P = 0x10000  # never dereferenced: every case fails validation or is empty


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_capi.LIB_PATH):
        from fp8_block_scaled_moe_amd import build
        build.build()
    return pkg.lib()


@pytest.mark.parametrize("c,mirror", [("moe_norm_args", _rows.NormArgs), ("moe_route_args", _rows.RouteArgs),
                                      ("moe_grouped_args", _rows.GroupedArgs)])
def test_struct_layout_matches_c(tmp_path, c, mirror):
    fields = [f for f, _ in mirror._fields_]
    body = "\n".join(f'  printf("%zu\\n", offsetof({c}, {f}));' for f in fields)
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"moe_rows.h\"\n"
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


NORM = dict(T=2, D=256, k=0, R=0, eps=1e-5, quant=1, residual=P, gamma=P, residual_out=P, out=P, q=P, scale=P)


@pytest.mark.parametrize("over,code", [
    (dict(T=0, D=-1), 0),                                   # an empty call, whatever the rest
    (dict(T=-1), INVALID), (dict(k=-1), INVALID), (dict(R=-1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(quant=4), UNSUPPORTED), (dict(quant=-1), UNSUPPORTED), (dict(T=1048577), UNSUPPORTED),
    (dict(D=0), UNSUPPORTED), (dict(D=192), UNSUPPORTED), (dict(D=16384 + 128), UNSUPPORTED),
    (dict(D=48, quant=3), UNSUPPORTED), (dict(D=12, quant=0, q=None, scale=None), UNSUPPORTED),
    (dict(residual=None), INVALID),                         # nothing to add
    (dict(residual_out=None, out=None, q=None, scale=None, quant=0), INVALID),
    (dict(q=None), INVALID), (dict(scale=None), INVALID), (dict(quant=0), INVALID),
    (dict(k=2), INVALID), (dict(k=2, y=P, pos=P), INVALID), (dict(y=P), INVALID), (dict(weights=P), INVALID),
    (dict(k=33, y=P, pos=P, weights=P, R=4), UNSUPPORTED),
    (dict(residual=P + 8), INVALID), (dict(delta=P + 2), INVALID), (dict(gamma=P + 8), INVALID),
    (dict(out=P + 8), INVALID), (dict(q=P + 8), INVALID), (dict(scale=P + 2), INVALID),
    (dict(k=1, R=1, y=P, pos=P + 2, weights=P), INVALID),
])
def test_norm_argument_errors(L, over, code):
    assert L.moe_add_rmsnorm_quant(fill(_rows.NormArgs, NORM, over), None) == code


ROUTE = dict(T=100, E=64, k=4, logits_dtype=0, local_begin=0, local_experts=64, routed_scale=1.0, logits=P, bias=P, ids=P,
             weights=P, offsets=P, rows=P, pos=P, workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(E=0), INVALID),
    (dict(routed_scale=float("inf")), INVALID), (dict(routed_scale=float("nan")), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(k=33), UNSUPPORTED), (dict(E=3), UNSUPPORTED), (dict(T=1048577), UNSUPPORTED),
    (dict(logits_dtype=2), UNSUPPORTED),
    (dict(local_begin=-1), INVALID), (dict(local_experts=0), INVALID), (dict(local_experts=65), INVALID),
    (dict(local_begin=1), INVALID), (dict(local_begin=2**31 - 1, local_experts=2), INVALID),
    (dict(logits=None), INVALID), (dict(bias=None), INVALID), (dict(ids=None), INVALID), (dict(weights=None), INVALID),
    (dict(offsets=None), INVALID), (dict(rows=None), INVALID), (dict(pos=None), INVALID),
    (dict(logits=P + 2), INVALID), (dict(logits=P + 1, logits_dtype=1), INVALID), (dict(pos=P + 2), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace=P + 2), INVALID),
    (dict(workspace_bytes=255), SMALL),
])
def test_route_argument_errors(L, over, code):
    assert L.moe_route_rows(fill(_rows.RouteArgs, ROUTE, over), None) == code


def test_route_workspace(L):
    """Nothing for a few tokens; it grows with tokens and experts."""
    assert L.moe_route_rows_workspace(0, 8) == 0 and L.moe_route_rows_workspace(32, 1024) == 0
    sizes = [L.moe_route_rows_workspace(T, 64) for T in (33, 65, 100, 1000, 8192, 8193, 65536, 65537, 1048576)]
    assert all(s >= 256 and s % 4 == 0 for s in sizes)
    assert L.moe_route_rows_workspace(1000, 128) == 2 * L.moe_route_rows_workspace(1000, 64)
    assert L.moe_route_rows_workspace(1048576, 1024) < 1 << 28


GROUPED = dict(R=4, X=4, E=2, N=256, K=256, quant=1, limit=7.0, x=P, x_scale=P, offsets=P, w=P, w_scale=P, out=P,
               out_scale=P)


@pytest.mark.parametrize("over,code", [
    (dict(R=0, X=0, x=None), 0),                            # an empty call
    (dict(R=-1), INVALID), (dict(X=-1), INVALID), (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(N=320), UNSUPPORTED), (dict(K=192), UNSUPPORTED),
    (dict(N=131072 + 256), UNSUPPORTED), (dict(K=131072 + 128), UNSUPPORTED),
    (dict(quant=0), UNSUPPORTED), (dict(quant=4), UNSUPPORTED),
    (dict(X=3), INVALID), (dict(X=0, rows=P), INVALID),
    (dict(R=2**31 - 1, X=2**31 - 1), UNSUPPORTED), (dict(R=2**25, X=2**25, N=8192), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(x_scale=None), INVALID), (dict(offsets=None), INVALID), (dict(w=None), INVALID),
    (dict(w_scale=None), INVALID), (dict(out=None), INVALID),
    (dict(x=P + 8), INVALID), (dict(w=P + 8), INVALID), (dict(out=P + 8), INVALID), (dict(rows=P + 2), INVALID),
    (dict(x_scale=P + 2), INVALID), (dict(x_scale=P + 2, quant=3), INVALID), (dict(w_scale=P + 2), INVALID), (dict(offsets=P + 2), INVALID),
])
def test_grouped_argument_errors(L, over, code):
    assert L.moe_grouped_gemm(fill(_rows.GroupedArgs, GROUPED, over), None) == code
    assert L.moe_grouped_swiglu(fill(_rows.GroupedArgs, GROUPED, over), None) == code


def test_grouped_own_errors(L):
    # the SwiGLU takes whole 128-column blocks of up and of gate rows, a positive limit and a scale array
    assert L.moe_grouped_swiglu(fill(_rows.GroupedArgs, GROUPED, dict(N=384)), None) == UNSUPPORTED
    for limit in (0.0, -1.0, float("nan")):
        assert L.moe_grouped_swiglu(fill(_rows.GroupedArgs, GROUPED, dict(limit=limit)), None) == INVALID
    assert L.moe_grouped_swiglu(fill(_rows.GroupedArgs, GROUPED, dict(out_scale=None)), None) == INVALID


def test_grouped_sums(L):
    # the kind of sums is the plain product's own choice
    for sums in (-1, 2):
        assert L.moe_grouped_gemm(fill(_rows.GroupedArgs, GROUPED, dict(sums=sums)), None) == UNSUPPORTED
    for sums in (-1, 1, 2):
        assert L.moe_grouped_swiglu(fill(_rows.GroupedArgs, GROUPED, dict(sums=sums)), None) == UNSUPPORTED
    with pytest.raises(ValueError, match="sums"):
        pkg.grouped_gemm(*grouped_args(), sums="bf16")


def test_grouped_workspace(L):
    """Something where K can be split over workgroups, nothing where the tiles
    fill the GPU or K is short; too little of it and a misaligned one are
    errors, none at all is not."""
    need = L.moe_grouped_gemm_workspace(4, 2, 256, 4096)
    assert need and need % (4 * 256 * 4) == 0
    assert L.moe_grouped_swiglu_workspace(4, 2, 256, 4096)
    for f in (L.moe_grouped_gemm_workspace, L.moe_grouped_swiglu_workspace):
        assert f(4, 2, 256, 1920) == 0 and f(100000, 256, 4096, 4096) == 0
        assert f(0, 2, 256, 4096) == f(4, 0, 256, 4096) == f(4, 2, 0, 4096) == f(4, 2, 256, 0) == f(-1, 2, 256, 4096) == 0
        # never more than one part for each of 256 CUs
        for R in (1, 3, 100, 5000, 32768):
            assert f(R, 8, 512, 8192) <= 256 * 256 * 256 * 4
    for call in (L.moe_grouped_gemm, L.moe_grouped_swiglu):
        for over, code in ((dict(workspace=P, workspace_bytes=need - 1), SMALL), (dict(workspace=P + 8, workspace_bytes=need), INVALID)):
            assert call(fill(_rows.GroupedArgs, GROUPED, dict(K=4096, **over)), None) == code


def test_null_argument_blocks(L):
    for f in (L.moe_add_rmsnorm_quant, L.moe_route_rows, L.moe_grouped_gemm, L.moe_grouped_swiglu):
        assert f(None, None) == INVALID


# ---- the binding: shapes, types and layouts are checked before the device -----------------------

BF = torch.bfloat16


def norm_args(T=3, D=256, k=2, R=6):
    return dict(residual=torch.zeros(T, D, dtype=BF), gamma=torch.zeros(D, dtype=BF), delta=torch.zeros(T, D, dtype=BF),
                y=torch.zeros(R, D, dtype=BF), pos=torch.zeros(T, k, dtype=torch.int32), weights=torch.zeros(T, k))


BAD_NORM = {
    "residual 1-D": dict(residual=torch.zeros(256, dtype=BF)),
    "residual dtype": dict(residual=torch.zeros(3, 256)),
    "delta shape": dict(delta=torch.zeros(2, 256, dtype=BF)),
    "delta strided": dict(delta=torch.zeros(3, 512, dtype=BF)[:, ::2]),
    "delta misaligned": dict(delta=torch.zeros(3 * 256 + 4, dtype=BF)[4:].view(3, 256)),
    "gamma length": dict(gamma=torch.zeros(128, dtype=BF)),
    "y width": dict(y=torch.zeros(6, 128, dtype=BF)),
    "y missing": dict(y=None),
    "pos dtype": dict(pos=torch.zeros(3, 2, dtype=torch.int64)),
    "pos tokens": dict(pos=torch.zeros(2, 2, dtype=torch.int32)),
    "weights shape": dict(weights=torch.zeros(3, 3)),
    "weights missing": dict(weights=None),
    "no rows in y": dict(y=torch.zeros(0, 256, dtype=BF)),
    "quant name": dict(quant="fp4"),
    "nothing wanted": dict(quant=None, want_out=False, want_residual=False),
    "in place without residual": dict(residual=None, inplace=True),
}


@pytest.mark.parametrize("what", sorted(BAD_NORM))
def test_norm_binding_refuses(what):
    with pytest.raises(ValueError) as e:
        pkg.add_rmsnorm_quant(**{**norm_args(), **BAD_NORM[what]})
    assert "on a GPU" not in str(e.value)


@pytest.mark.parametrize("D,quant", [(192, "fp8"), (48, "mxfp8"), (12, None), (16384 + 128, "fp8")])
def test_norm_binding_refuses_widths(D, quant):
    with pytest.raises(ValueError, match="multiple of"):
        pkg.add_rmsnorm_quant(torch.zeros(1, D, dtype=BF), None, quant=quant)


def test_binding_needs_a_gpu():
    with pytest.raises(ValueError, match="on a GPU"):
        pkg.add_rmsnorm_quant(**norm_args())
    with pytest.raises(ValueError, match="at least one"):
        pkg.add_rmsnorm_quant(None, None)
    with pytest.raises(ValueError, match="on a GPU"):
        pkg.route_rows(torch.zeros(2, 8), torch.zeros(8), top_k=2, routed_scale=1.0)
    with pytest.raises(ValueError, match="on a GPU"):
        pkg.grouped_gemm(*grouped_args())
    with pytest.raises(ValueError, match="on a GPU"):
        pkg.grouped_swiglu(*grouped_args(), limit=7.0)


def test_sizes_past_32_bits_are_refused():
    """Lengths that the C ABI's 32-bit sizes would cut off (views of one row:
    nothing is allocated)."""
    many = 2**32 + 1
    long = lambda t: t.expand(many, *t.shape[1:])  # noqa: E731
    with pytest.raises(ValueError, match="tokens"):
        pkg.add_rmsnorm_quant(long(torch.zeros(1, 8, dtype=BF)), None, quant=None)
    with pytest.raises(ValueError, match="tokens"):
        pkg.route_rows(long(torch.zeros(1, 8)), torch.zeros(8), top_k=1, routed_scale=1.0)
    with pytest.raises(ValueError, match="rows"):
        pkg.add_rmsnorm_quant(**{**norm_args(), "y": long(torch.zeros(1, 256, dtype=BF))})
    for i in (0, 1):
        args = grouped_args()
        args[0] = long(torch.zeros(1, 256, dtype=torch.uint8)) if i == 0 else args[0]
        rows = long(torch.zeros(1, dtype=torch.int32)) if i else None
        with pytest.raises(ValueError, match="2\\^31"):
            pkg.grouped_gemm(*args, rows=rows)
        with pytest.raises(ValueError, match="2\\^31"):
            pkg.grouped_swiglu(*args, rows=rows, limit=7.0)


@pytest.mark.parametrize("args,kw", [
    ((torch.zeros(8), torch.zeros(8)), dict(top_k=2)),
    ((torch.zeros(2, 8).double(), torch.zeros(8)), dict(top_k=2)),
    ((torch.zeros(2, 8), torch.zeros(7)), dict(top_k=2)),
    ((torch.zeros(2, 8), torch.zeros(8)), dict(top_k=0)),
    ((torch.zeros(2, 8), torch.zeros(8)), dict(top_k=9)),
    ((torch.zeros(2, 1025), torch.zeros(1025)), dict(top_k=2)),
    ((torch.zeros(2, 8), torch.zeros(8)), dict(top_k=2, local_begin=4, local_experts=5)),
    ((torch.zeros(2, 8), torch.zeros(8)), dict(top_k=2, local_begin=8)),
    ((torch.zeros(2, 16)[:, ::2], torch.zeros(8)), dict(top_k=2)),
])
def test_route_binding_refuses(args, kw):
    with pytest.raises(ValueError) as e:
        pkg.route_rows(*args, routed_scale=1.0, **kw)
    assert "on a GPU" not in str(e.value)


def grouped_args(R=5, E=3, N=256, K=256):
    u8 = torch.uint8
    return [torch.zeros(R, K, dtype=u8), torch.ones(R, K // 128), torch.zeros(E, N, K, dtype=u8),
            torch.ones(E, N // 128, K // 128), torch.zeros(E + 1, dtype=torch.int32)]


BAD_GROUPED = {
    "x 1-D": (0, torch.zeros(256, dtype=torch.uint8)),
    "x dtype": (0, torch.zeros(5, 256)),
    "x width": (0, torch.zeros(5, 128, dtype=torch.uint8)),
    "x odd width": (0, torch.zeros(5, 200, dtype=torch.uint8)),
    "x_scale shape": (1, torch.ones(5, 1)),
    "x_scale bytes shape": (1, torch.ones(5, 2, dtype=torch.uint8)),
    "x_scale dtype": (1, torch.ones(5, 2).double()),
    "w 2-D": (2, torch.zeros(256, 256, dtype=torch.uint8)),
    "w rows": (2, torch.zeros(3, 200, 256, dtype=torch.uint8)),
    "w transposed": (2, torch.zeros(3, 256, 256, dtype=torch.uint8).transpose(1, 2)),
    "w_scale shape": (3, torch.ones(3, 256, 2)),
    "offsets short": (4, torch.zeros(3, dtype=torch.int32)),
    "offsets dtype": (4, torch.zeros(4, dtype=torch.int64)),
}


@pytest.mark.parametrize("what", sorted(BAD_GROUPED))
def test_grouped_binding_refuses(what):
    args = grouped_args()
    i, t = BAD_GROUPED[what]
    args[i] = t
    for call in (lambda: pkg.grouped_gemm(*args), lambda: pkg.grouped_swiglu(*args, limit=7.0)):
        with pytest.raises(ValueError) as e:
            call()
        assert "on a GPU" not in str(e.value)


@pytest.mark.parametrize("kw", [dict(rows=torch.zeros(4, dtype=torch.int64)), dict(rows=torch.zeros(2, 2, dtype=torch.int32)),
                                dict(rows=[0, 1])])
def test_grouped_binding_refuses_rows(kw):
    with pytest.raises(ValueError):
        pkg.grouped_gemm(*grouped_args(), **kw)


def test_grouped_binding_refuses_options():
    with pytest.raises(ValueError, match="limit"):
        pkg.grouped_swiglu(*grouped_args(), limit=0.0)
    with pytest.raises(ValueError, match="multiple of 128"):
        pkg.grouped_swiglu(*grouped_args(N=384), limit=7.0)
    args = grouped_args()
    args[0], args[1] = args[0][:0], args[1][:0]
    with pytest.raises(ValueError, match="no rows"):
        pkg.grouped_gemm(*args, rows=torch.zeros(2, dtype=torch.int32))


def test_assembly_names_the_registers_it_writes():
    """Every asm statement that writes M0 says so: the compiler uses it too."""
    import re

    csrc, seen = os.path.join(ROOT, "fp8_block_scaled_moe_amd", "csrc"), 0
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            for stmt in re.findall(r"asm volatile\(.*?\);", f.read(), re.S):
                if "s_mov_b32 m0" in stmt:
                    seen += 1
                    assert re.search(r':\s*"m0"', stmt), f"{name}: {stmt}"
    assert seen
