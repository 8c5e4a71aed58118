"""moe_dense_gemm in every form that it has: sizes that take it (test_dense_plan_host.py
holds them to that), N a multiple of 8 and odd, a K that ends inside a block. The bound
of an element is test_gpu_dense.py's."""

from __future__ import annotations

import ctypes

import pytest
import torch

from fp8_block_scaled_moe_amd import _block, _capi, dense_gemm, lib

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16

# (form, parts of K): sizes
FORMS = {
    ("strip 4x4", 1): [(1, 256, 7168), (2, 40, 4104), (8, 991, 39832), (23, 280, 32296)],
    ("strip 16x16", 1): [(5, 40, 136), (109, 576, 31824), (1316, 45, 33736)],
    ("strip 16x32", 1): [(7, 7160, 39904), (2676, 19, 39336)],
    ("strip 32x32", 1): [(142, 1592, 8848), (94, 2327, 9144)],
    ("strip 32x64", 1): [(9427, 40, 5304), (21, 18571, 5128)],
    ("64x128", 1): [(420, 4544, 1048), (1426, 1359, 1032)],
    ("64x128", 2): [(168, 3256, 3656), (4306, 105, 4424)],
    ("64x128", 4): [(36, 4328, 12856), (36, 4691, 11800)],
    ("64x128", 8): [(35, 2856, 20000), (338, 325, 18200), (59, 1856, 26600)],
    ("128x128", 1): [(1790, 2216, 504), (353, 6557, 864)],
    ("128x128", 2): [(9014, 40, 6576), (8965, 37, 6120), (774, 1280, 7816), (317, 3711, 7728)],
    ("128x128", 4): [(70, 5528, 5160), (72, 5457, 5080)],
    ("128x128, two a CU", 1): [(1341, 5488, 272), (10845, 699, 264)],
    ("256x256", 1): [(3861, 2488, 208), (13875, 693, 208)],
    ("256x256 and halves", 1): [(929, 19224, 112), (369, 11681, 464)],
}
SIZES = [(*form, *size) for form, sizes in FORMS.items() for size in sizes]


def make(T, N, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return dict(x=normal(T, K).to(BF), w=(normal(N, K) * K**-0.5).to(BF), bias=normal(N), residual=normal(T, N).to(BF))


def exact(d, relu):
    """The values in float64, and the bound of their sums: K / 16 additions in a row and 64 more, 2^-23 of the
    magnitudes each, and 8 of what is added."""
    x, w = d["x"].double(), d["w"].double()
    before = x @ w.t() + d["bias"].double()
    out = (before.clamp_min(0) if relu else before) + d["residual"].double()
    most = (x.shape[1] / 16 + 64) * 2.0**-23 * (x.abs() @ w.abs().t())
    return out, most + 8 * 2.0**-23 * (before.abs() + out.abs() + d["bias"].double().abs() + d["residual"].double().abs())


@pytest.mark.parametrize("form,splits,T,N,K", SIZES)
def test_every_form(form, splits, T, N, K):
    d = make(T, N, K, T + N)
    for act, dtype in ((None, torch.float32), ("relu", BF)):
        out, most = exact(d, act == "relu")
        most = most + (out.abs() + most) * torch.finfo(dtype).eps / 2
        got = dense_gemm(**d, act=act, out_dtype=dtype)
        off = (got.double() - out).abs()
        assert bool((off <= most).all()), f"{int((off > most).sum())} values outside, the worst {float((off / most).max())} times"
        assert torch.equal(got, dense_gemm(**d, act=act, out_dtype=dtype))


@pytest.mark.parametrize("form,splits,T,N,K", [s for s in SIZES if s[1] > 1])
def test_parts_of_k_stay_in_their_workspace(form, splits, T, N, K):
    d = make(T, N, K, 7)
    need = lib().moe_dense_gemm_workspace(T, N, K)
    assert need == splits * T * ((N + 7) // 8 * 8) * 4
    ws = torch.full((need + 256,), 170, dtype=torch.uint8, device=DEV)
    out = torch.full((T * N + 256,), 77.0, device=DEV)
    a = _block.DenseArgs(T, N, K, 0, 0, 0, 1, K, K, N, d["x"].data_ptr(), d["w"].data_ptr(), d["bias"].data_ptr(), d["residual"].data_ptr(),
                         out.data_ptr(), ws.data_ptr(), need)
    assert lib().moe_dense_gemm(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == _capi.OK
    assert (out[T * N:] == 77.0).all() and (ws[need:] == 170).all()
    assert torch.equal(out[: T * N].view(T, N), dense_gemm(**d, out_dtype=torch.float32))


@pytest.mark.parametrize("T,N,K", [(1, 12288, 5120), (3, 20481, 16392), (40, 16384, 12288), (300, 10240, 20488), (2000, 28672, 8200), (700, 9000, 24576)])
def test_wide_layers(T, N, K):
    """Weights with more than 8,192 rows or columns."""
    test_every_form("", 0, T, N, K)


@pytest.mark.parametrize("T,N,K", [(1, 40, 72), (3, 264, 72), (40, 264, 200), (300, 301, 328), (1300, 264, 136)])
def test_every_other_row(T, N, K):
    """Rows of x, w and the residual twice as far apart; those between are NaN and stay out."""
    d = make(T, N, K, 9)
    apart = {}
    for n in ("x", "w", "residual"):
        both = torch.full((2 * d[n].shape[0], d[n].shape[1]), float("nan"), dtype=BF, device=DEV)
        both[::2] = d[n]
        apart[n] = both[::2]
        assert d[n].shape[0] == 1 or not apart[n].is_contiguous()
    assert torch.equal(dense_gemm(**{**d, **apart}), dense_gemm(**d))
