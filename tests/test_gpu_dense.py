"""moe_dense_gemm on the GPU against float64.

Bound of an element. The products of BF16 values are exact in FP32. K of them
are added in FP32 by K / 16 additions or fewer in a row, and 64 more at most
where waves and parts of K are joined, each off by at most 2^-23 of the sum of
the magnitudes S (2^-24 for a rounding, twice that where an instruction cuts
off): (K / 16 + 64) 2^-23 S. The bias, the activation (slope at most 1.13, its
own error 4 * 2^-23 of max(|v|, |act|, 1)) and the residual add at most 8 *
2^-23 of their values, the output half a step of its type."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from fp8_block_scaled_moe_amd import _block, _capi, dense_gemm, lib
from oracle import block as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh", "sigmoid"]


def host(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def make(T, N, K, seed, bias=None, residual=None, pad=0, scale=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K + pad, generator=g)
    w = torch.randn(N, K, generator=g) * (K**-0.5 if scale is None else scale)
    d = dict(x=x.to(BF).to(DEV)[:, :K], w=w.to(BF).to(DEV))
    if bias:
        d["bias"] = torch.randn(N, generator=g).to(bias).to(DEV)
    if residual:
        d["residual"] = torch.randn(T, N, generator=g).to(residual).to(DEV)
    return d


def bound(d, K, act, out, before, dtype):
    x, w = np.abs(host(d["x"])), np.abs(host(d["w"]))
    mag = np.abs(before)
    err = (K / 16 + 64) * 2.0**-23 * (x @ w.T)
    rest = mag + np.abs(out) + (1.0 if act else 0.0)
    for n in ("bias", "residual"):
        if d.get(n) is not None:
            rest = rest + np.abs(host(d[n]))
    err = 1.13 * err + 8 * 2.0**-23 * rest
    return err + (np.abs(out) + err) * torch.finfo(dtype).eps / 2 + 1e-38


def check(d, act=None, dtype=BF, **kw):
    got = dense_gemm(**d, act=act, out_dtype=dtype, **kw)
    torch.cuda.synchronize()
    assert got.dtype == dtype and got.is_contiguous()
    out, before = ref.dense(host(d["x"]), host(d["w"]), host(d.get("bias")), act, host(d.get("residual")))
    assert got.shape == out.shape
    off = np.abs(host(got) - out)
    most = bound(d, d["x"].shape[1], act, out, before, dtype)
    worst = np.unravel_index(np.argmax(off / most), off.shape) if off.size else None
    assert (off <= most).all(), f"at {worst}: got {host(got)[worst]}, {out[worst]} within {most[worst]}"
    return got


# rows and columns around the tiles' sizes, K around the steps'
SIZES = [(1, 1, 8), (1, 256, 7168), (2, 7, 16), (3, 15, 24), (4, 16, 32), (5, 17, 40), (7, 31, 56), (8, 33, 64), (15, 63, 72), (16, 64, 128),
         (17, 65, 136), (31, 127, 200), (32, 128, 256), (33, 129, 264), (47, 255, 512), (48, 256, 520), (63, 257, 1000), (64, 100, 1024),
         (65, 300, 1032), (100, 8, 2048), (127, 384, 96), (128, 385, 64), (129, 512, 120), (200, 513, 320), (255, 130, 448), (256, 256, 192),
         (257, 511, 104), (300, 1, 1536), (384, 770, 88), (511, 1024, 640), (512, 640, 1088), (513, 264, 3584), (700, 520, 1920),
         (1025, 1, 64), (1030, 1032, 72), (2049, 272, 128), (4097, 24, 48), (9, 2056, 4104), (40, 4104, 264), (1, 5000, 512), (70, 3000, 8)]


@pytest.mark.parametrize("T,N,K", SIZES)
def test_sizes(T, N, K):
    check(make(T, N, K, T + N + K))
    check(make(T, N, K, T + N + K + 1, bias=BF, residual=BF), act="silu")
    check(make(T, N, K, T + N + K + 2, bias=torch.float32, residual=torch.float32), dtype=torch.float32)


# tiles of every size, whole and ragged rounds of them, K split over workgroups, rows that begin anywhere
LARGE = [(138, 3584, 7168), (200, 4096, 7160), (256, 4096, 7168), (256, 4093, 7168), (200, 4001, 6000), (350, 4090, 648), (363, 896, 7168),
         (300, 7168, 2048), (311, 7165, 520), (900, 7100, 328), (1900, 1000, 2056), (2300, 3000, 72), (3000, 7000, 136), (4200, 4600, 136),
         (4352, 4096, 72), (4500, 2600, 520), (4500, 2601, 1032), (5000, 2000, 1032), (6000, 2600, 520), (8192, 2048, 128), (8191, 896, 3584),
         (9078, 256, 1024), (10807, 1, 2472), (16384, 30, 64), (3, 8192, 8192), (64, 8191, 4096)]


def exact_on_gpu(d, act):
    """The same in FP64 on the GPU, and the bound."""
    x, w = d["x"].double(), d["w"].double()
    before = x @ w.t()
    mag = x.abs() @ w.abs().t()
    if d.get("bias") is not None:
        before = before + d["bias"].double()
    out = {None: lambda v: v, "relu": lambda v: v.clamp_min(0), "silu": lambda v: v / (1 + (-v).exp()),
           "gelu": lambda v: 0.5 * v * (1 + torch.erf(v * 0.5**0.5))}[act](before)
    res = d["residual"].double() if d.get("residual") is not None else torch.zeros_like(out)
    err = 1.13 * (x.shape[1] / 16 + 64) * 2.0**-23 * mag + 8 * 2.0**-23 * (before.abs() + out.abs() + 2 * res.abs() + 1.0 + 8.0)
    return out + res, err


@pytest.mark.parametrize("T,N,K", LARGE)
def test_large_sizes(T, N, K):
    for act, dtype, bias, residual in ((None, BF, None, None), ("silu", torch.float32, torch.float32, BF), ("gelu", BF, BF, torch.float32),
                                       ("relu", torch.float32, None, torch.float32)):
        d = make(T, N, K, T + K, bias=bias, residual=residual)
        got = dense_gemm(**d, act=act, out_dtype=dtype).double()
        out, err = exact_on_gpu(d, act)
        err = err + (out.abs() + err) * torch.finfo(dtype).eps / 2
        off = (got - out).abs()
        assert bool((off <= err).all()), f"{act} {dtype}: {int((off > err).sum())} values outside, the worst {float((off / err).max())} times"


@pytest.mark.parametrize("seed", range(40))
def test_drawn_sizes(seed):
    rng = np.random.default_rng(seed)
    size = lambda hi: int(round(np.exp(rng.uniform(0, np.log(hi)))))  # noqa: E731
    T, N, K = size(3000), size(3000), 8 * size(600)
    pick = lambda *v: v[int(rng.integers(len(v)))]  # noqa: E731
    check(make(T, N, K, seed, bias=pick(None, BF, torch.float32), residual=pick(None, BF, torch.float32), pad=pick(0, 8, 64)),
          act=pick(*ACTS), dtype=pick(BF, torch.float32))


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,N", [(5, 40), (300, 328)])
def test_activations(T, N, act, dtype):
    """Sums from -200 to 200, where every activation has reached its ends."""
    K = 16
    d = make(T, N, K, 7, bias=torch.float32, residual=BF, scale=0.0)
    d["x"] = torch.zeros(T, K, dtype=BF, device=DEV)
    d["x"][:, 0] = 1.0
    d["bias"] = torch.linspace(-200, 200, N, device=DEV) ** 3 / 40000
    d["residual"] = torch.zeros(T, N, dtype=BF, device=DEV)
    check(d, act=act, dtype=dtype)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("T", [5, 300])
def test_activations_far_out(T, act, dtype):
    """Sums of any size, where an activation is at its end: a NaN where the formula has one (minus infinity times
    0), values within 8 * 2^-23 of theirs and their rounding, those below 2^-118 within that (a reciprocal below the
    normal range may be 0)."""
    far = [float("inf"), 3.3e38, 2.4e38, 1e30, 1e20, 1e10, 200.0, 90.0, 87.5]
    d = make(T, 24, 16, 8, scale=0.0)
    d["bias"] = torch.tensor([s * v for v in far for s in (1.0, -1.0)] + [float("nan"), 0.0, -0.0, -88.5, -104.0, -126.5], device=DEV)
    got = host(dense_gemm(**d, act=act, out_dtype=dtype))
    with np.errstate(invalid="ignore"):
        want = ref.activation(host(d["bias"]), act)
        off = np.abs(got - want)
    most = np.abs(want) * (8 * 2.0**-23 + torch.finfo(dtype).eps / 2) + 2.0**-118
    assert (np.isnan(got) == np.isnan(want)).all()
    assert ((off <= most) | (got == want) | np.isnan(want)).all(), (got[0], want)


@pytest.mark.parametrize("T,N,K", [(1, 40, 8192), (9, 100, 4096), (70, 72, 8192), (260, 300, 4096), (513, 520, 2056)])
def test_exact_integers(T, N, K):
    """Integers whose sums FP32 holds: bit-equal whatever the order."""
    g = torch.Generator().manual_seed(K + T)
    x = torch.randint(-15, 16, (T, K), generator=g).to(BF).to(DEV)
    w = torch.randint(-15, 16, (N, K), generator=g).to(BF).to(DEV)
    got = dense_gemm(x, w, out_dtype=torch.float32)
    assert np.array_equal(host(got), host(x) @ host(w).T)


@pytest.mark.parametrize("T", [1, 20, 300])
def test_large_products_cancel(T):
    """2^100 - 2^100 + small: what FP32 keeps beside a large pair in turn."""
    K, N = 512, 64
    x = torch.ones(T, K, dtype=BF, device=DEV)
    w = torch.zeros(N, K, dtype=BF, device=DEV)
    w[:, 0], w[:, 1] = 2.0**100, -(2.0**100)
    w[:, 256:] = 1.0  # in other steps than the pair
    assert torch.equal(dense_gemm(x, w, out_dtype=torch.float32), torch.full((T, N), 256.0, device=DEV))


@pytest.mark.parametrize("T,N,K", [(1, 256, 7168), (16, 256, 7168), (200, 256, 7168), (600, 512, 7168)])
def test_sums_on_average(T, N, K):
    """The root mean square error of FP32 sums: K / 32 additions in a row, each off by
    2^-24 / sqrt 3 of a running sum that grows to the result's size, are sqrt(K / 32 / 2)
    of that; 2^-21 of the results' size is three times it for K = 7168."""
    d = make(T, N, K, 5)
    got = host(dense_gemm(**d, out_dtype=torch.float32))
    out = host(d["x"]) @ host(d["w"]).T
    assert np.sqrt(np.mean((got - out) ** 2)) <= 2.0**-21 * np.sqrt(np.mean(out**2))


@pytest.mark.parametrize("T,N,K", [(3, 40, 72), (40, 264, 200), (300, 300, 328)])
def test_slices(T, N, K):
    """Columns of wider matrices; what lies beside them is NaN and stays out."""
    d = make(T, N, K, 11)
    nan = float("nan")
    wide_x = torch.full((T, K + 48), nan, dtype=BF, device=DEV)
    wide_w = torch.full((N, K + 16), nan, dtype=BF, device=DEV)
    wide_r = torch.full((T, N + 13), nan, dtype=BF, device=DEV)
    x, w, r = wide_x[:, 16:16 + K], wide_w[:, 8:8 + K], wide_r[:, 5:5 + N]
    x.copy_(d["x"])
    w.copy_(d["w"])
    r.normal_(generator=torch.Generator(device=DEV).manual_seed(3))
    got = check(dict(x=x, w=w, residual=r), act="relu")
    assert torch.equal(got, dense_gemm(x.contiguous(), w.contiguous(), act="relu", residual=r.contiguous()))
    # every other row, and FP32 residual rows at odd places
    both = torch.randn(2 * T, N + 3, device=DEV)
    check(dict(x=wide_x.nan_to_num(0.0)[:, :K][::1], w=w, residual=both[::2, 1:N + 1]))


@pytest.mark.parametrize("T,N,K", [(1, 40, 64), (20, 40, 136), (70, 72, 200), (300, 264, 328)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_row_and_column(T, N, K, bad):
    d = make(T, N, K, 13)
    want = dense_gemm(**d)
    t, n = T // 2, N // 3
    d["x"][t, K - 1] = bad
    got = dense_gemm(**d)
    keep = torch.arange(T, device=DEV) != t
    assert torch.equal(got[keep], want[keep]) and not got[t].isfinite().any()
    d = make(T, N, K, 13)
    d["w"][n, 0] = bad
    got = dense_gemm(**d)
    keep = torch.arange(N, device=DEV) != n
    assert torch.equal(got[:, keep], want[:, keep]) and not got[:, n].isfinite().any()


def test_relu_keeps_a_nan():
    x, w = torch.ones(2, 8, dtype=BF, device=DEV), torch.ones(9, 8, dtype=BF, device=DEV)
    x[1, 3] = float("nan")
    got = dense_gemm(x, w, act="relu")
    assert got[1].isnan().all() and (got[0] == 8).all()


@pytest.mark.parametrize("T,N,K", [(1, 256, 7168), (33, 200, 4096), (256, 4096, 7168), (509, 512, 7168), (700, 768, 512), (4500, 2600, 264)])
def test_same_bits_and_rows_alone(T, N, K):
    """A call gives the same bits again, and a row's do not depend on the others' values."""
    d = make(T, N, K, 17, bias=BF)
    a = dense_gemm(**d, out_dtype=torch.float32)
    assert torch.equal(a, dense_gemm(**d, out_dtype=torch.float32))
    other = dict(d, x=d["x"].clone())
    other["x"][: T - 1] *= -3.0
    assert torch.equal(a[T - 1], dense_gemm(**other, out_dtype=torch.float32)[T - 1])


def raw(d, out, workspace=None, nbytes=0, T=None, **over):
    x, w = d["x"], d["w"]
    T, (N, K) = x.shape[0] if T is None else T, w.shape
    a = _block.DenseArgs(T, N, K, 0, 1 if out.dtype == BF else 0, 0, 0, x.stride(0), w.stride(0), N, x.data_ptr(), w.data_ptr(), None,
                         None, out.data_ptr(), workspace, nbytes)
    for n, v in over.items():
        setattr(a, n, v)
    return lib().moe_dense_gemm(ctypes.byref(a), torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("T,N,K", [(1, 30, 64), (13, 33, 136), (100, 130, 1024), (257, 264, 512), (509, 300, 2048), (256, 4091, 7168),
                                   (256, 4096, 7168), (3000, 2603, 72), (4500, 2600, 264)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_nothing_behind_the_output_is_written(T, N, K, dtype):
    d = make(T, N, K, 19)
    need = lib().moe_dense_gemm_workspace(T, N, K)
    ws = torch.full((need + 64,), 170, dtype=torch.uint8, device=DEV)
    out = torch.full((T * N + 64,), 77.0, dtype=dtype, device=DEV)
    assert raw(d, out, ws.data_ptr() if need else None, need) == _capi.OK
    assert (out[T * N:] == 77.0).all() and (ws[need:] == 170).all()
    assert torch.equal(out[: T * N].view(T, N), dense_gemm(**d, out_dtype=dtype))


@pytest.mark.parametrize("T,N,K", [(1, 256, 7168), (200, 256, 7168), (256, 4096, 7168)])
def test_without_a_workspace(T, N, K):
    """The product is right without one, too."""
    d = make(T, N, K, 23)
    out = torch.empty(T, N, dtype=torch.float32, device=DEV)
    assert raw(d, out) == _capi.OK
    exact, err = exact_on_gpu(d, None)
    assert bool(((out.double() - exact).abs() <= err).all())


def test_empty_and_single_rows():
    d = make(0, 40, 64, 1, bias=BF, residual=BF)
    assert dense_gemm(**d).shape == (0, 40)
    # strides of a single row are anything
    x = torch.randn(64, 1, device=DEV).to(BF).t()  # [1, 64], stride (1, 1)
    w = torch.randn(64, device=DEV).to(BF).as_strided((1, 64), (3, 1))
    check(dict(x=x, w=w, residual=torch.randn(1, 1, device=DEV)))


@pytest.mark.parametrize("T,N,K", [(1, 256, 7168), (130, 256, 4096), (256, 4096, 7168), (600, 1024, 512)])
def test_captured_and_replayed(T, N, K):
    """Two calls in one graph, replayed with eager work between, new inputs each time."""
    d = make(T, N, K, 29, bias=BF)
    e = make(T, K, N, 30)
    d["w"], y = d["w"], None
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for _ in range(2):
            y = dense_gemm(**d, act="silu")
            z = dense_gemm(y, e["w"], out_dtype=torch.float32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = dense_gemm(**d, act="silu")
        z = dense_gemm(y, e["w"], out_dtype=torch.float32)
    for seed in (1, 2, 3):
        d["x"].copy_(make(T, N, K, seed)["x"])
        graph.replay()
        eager = dense_gemm(**d, act="silu")
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(z, dense_gemm(eager, e["w"], out_dtype=torch.float32))


def test_two_streams_and_a_given_stream():
    """Calls in flight at once have workspaces of their own."""
    a, b = make(256, 4096, 7168, 31), make(256, 4096, 7168, 32)
    assert lib().moe_dense_gemm_workspace(256, 4096, 7168)
    wa, wb = dense_gemm(**a), dense_gemm(**b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(s1):
            got.append((wa, dense_gemm(**a)))
        got.append((wb, dense_gemm(**b, stream=s2)))
    torch.cuda.synchronize()
    assert all(torch.equal(want, have) for want, have in got)


def test_offsets_past_32_bits():
    """Rows 2^23 - 8 values apart, the largest stride, so that offsets of x, w and the
    residual pass 2^32 values; outputs past 2^31 values."""
    K, N, T, ld = 64, 24, 600, 2**23 - 8
    big = torch.empty(T * ld, dtype=BF, device=DEV)
    x, r, w = big.as_strided((T, K), (ld, 1)), big.as_strided((T, N), (ld, 1), 1024), big.as_strided((T, K), (ld, 1), 2048)
    for t in (x, r, w):
        t.normal_()
    assert T * ld > 2**32
    check(dict(x=x, w=torch.randn(N, K, device=DEV).to(BF), residual=r))
    check(dict(x=torch.randn(5, K, device=DEV).to(BF), w=w))
    check(dict(x=x, w=w))
    wide = w
    del big, x, r, wide
    T, N = 300000, 7200
    x, w = torch.randn(T, 8, device=DEV).to(BF), torch.randn(N, 8, device=DEV).to(BF)
    out = dense_gemm(x, w)
    assert T * N > 2**31
    rows = torch.tensor([0, 1, T // 2, 298260, 298262, T - 1], device=DEV)
    exact = host(x[rows]) @ host(w).T
    most = bound(dict(x=x[rows], w=w), 8, None, exact, exact, BF)
    assert (np.abs(host(out[rows]) - exact) <= most).all()


def test_other_dtypes_of_views():
    """A weight that is a half of a fused matrix, an x that is one token of a batch."""
    fused = torch.randn(2 * 40, 128, device=DEV).to(BF)
    x = torch.randn(6, 4, 128, device=DEV).to(BF)
    check(dict(x=x[:, 1], w=fused[40:]))
    check(dict(x=x[2], w=fused[::2]))
