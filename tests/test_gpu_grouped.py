"""moe_grouped_gemm and moe_grouped_swiglu on the GPU against the formula in
64 bits (torch FP64 products per expert; the inputs are e4m3 codes and
binary32 scales, exact in FP64).

Bound of the product: a 128-wide block's exact products are added in FP32 (at
most 127 additions in some order), its scales are applied in at most three
FP32 operations, and the K/128 partials are added in FP32. With an error of
one unit 2^-23 each (either rounding or truncation), the result is within
(128 + K/128 + 3) * 2^-23 * sum |terms| of the exact one. So it is for the
SwiGLU, whose codes are decided from these sums.

moe_grouped_gemm, whose rows are rounded to BF16, uses the FP8 matrix
instruction, which adds eight products at a time, each cut off 14 bits below
the power of two of the group's largest (measured one product at a time; the
sums of eight are then added in FP32). Seven products of a group lose at most
2^-14 of its largest one each: 7 * 2^-14 * sum |terms| more, at the very most.
The BF16 output is the rounding of such a value: between the roundings of
exact -+ bound."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from fp8_block_scaled_moe_amd import grouped_gemm, grouped_swiglu

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F8 = torch.float8_e4m3fn
LIMIT = 7.0


def codes(gen, shape, std):
    return (torch.randn(shape, generator=gen, device=DEV) * std).clamp(-448, 448).to(F8)


def make(counts, N, K, seed, quant="fp8", gather=False, std=107.0, extra=3):
    """Inputs for experts with these row counts; with gather the rows are
    drawn, with repeats, from fewer tokens; `extra` rows lie behind the last."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    E, R = len(counts), sum(counts)
    X = max(1, R // 2 + 1) if gather else R + extra
    d = {"w": codes(gen, (E, N, K), std), "w_scale": torch.rand(E, N // 128, K // 128, generator=gen, device=DEV) * 1.5 + 0.5}
    d["w_scale"] /= std * K**0.5
    d["x"] = codes(gen, (X, K), 100.0)
    if quant == "fp8":
        d["x_scale"] = torch.exp2(torch.randn(X, K // 128, generator=gen, device=DEV)) / 100.0
    else:
        d["x_scale"] = torch.randint(115, 125, (X, K // 32), generator=gen, device=DEV).to(torch.uint8)
    d["offsets"] = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
    d["rows"] = torch.randint(0, X, (R + extra,), generator=gen, device=DEV, dtype=torch.int32) if gather else None
    return d


def exact(d, more=0.0):
    """(g, its bound) in FP64 for the rows up to offsets[-1]."""
    ends = d["offsets"].tolist()
    K = d["x"].shape[1]
    x = d["x"].double()
    if d["x_scale"].dtype == torch.uint8:
        x = x * torch.exp2(d["x_scale"].double() - 127).repeat_interleave(32, 1)
    else:
        x = x * d["x_scale"].double().repeat_interleave(128, 1)
    if d["rows"] is not None:
        ok = (d["rows"] >= 0) & (d["rows"] < x.shape[0])
        x = torch.where(ok[:, None], x[d["rows"].long().clamp(0, x.shape[0] - 1)], torch.zeros((), dtype=torch.float64, device=DEV))
    g = torch.zeros(ends[-1], d["w"].shape[1], dtype=torch.float64, device=DEV)
    t = torch.zeros_like(g)
    for e in range(len(ends) - 1):
        lo, hi = ends[e], ends[e + 1]
        if hi > lo:
            w = d["w"][e].double() * d["w_scale"][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            g[lo:hi] = x[lo:hi] @ w.t()
            t[lo:hi] = x[lo:hi].abs() @ w.abs().t()
    return g, t * ((128 + K // 128 + 3) * 2.0**-23 + more)


def call_gemm(d):
    return grouped_gemm(d["x"], d["x_scale"], d["w"], d["w_scale"], d["offsets"], rows=d["rows"])


def check_gemm(d, more=0.0):
    y = call_gemm(d)
    g, bound = exact(d, 7 * 2.0**-14)
    n = g.shape[0]
    got = y[:n].double()
    # a value within the bound, rounded once; BF16 rounding is monotone
    bf16 = lambda v: v.float().to(torch.bfloat16).double()  # noqa: E731
    bad = (got < bf16(g - bound - more)) | (got > bf16(g + bound + more))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values outside, first at {torch.nonzero(bad)[0].tolist()}"
    return y


def check_swiglu(d):
    h, s = grouped_swiglu(d["x"], d["x_scale"], d["w"], d["w_scale"], d["offsets"], limit=LIMIT, rows=d["rows"])
    g, bound = exact(d)
    n, I = g.shape[0], g.shape[1] // 2
    up, gate = g[:, :I].clamp(-LIMIT, LIMIT), g[:, I:].clamp_max(LIMIT)
    silu = gate * torch.sigmoid(gate)
    act = silu * up
    # |silu'| < 1.1; the hardware's exp2 and reciprocal and the FP32 steps
    # around them: |gate| + 4 units of 2^-23
    err = 1.1 * bound[:, I:] * up.abs() + (silu.abs() + 1.1 * bound[:, I:]) * bound[:, :I] + act.abs() * (gate.abs() + 4) * 2.0**-23
    block = lambda v: v.view(n, I // 128, 128).amax(-1)  # noqa: E731
    sg = s[:n].double()
    ws = block(act.abs()).clamp_min(1e-10) / 448.0
    assert ((sg - ws).abs() <= block(err) / 448.0 + ws * 2.0**-23).all(), "scales"
    # the code is the rounding of a value within the error of act / scale
    # (scale as returned; its reciprocal and the product round once each)
    spread = sg.repeat_interleave(128, 1)
    e = err + act.abs() * 2.0**-22
    f8 = lambda v: v.clamp(-448, 448).float().to(F8).double()  # noqa: E731
    lo, hi = f8((act - e) / spread), f8((act + e) / spread)
    got = h[:n].view(F8).double()
    bad = (got < lo) | (got > hi)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} codes outside, first at {torch.nonzero(bad)[0].tolist()}"
    return h, s


RAGGED = [0, 1, 15, 16, 17, 0, 63, 64, 65, 2]
BIG = [127, 128, 129, 0, 255, 256, 257, 300, 1, 513]


@pytest.mark.parametrize("quant", ["fp8", "mxfp8"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 5], RAGGED, BIG, [0, 0, 700]], ids=["one", "few", "ragged", "big", "last"])
def test_gemm_counts(counts, gather, quant):
    check_gemm(make(counts, 384, 640, 1, quant, gather))


@pytest.mark.parametrize("quant", ["fp8", "mxfp8"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 5], RAGGED, BIG, [0, 0, 700]], ids=["one", "few", "ragged", "big", "last"])
def test_swiglu_counts(counts, gather, quant):
    check_swiglu(make(counts, 768, 640, 2, quant, gather))


@pytest.mark.parametrize("N,K", [(128, 128), (128, 256), (256, 384), (640, 128), (1408, 1408), (256, 7168), (7168, 256), (512, 16384)])
@pytest.mark.parametrize("counts", [[2, 0, 1], [5, 40, 9], [150, 30, 290]], ids=["few", "some", "many"])
def test_gemm_sizes(N, K, counts):
    check_gemm(make(counts, N, K, 3))


@pytest.mark.parametrize("I,K", [(128, 128), (128, 512), (384, 256), (1408, 1408), (256, 7168), (2048, 256)])
@pytest.mark.parametrize("counts", [[2, 0, 1], [5, 40, 9], [150, 30, 290]], ids=["few", "some", "many"])
def test_swiglu_sizes(I, K, counts):
    check_swiglu(make(counts, 2 * I, K, 4))


@pytest.mark.parametrize("E,R", [(1, 1), (1, 1000), (256, 40), (300, 2000), (1024, 100), (1024, 5000), (257, 20000)])
def test_many_experts(E, R):
    counts = np.bincount(np.random.default_rng(E + R).integers(0, E, R), minlength=E).tolist()
    check_gemm(make(counts, 256, 256, 5, gather=True))
    check_swiglu(make(counts, 256, 256, 6, gather=True))


def test_exact_integers():
    """Small integers and power-of-two scales: every sum is exact in FP32, so
    the output has to be the exact value's BF16 rounding, whichever order it
    is summed in."""
    for counts in ([3, 0, 20], [100, 260]):
        for quant in ("fp8", "mxfp8"):
            d = make(counts, 256, 512, 7, quant)
            gen = torch.Generator(device=DEV).manual_seed(8)
            d["x"] = torch.randint(-7, 8, d["x"].shape, generator=gen, device=DEV).float().to(F8)
            d["w"] = torch.randint(-7, 8, d["w"].shape, generator=gen, device=DEV).float().to(F8)
            d["w_scale"] = torch.exp2(torch.randint(-2, 3, d["w_scale"].shape, generator=gen, device=DEV).float())
            if quant == "fp8":
                d["x_scale"] = torch.exp2(torch.randint(-2, 3, d["x_scale"].shape, generator=gen, device=DEV).float())
            else:
                d["x_scale"] = torch.randint(125, 130, d["x_scale"].shape, generator=gen, device=DEV).to(torch.uint8)
            assert torch.equal(call_gemm(d)[: sum(counts)], exact(d)[0].float().to(torch.bfloat16))


def test_every_code():
    """All finite e4m3 codes in x and w, subnormals among them."""
    d = make([40, 3], 256, 512, 9)
    finite = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(10)
    for n in ("x", "w"):
        d[n] = finite[torch.randint(0, 254, d[n].shape, generator=gen, device=DEV)].view(F8)
    check_gemm(d)


def test_e8m0_range():
    """E8M0 bytes over the range whose products stay finite, 0 included."""
    d = make([20, 100], 256, 512, 11, "mxfp8")
    gen = torch.Generator(device=DEV).manual_seed(12)
    d["x_scale"] = torch.randint(0, 200, d["x_scale"].shape, generator=gen, device=DEV).to(torch.uint8)
    d["x_scale"][0, :] = 0
    d["w_scale"][:] = 1.0
    check_gemm(d, 2.0**-126)  # results below the smallest normal may be flushed


@pytest.mark.parametrize("counts", [[3, 2], [40, 30], [300, 200]], ids=["few", "some", "many"])
def test_e8m0_scales_far_apart(counts):
    """A block's 32 positions with a scale 2^30 above their neighbours', whose
    codes (then whose weights) are zero: the neighbours' products are all
    there is, and no bit of them may be lost."""
    d = make(counts, 256, 512, 27, "mxfp8")
    gen = torch.Generator(device=DEV).manual_seed(28)
    s = torch.randint(100, 105, d["x_scale"].shape, generator=gen, device=DEV)
    s[:, 1::4] = 135
    d["x_scale"] = s.to(torch.uint8)
    d["w_scale"] *= 2.0**18
    far = (torch.arange(512, device=DEV) // 32) % 4 == 1
    for n in ("x", "w"):
        full = d[n].clone()
        d[n].view(torch.uint8)[..., far] = 0
        check_gemm(d)
        check_swiglu(d)
        d[n] = full


@pytest.mark.parametrize("counts", [[3, 1], [40, 30], [300, 200]], ids=["few", "some", "many"])
def test_rows_behind_the_last_stay(counts):
    """Rows of the output from offsets[E] on are left as they were."""
    import ctypes
    from fp8_block_scaled_moe_amd import _rows, lib

    d = make(counts, 256, 256, 13, extra=50)
    R, n = d["x"].shape[0], sum(counts)
    st = torch.cuda.current_stream().cuda_stream
    sizes = (R, R, len(counts), 256, 256, 1)
    ptrs = (d["x"].data_ptr(), d["x_scale"].data_ptr(), None, d["offsets"].data_ptr(), d["w"].data_ptr(), d["w_scale"].data_ptr())
    out = torch.full((R, 256), 3.0, dtype=torch.bfloat16, device=DEV)
    assert lib().moe_grouped_gemm(ctypes.byref(_rows.GroupedArgs(*sizes, 0.0, *ptrs, out.data_ptr(), None)), st) == 0
    assert (out[n:] == 3.0).all() and torch.equal(out[:n], call_gemm(d)[:n])
    h, s = torch.full((R, 128), 9, dtype=torch.uint8, device=DEV), torch.full((R, 1), 5.0, device=DEV)
    a = _rows.GroupedArgs(*sizes, LIMIT, *ptrs, h.data_ptr(), s.data_ptr())
    assert lib().moe_grouped_swiglu(ctypes.byref(a), st) == 0
    assert (h[n:] == 9).all() and (s[n:] == 5.0).all()


def parts(d, glu):
    """Parts of K that the call's workspace is for (1: none)."""
    from fp8_block_scaled_moe_amd import lib

    R = d["x"].shape[0] if d["rows"] is None else d["rows"].shape[0]
    E, N, K = d["w"].shape
    f = lib().moe_grouped_swiglu_workspace if glu else lib().moe_grouped_gemm_workspace
    return max(1, f(R, E, N, K) // (R * N * 4))


# few and ragged rows, with a K that is split unevenly
@pytest.mark.parametrize("quant", ["fp8", "mxfp8"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 5], RAGGED, [150, 0, 300]], ids=["one", "few", "ragged", "many"])
def test_split_over_k(counts, gather, quant):
    d = make(counts, 256, 128 * 37, 29, quant, gather)
    assert parts(d, False) > 1 and parts(d, True) > 1
    n = sum(counts)
    y, (h, s) = check_gemm(d), check_swiglu(d)
    again, (h2, s2) = call_gemm(d), grouped_swiglu(d["x"], d["x_scale"], d["w"], d["w_scale"], d["offsets"], limit=LIMIT, rows=d["rows"])
    assert torch.equal(y[:n], again[:n]) and torch.equal(h[:n], h2[:n]) and torch.equal(s[:n], s2[:n])


@pytest.mark.parametrize("K", [2048, 2176, 16384])
def test_split_sizes(K):
    """The shortest split K, one block more, a long one; an odd tile of columns."""
    d = make([2, 0, 1, 30], 384, K, 30)
    assert parts(d, False) > 1
    check_gemm(d)
    d = make([2, 0, 1, 30], 768, K, 31)
    assert parts(d, True) > 1
    check_swiglu(d)


def test_long_k_turned():
    """K = 4096, enough tiles not to be split: tiles of an expert with one row
    tile begin at blocks of their own, others at the first, with the same sums."""
    counts = [(7 * e) % 23 for e in range(38)] + [140, 300]
    d = make(counts, 1024, 4096, 36, gather=True)
    assert parts(d, False) == parts(d, True) == 1
    check_gemm(d)
    h, s = check_swiglu(d)
    again = grouped_swiglu(d["x"], d["x_scale"], d["w"], d["w_scale"], d["offsets"], limit=LIMIT, rows=d["rows"])
    n = sum(counts)
    assert torch.equal(h[:n], again[0][:n]) and torch.equal(s[:n], again[1][:n])


def test_split_calls_captured_and_at_once():
    """Split calls in two graphs and on two streams: each replay, with eager
    calls and new inputs between them, equals the eager result."""
    ds = [make([3, 0, 17], 256, 2048, 33 + i, extra=0) for i in range(2)]
    both = lambda d: (call_gemm(d), *grouped_swiglu(d["x"], d["x_scale"], d["w"], d["w_scale"], d["offsets"], limit=LIMIT))  # noqa: E731
    assert all(parts(d, glu) > 1 for d in ds for glu in (False, True))
    for d in ds:
        both(d)
    torch.cuda.synchronize()
    graphs = []
    for d in ds:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(d)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in ds]
    gen = torch.Generator(device=DEV).manual_seed(35)
    for _ in range(4):
        for d in ds:
            d["x"].copy_(codes(gen, d["x"].shape, 100.0))
        want = [both(d) for d in ds]
        torch.cuda.synchronize()
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        eager = []
        for d, st in zip(ds, streams):
            with torch.cuda.stream(st):
                eager.append(both(d))
        torch.cuda.synchronize()
        for w, e, (_, o) in zip(want, eager, graphs):
            assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(w, e, o))


def test_split_leaves_other_rows_alone():
    """With a workspace, as without: rows behind the last and before the first
    group stay, rows with an index out of range are zeros, a NaN stays in its
    row; a workspace past the need is not written behind it."""
    import ctypes
    from fp8_block_scaled_moe_amd import _rows, lib

    d = make([7, 40], 256, 2048, 32, gather=True, extra=9)
    d["rows"][5], d["rows"][20] = -1, 2**30
    d["x"].view(torch.uint8)[int(d["rows"][11]), 1500] = 0x7F
    d["offsets"][0] = 2
    R, L, st = d["rows"].shape[0], lib(), torch.cuda.current_stream().cuda_stream
    nan = (d["rows"] == d["rows"][11])[2:47]
    zero = torch.zeros(45, dtype=torch.bool, device=DEV)
    zero[[3, 18]] = True
    ptrs = (d["x"].data_ptr(), d["x_scale"].data_ptr(), d["rows"].data_ptr(), d["offsets"].data_ptr(), d["w"].data_ptr(),
            d["w_scale"].data_ptr())
    for glu in (False, True):
        need = (L.moe_grouped_swiglu_workspace if glu else L.moe_grouped_gemm_workspace)(R, 2, 256, 2048)
        assert need > 0
        ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        out = torch.full((R, 128 if glu else 512), 9, dtype=torch.uint8, device=DEV)
        s = torch.full((R, 1), 5.0, device=DEV)
        a = _rows.GroupedArgs(R, d["x"].shape[0], 2, 256, 2048, 1, LIMIT, *ptrs, out.data_ptr(), s.data_ptr(), ws.data_ptr(), need)
        assert (L.moe_grouped_swiglu if glu else L.moe_grouped_gemm)(ctypes.byref(a), st) == 0
        torch.cuda.synchronize()
        assert (ws[need:] == 0x5A).all()
        for t, was in ((out, 9), (s, 5.0)):
            assert (t[:2] == was).all() and (t[47:] == was).all()
        rows = out[2:47]
        assert not rows[zero].any()
        if glu:
            assert ((rows[nan] & 0x7F) == 0x7F).all() and not ((rows[~nan] & 0x7F) == 0x7F).any()
        else:
            y = out.view(torch.bfloat16)[2:47]
            assert torch.isnan(y[nan]).all() and not torch.isnan(y[~nan]).any()


@pytest.mark.parametrize("counts", [[4, 2], [40, 30], [300, 200]], ids=["few", "some", "many"])
def test_rows_outside_give_zeros(counts):
    d = make(counts, 256, 256, 14, gather=True, extra=0)
    d["rows"][1], d["rows"][-1], d["rows"][2] = -1, d["x"].shape[0], -(2**31)
    y = check_gemm(d)
    assert not y[[1, 2, -1]].any()
    h, s = check_swiglu(d)
    assert not h[[1, 2, -1]].any()


@pytest.mark.parametrize("counts", [[4, 2], [40, 30], [300, 200]], ids=["few", "some", "many"])
def test_offsets_outside_are_clamped(counts):
    """Offsets past R or below 0 end at R or begin at 0."""
    d = make(counts, 256, 256, 15, extra=0)
    want = call_gemm(d)
    d["offsets"][0], d["offsets"][-1] = -5, 2**31 - 1
    assert torch.equal(call_gemm(d), want)


@pytest.mark.parametrize("counts", [[4, 2], [40, 30], [300, 200]], ids=["few", "some", "many"])
def test_rows_before_the_first_stay(counts):
    """Offsets that do not begin at 0: the rows before the first expert's are
    no expert's."""
    d = make(counts, 256, 256, 24, extra=0)
    want = call_gemm(d)
    full = d["offsets"].clone()
    d["offsets"][0] = 3
    y = call_gemm(d)
    assert torch.equal(y[3:], want[3:])
    d["offsets"][:] = full


def test_offsets_in_disorder_stay_inside():
    """Offsets that do not ascend give some rows or other, and leave those
    from the last offset's clamp on and everything around the output alone."""
    import ctypes
    from fp8_block_scaled_moe_amd import _rows, lib

    d = make([100] * 8, 256, 256, 25, extra=0)
    d["offsets"][:] = torch.tensor([0, 700, 20, 5, -9, 300, 2**31 - 1, 90, 400], dtype=torch.int32)
    R = d["x"].shape[0]
    big = torch.full((R + 64, 256), 3.0, dtype=torch.bfloat16, device=DEV)
    out = big[32:32 + R]
    a = _rows.GroupedArgs(R, R, 8, 256, 256, 1, 0.0, d["x"].data_ptr(), d["x_scale"].data_ptr(), None, d["offsets"].data_ptr(),
                          d["w"].data_ptr(), d["w_scale"].data_ptr(), out.data_ptr(), None)
    assert lib().moe_grouped_gemm(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert (big[:32] == 3.0).all() and (big[32 + R:] == 3.0).all()


def test_a_share_of_many_rows():
    """Room for many more rows than there are (one GPU's share): the same
    bits as with room for just these."""
    d = make([70, 0, 200, 30], 512, 384, 26, gather=True, extra=0)
    want, (wh, ws) = call_gemm(d), check_swiglu(d)
    d["rows"] = torch.cat([d["rows"], torch.full((9000,), -3, dtype=torch.int32, device=DEV)])
    assert torch.equal(call_gemm(d)[:300], want)
    h, s = grouped_swiglu(d["x"], d["x_scale"], d["w"], d["w_scale"], d["offsets"], limit=LIMIT, rows=d["rows"])
    assert torch.equal(h[:300], wh) and torch.equal(s[:300], ws)


@pytest.mark.parametrize("counts", [[4, 2], [40, 30], [300, 200]], ids=["few", "some", "many"])
def test_nan_stays_in_its_row(counts):
    """A NaN code in a row of x, or in another expert's weights, reaches only
    the rows that contain it."""
    d = make(counts, 256, 256, 16, extra=0)
    want_y, want_h = call_gemm(d), check_swiglu(d)
    d["x"].view(torch.uint8)[1, 77] = 0x7F
    y = call_gemm(d)
    keep = torch.arange(y.shape[0], device=DEV) != 1
    assert torch.isnan(y[1]).all() and torch.equal(y[keep], want_y[keep])
    h, s = grouped_swiglu(d["x"], d["x_scale"], d["w"], d["w_scale"], d["offsets"], limit=LIMIT)
    assert ((h[1] & 0x7F) == 0x7F).all() and torch.equal(h[keep], want_h[0][keep]) and torch.equal(s[keep], want_h[1][keep])
    d = make(counts, 256, 256, 16, extra=0)
    d["w"].view(torch.uint8)[1, 200, 100] = 0xFF
    y = call_gemm(d)
    assert torch.isnan(y[counts[0] :, 200]).all()
    assert torch.equal(y[: counts[0]], want_y[: counts[0]])
    cols = torch.arange(256, device=DEV) != 200
    assert torch.equal(y[:, cols], want_y[:, cols])


def test_saturated_swiglu():
    """Large products: both clamps act, a very negative gate gives zero."""
    for counts in ([3, 2], [300, 200]):
        d = make(counts, 512, 256, 17)
        d["w_scale"] *= 1000.0
        check_swiglu(d)


def test_zero_inputs():
    d = make([2, 0, 40], 256, 256, 18)
    d["x"] = torch.zeros_like(d["x"].view(torch.uint8)).view(F8)
    assert not call_gemm(d)[:42].any()
    h, s = check_swiglu(d)
    assert not h[:42].any() and torch.equal(s[:42], torch.full_like(s[:42], np.float32(1e-10) / np.float32(448.0)))


def test_empty():
    d = make([1], 256, 256, 19, extra=0)
    d["x"], d["x_scale"] = d["x"][:0], d["x_scale"][:0]
    d["offsets"].zero_()
    assert call_gemm(d).shape == (0, 256)
    h, s = grouped_swiglu(d["x"], d["x_scale"], d["w"], d["w_scale"], d["offsets"], limit=LIMIT)
    assert h.shape == (0, 128) and s.shape == (0, 1)
    d = make([3, 2], 256, 256, 20)  # rows, but none of them grouped
    d["offsets"].zero_()
    call_gemm(d)
    torch.cuda.synchronize()


@pytest.mark.parametrize("counts", [[4, 2], [40, 30], [300, 200]], ids=["few", "some", "many"])
def test_same_bits_every_time_and_wherever_a_row_stands(counts):
    """No order-dependent sums: a repeated call is bit-identical, and a row's
    result does not depend on its place among the rows of its expert."""
    d = make(counts, 512, 640, 21, extra=0)
    a, b = call_gemm(d), call_gemm(d)
    assert torch.equal(a, b)
    d["rows"] = torch.cat([torch.arange(counts[0]).flip(0), counts[0] + torch.arange(counts[1]).flip(0)]).int().to(DEV)
    assert torch.equal(call_gemm(d)[d["rows"].long()], a)


def test_weights_past_32_bits():
    """Expert offsets past 4 GiB: the last of 300 experts of 2048 x 7168."""
    E, N, K = 300, 2048, 7168
    big = make([6], N, K, 23, extra=0)
    w = torch.zeros(E, N, K, dtype=torch.uint8, device=DEV)
    w[-1] = big["w"][0].view(torch.uint8)
    ws = torch.zeros(E, N // 128, K // 128, device=DEV)
    ws[-1] = big["w_scale"][0]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[-1] = 6
    y = grouped_gemm(big["x"], big["x_scale"], w, ws, offsets)
    g, bound = exact(big, 7 * 2.0**-14)
    bf16 = lambda v: v.float().to(torch.bfloat16).double()  # noqa: E731
    assert ((y.double() >= bf16(g - bound)) & (y.double() <= bf16(g + bound))).all()


def bf16(v):
    return v.float().to(torch.bfloat16).double()


def check_gemm_sums(d):
    """As check_gemm, within the bound of FP32 sums, and closer still on
    average. The instructions leave a block's sum of 128 off by less than 2^-26
    of its typical size (measured over random codes), and each of the K/128
    additions rounds by half a unit at most, at random: sqrt(K/128) * 2^-24,
    at most 2^-21 of a row's root mean square here. A value that is off by e
    before its rounding lands on the neighbour, a step away, once in step / 2e
    times, so the mean square of the rows' distance from the exact ones,
    rounded, is at most 2 e step; a step is at most 2^-7 of the value:
    sqrt(2 * 2^-21 * 2^-7) < 2^-13 of the root mean square. The sums of the FP8
    instruction (2^-16) are twice as far off."""
    y = call_gemm(d)
    g, bound = exact(d)
    got = y[: g.shape[0]].double()
    bad = (got < bf16(g - bound)) | (got > bf16(g + bound))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values outside, first at {torch.nonzero(bad)[0].tolist()}"
    off = (got - bf16(g)).square().mean().sqrt() / g.square().mean().sqrt()
    assert off <= 2.0**-13, f"off by {off:.3g} of the root mean square"
    return y


# few rows, all tiles' heights, K split and K turned
@pytest.mark.parametrize("quant", ["fp8", "mxfp8"])
@pytest.mark.parametrize("counts,N,K", [([70], 1408, 640), (RAGGED, 640, 1408), (BIG, 384, 1024), ([150, 0, 300], 256, 7168),
                                        ([(7 * e) % 23 for e in range(38)] + [140, 300], 1024, 4096)],
                         ids=["one", "ragged", "big", "split", "turned"])
def test_gemm_sums_in_fp32(counts, N, K, quant):
    check_gemm_sums(make(counts, N, K, 41, quant, gather=True))


@pytest.mark.parametrize("quant", ["fp8", "mxfp8"])
@pytest.mark.parametrize("counts,N,K", [([3], 128, 128), (BIG, 384, 512), ([5, 0, 140], 256, 2048)], ids=["one", "big", "split"])
def test_large_products_that_cancel(counts, N, K, quant):
    """Two products of 448 * 448 of opposite signs in each group of eight
    columns, the others multiples of 2^-4 up to 7: all sums are multiples of
    2^-4 below 2^19 and so exact in FP32, and the small products are the
    result, so the output has to be its BF16 rounding."""
    d = make(counts, N, K, 42, quant)
    gen = torch.Generator(device=DEV).manual_seed(43)
    small = lambda shape: (torch.randint(-7, 8, shape, generator=gen, device=DEV) * 0.25)  # noqa: E731
    x, w = small(d["x"].shape), small(d["w"].shape)
    x[:, 0::8], x[:, 5::8] = 448.0, 448.0
    w[..., 0::8], w[..., 5::8] = 448.0, -448.0
    d["x"], d["w"] = x.to(F8), w.to(F8)
    d["w_scale"].fill_(1.0)
    if quant == "fp8":
        d["x_scale"].fill_(1.0)
    else:
        d["x_scale"].fill_(127)
    g, _ = exact(d)
    assert g.abs().max() < 2.0**12
    assert torch.equal(call_gemm(d)[: g.shape[0]], g.float().to(torch.bfloat16))


def fp8_sums(d):
    return grouped_gemm(d["x"], d["x_scale"], d["w"], d["w_scale"], d["offsets"], rows=d["rows"], sums="fp8")


# on the FP8 instruction, within its bound: every tile's height, K split, turned and neither
@pytest.mark.parametrize("quant", ["fp8", "mxfp8"])
@pytest.mark.parametrize("counts,N,K", [([1], 128, 128), (RAGGED, 384, 640), (BIG, 384, 640), ([40, 100, 170, 230], 256, 1024),
                                        ([2, 0, 150, 300], 256, 128 * 37), ([(7 * e) % 23 for e in range(38)] + [140, 300], 1024, 4096)],
                         ids=["one", "ragged", "big", "heights", "split", "turned"])
def test_gemm_sums_of_the_fp8_instruction(counts, N, K, quant):
    d = make(counts, N, K, 44, quant, gather=True)
    d["rows"][0] = -1
    y = fp8_sums(d)
    g, bound = exact(d, 7 * 2.0**-14)
    n = g.shape[0]
    got = y[:n].double()
    assert ((got >= bf16(g - bound)) & (got <= bf16(g + bound))).all()
    assert not y[0].any() and torch.equal(fp8_sums(d)[:n], y[:n])
    d["x"].view(torch.uint8)[int(d["rows"][n - 1]), 77] = 0x7F
    nan = (d["rows"][:n] == d["rows"][n - 1]) & (d["rows"][:n] >= 0)
    z = fp8_sums(d)[:n]
    assert torch.isnan(z[nan]).all() and torch.equal(z[~nan], y[:n][~nan])


def far_apart(counts, N, K, seed, apart, zeros, every=1):
    """A block's second 32 positions with a scale 2^apart above the others',
    whose codes (`zeros` "x") or whose weights ("w") are zero, in every
    `every`-th row (the others have scales alike), and weight scales that make the
    results of the order of one."""
    d = make(counts, N, K, seed, "mxfp8")
    gen = torch.Generator(device=DEV).manual_seed(seed + 1)
    low = min(100, 254 - apart)
    s = torch.randint(max(low - 4, 0), low + 1, d["x_scale"].shape, generator=gen, device=DEV)
    s[::every, 1::4] = low + apart
    d["x_scale"] = s.to(torch.uint8)
    d["w_scale"] *= 2.0 ** (127 - low) / 100.0
    at = (torch.arange(K, device=DEV) // 32) % 4 == 1
    if zeros == "x":
        d["x"].view(torch.uint8)[::every, at] = 0
    else:
        d["w"].view(torch.uint8)[..., at] = 0
    return d


@pytest.mark.parametrize("zeros", ["x", "w"])
@pytest.mark.parametrize("apart", [64, 96, 97, 112, 120, 126, 127, 160, 254])
@pytest.mark.parametrize("counts,N,K", [([3, 40], 256, 512), ([150, 20, 300], 256, 256), ([2, 33], 256, 2048 + 128)],
                         ids=["few", "many", "split"])
def test_e8m0_scales_any_distance_apart(counts, N, K, apart, zeros):
    d = far_apart(counts, N, K, 45, apart, zeros)
    assert not torch.isnan(check_gemm(d, 2.0**-126)[: sum(counts)]).any()
    check_swiglu(d)


@pytest.mark.parametrize("counts", [[3, 40], [150, 20, 300]], ids=["few", "many"])
def test_rows_with_scales_far_apart_beside_others(counts):
    """Every third row only: each is right, and the others have the bits that
    they have among their like."""
    d = far_apart(counts, 512, 384, 47, 140, "x", every=3)
    y, (h, s) = check_gemm(d, 2.0**-126), check_swiglu(d)
    d["x_scale"][::3, 1::4] = d["x_scale"][::3, 0::4]  # nothing far apart any more
    y2, (h2, s2) = check_gemm(d), check_swiglu(d)
    n = sum(counts)
    keep = torch.arange(n, device=DEV) % 3 != 0
    assert torch.equal(y[:n][keep], y2[:n][keep])
    assert torch.equal(h[:n][keep], h2[:n][keep]) and torch.equal(s[:n][keep], s2[:n][keep])


@pytest.mark.parametrize("counts", [[3, 40], [150, 20, 300]], ids=["few", "many"])
def test_e8m0_bytes_from_0_to_230(counts):
    """Bytes all over the range, 0 among them: the largest of a row decide."""
    d = make(counts, 256, 512, 48, "mxfp8")
    gen = torch.Generator(device=DEV).manual_seed(49)
    d["x_scale"] = torch.randint(0, 231, d["x_scale"].shape, generator=gen, device=DEV).to(torch.uint8)
    d["w_scale"] *= 2.0**-110
    check_gemm(d, 2.0**-126)
    check_swiglu(d)


@pytest.mark.parametrize("split", [False, True])
def test_swiglu_exponential(split):
    """One hidden value a row, gate -+x and up x / 4 for a scale x of the row,
    so that the hidden's scale tells it: gates from -20 to 7, none less exact
    than others. The hardware's exponential and reciprocal are within a unit of
    2^-23 each, the constant's rounding is another 20 / 42, and 1 + e, its
    correction, the two products and the division by 448 round by a half each: 5."""
    K = 2048 if split else 128
    R = 4000 if not split else 200
    gen = torch.Generator(device=DEV).manual_seed(50)
    xs = torch.rand(R, generator=gen, device=DEV) * 20.0 + 0.01
    one = torch.tensor(1.0, device=DEV).to(F8)
    x, w = torch.zeros(R, K, device=DEV).to(F8), torch.zeros(2, 256, K, device=DEV).to(F8)
    x[:, 5] = one
    w[:, 7, 5] = (one.float() / 4).to(F8)            # up
    w[0, 128 + 7, 5], w[1, 128 + 7, 5] = one, (-one.float()).to(F8)  # gate
    scale = torch.ones(R, K // 128, device=DEV)
    scale[:, 0] = xs
    offsets = torch.tensor([0, R // 2, R], dtype=torch.int32, device=DEV)
    _, s = grouped_swiglu(x, scale, w, torch.ones(2, 2, K // 128, device=DEV), offsets, limit=7.0)
    g = torch.where(torch.arange(R, device=DEV) < R // 2, xs, -xs).double().clamp_max(7.0)
    act = (g * torch.sigmoid(g) * (xs.double() / 4)).abs()
    assert act.min() > 1e-9
    assert ((s[:, 0].double() * 448.0 - act).abs() <= act * 5 * 2.0**-23).all()


@pytest.mark.parametrize("quant", ["fp8", "mxfp8"])
@pytest.mark.parametrize("counts,N,K", [([3, 0, 17, 40], 256, 2048), ([(7 * e) % 23 for e in range(38)] + [140, 300], 1024, 4096)],
                         ids=["split", "turned"])
def test_place_of_a_row_among_its_experts(counts, N, K, quant):
    """Where K is split, and where tiles begin at blocks of their own: an
    expert's rows the other way round have the same bits, and so have they beside
    other experts' other rows."""
    d = make(counts, N, K, 51, quant, extra=0)
    n = sum(counts)
    swiglu = lambda: grouped_swiglu(d["x"], d["x_scale"], d["w"], d["w_scale"], d["offsets"], limit=LIMIT, rows=d["rows"])  # noqa: E731
    y, (h, s) = call_gemm(d), swiglu()
    ends = d["offsets"].tolist()
    d["rows"] = torch.cat([torch.arange(lo, hi).flip(0) for lo, hi in zip(ends, ends[1:])]).int().to(DEV)
    at = d["rows"].long()
    y2, (h2, s2) = call_gemm(d), swiglu()
    assert torch.equal(y2, y[at]) and torch.equal(h2, h[at]) and torch.equal(s2, s[at])
    last = ends[-2]
    d["x"][:last] = d["x"][:last].flip(1)
    y3, (h3, s3) = call_gemm(d), swiglu()
    assert torch.equal(y3[last:n], y2[last:n]) and torch.equal(h3[last:n], h2[last:n]) and torch.equal(s3[last:n], s2[last:n])
    assert not torch.equal(y3[:last], y2[:last])


def test_a_share_of_the_experts_within_the_bound():
    """K a multiple of 4096: an expert's rows in a call for a share of the
    experts may differ in their last FP32 bits, and stay within the bound."""
    counts = [(7 * e) % 23 for e in range(60)]
    d = make(counts, 1024, 4096, 52, extra=0)
    check_gemm_sums(d)
    lo, hi = 20, 60
    at = int(d["offsets"][lo])
    part = dict(d, w=d["w"][lo:hi].contiguous(), w_scale=d["w_scale"][lo:hi].contiguous(), x=d["x"][at:].contiguous(),
                x_scale=d["x_scale"][at:].contiguous(), offsets=d["offsets"][lo:] - at)
    check_gemm_sums(part)
    check_swiglu(part)


@pytest.mark.parametrize("quant", ["fp8", "mxfp8"])
@pytest.mark.parametrize("counts,N,K", [([3, 0, 17, 140], 384, 2048), ([(7 * e) % 23 for e in range(38)] + [140, 300], 1024, 4096),
                                        ([40, 100, 170, 230], 384, 1408)], ids=["split", "turned", "heights"])
def test_exact_integers_of_a_long_k(counts, N, K, quant):
    """Integers up to 7 and scales of one: sums below 4096 * 49 < 2^18, exact in
    FP32 in any order, so that one product too many or too few shows."""
    d = make(counts, N, K, 53, quant, gather=True)
    gen = torch.Generator(device=DEV).manual_seed(54)
    d["x"] = torch.randint(-7, 8, d["x"].shape, generator=gen, device=DEV).float().to(F8)
    d["w"] = torch.randint(-7, 8, d["w"].shape, generator=gen, device=DEV).float().to(F8)
    d["w_scale"].fill_(1.0)
    d["x_scale"].fill_(1.0 if quant == "fp8" else 127)
    want = exact(d)[0].float().to(torch.bfloat16)
    assert torch.equal(call_gemm(d)[: sum(counts)], want)
    # no product of eight such codes is 2^14 below another: the FP8 instruction is exact too
    assert torch.equal(fp8_sums(d)[: sum(counts)], want)


@pytest.mark.parametrize("quant", ["fp8", "mxfp8"])
@pytest.mark.parametrize("counts,N,K", [([70, 3], 1024, 640), ([150, 0, 300], 512, 7168), ([(7 * e) % 23 for e in range(38)] + [140, 300], 1024, 4096)],
                         ids=["short", "split", "turned"])
def test_swiglu_sums_in_fp32(counts, N, K, quant):
    """The hidden's scales on average. up and gate are off by 2^-21 of their
    root mean square (see check_gemm_sums) and lie above it at a block's maximum;
    2.1 * 2^-21 and the activation's 5 * 2^-23 are below 2^-19 of the scale."""
    d = make(counts, N, K, 55, quant, gather=True)
    if quant == "mxfp8":
        d["x_scale"].fill_(120)
    _, s = check_swiglu(d)
    g, _ = exact(d)
    n, I = g.shape[0], g.shape[1] // 2
    act = g[:, I:].clamp_max(LIMIT) * torch.sigmoid(g[:, I:].clamp_max(LIMIT)) * g[:, :I].clamp(-LIMIT, LIMIT)
    ws = act.abs().view(n, I // 128, 128).amax(-1) / 448.0
    assert (s[:n].double() / ws - 1.0).square().mean().sqrt() <= 2.0**-19


@pytest.mark.parametrize("split", [False, True])
def test_swiglu_without_a_limit(split):
    """limit = infinity: ordinary values as with a limit above them, and gates up
    to the largest value give no NaN."""
    K = 2048 if split else 256
    d = make([5, 40], 256, K, 56, extra=0)
    call = lambda limit: grouped_swiglu(d["x"], d["x_scale"], d["w"], d["w_scale"], d["offsets"], limit=limit)  # noqa: E731
    (h, s), (h2, s2) = call(float("inf")), call(1e30)
    assert torch.equal(h, h2) and torch.equal(s, s2)
    one = torch.zeros(45, K, device=DEV)
    one[:, 3], one[:, 130] = 1.0, 1.0
    d["x"], d["w"] = one.to(F8), torch.zeros_like(d["w"].float()).to(F8)
    d["w"][:, 9, 130], d["w"][:, 128 + 9, 3] = 1.0, 1.0  # up of the second block's scale, gate of the first's
    d["x_scale"].fill_(2.0**-60)
    gate = torch.linspace(1e38, 3.4e38, 45, device=DEV)
    gate[0] = 50.0
    d["x_scale"][:, 0] = gate
    d["w_scale"].fill_(1.0)
    h, s = call(float("inf"))
    act = gate.double().clamp_max(2.0**127) * 2.0**-60
    assert ((s[:, 0].double() * 448.0 / act.clamp_min(1e-10) - 1.0).abs() < 2.0**-20).all()
    assert (h.view(F8)[1:, 9].float() == 448.0).all() and not h[1:, :9].any() and not h[1:, 10:].any()
