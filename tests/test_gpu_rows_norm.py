"""moe_add_rmsnorm_quant on the GPU against oracle/rows.py.

The sum and the statistics are taken in FP64 on both sides and every later
step is one binary32 operation, so residual, rows, codes and scales have to be
bit-equal: two FP64 sums of at most 16,384 terms in different orders differ by
less than 16,384 * 2^-53 < 2^-38 of their magnitude, so the binary32 rounding of rstd
(and of a sum of weighted rows) differs only where the exact value lies within
2^-38 of a rounding border, one value in 2^13 times fewer than could be met
here for rstd (a few hundred rows), and for the weighted sums (k <= 32 terms:
within 2^-47) one in 2^22. The inputs are seeded, so a pass stays a pass."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from fp8_block_scaled_moe_amd import add_rmsnorm_quant
from oracle import rows as ref
from oracle.codecs import bf16_round

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-5


def bf16(v):
    return torch.from_numpy(np.asarray(v, np.float32)).to(torch.bfloat16).to(DEV)


def host(t):
    return t.cpu().numpy() if t.dtype in (torch.uint8, torch.int32) else t.float().cpu().numpy().astype(np.float64)


def make(T, D, k, seed, spread=True):
    rng = np.random.default_rng(seed)
    size = 2.0 ** rng.integers(-20, 20, size=(T, 1)) if spread else 1.0
    d = {"residual": bf16_round(rng.standard_normal((T, D)) * size), "delta": bf16_round(rng.standard_normal((T, D)) * size),
         "gamma": bf16_round(rng.uniform(0.5, 1.5, D)), "y": None, "pos": None, "weights": None}
    if k:
        R = T * k + 3
        d["y"] = bf16_round(rng.standard_normal((R, D)))
        d["pos"] = rng.permutation(R)[: T * k].reshape(T, k).astype(np.int32)
        d["weights"] = rng.uniform(0.0, 1.0, (T, k)).astype(np.float32)
    return d


def device(d):
    t = {n: None if d[n] is None else bf16(d[n]) for n in ("residual", "delta", "gamma", "y")}
    t["pos"] = None if d["pos"] is None else torch.from_numpy(d["pos"]).to(DEV)
    t["weights"] = None if d["weights"] is None else torch.from_numpy(d["weights"]).to(DEV)
    return t


def check(d, quant, **kw):
    got = add_rmsnorm_quant(eps=EPS, quant=quant, **device(d), **kw)
    torch.cuda.synchronize()
    h = ref.sum_rows(d["residual"], d["delta"], d["y"], d["pos"], d["weights"])
    v = h if d["gamma"] is None else ref.norm_rows(h, d["gamma"], EPS)
    res, out, q, s = got
    assert np.array_equal(host(res), bf16_round(h))
    assert np.array_equal(host(out), bf16_round(v))
    if quant is None:
        assert q is None and s is None
    else:
        wq, ws = ref.quantize_rows(v, quant)
        assert np.array_equal(host(s), ws), f"{np.sum(host(s) != ws)} scales differ"
        assert np.array_equal(host(q), wq), f"{np.sum(host(q) != wq)} codes differ"
    return got


# every width at which another number of chunks or of threads begins, the narrowest and the widest, odd ones
WIDTHS = [128, 256, 1408, 2048, 2048 + 128, 4096, 4096 + 128, 7168, 8192, 8192 + 128, 16384 - 128, 16384]


@pytest.mark.parametrize("quant", ["fp8", "fp8_p2", "mxfp8"])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(D, quant):
    check(make(3, D, 0, D), quant)


@pytest.mark.parametrize("D,quant", [(8, None), (24, None), (2056, None), (32, "mxfp8"), (96, "mxfp8"), (4096 + 96, "mxfp8"),
                                     (8192 + 32, "mxfp8"), (16376, None)])
def test_narrow_units(D, quant):
    check(make(5, D, 0, D), quant)


@pytest.mark.parametrize("T", [1, 2, 255, 257, 1000])
def test_tokens(T):
    check(make(T, 256, 2, T), "fp8")


@pytest.mark.parametrize("k", [1, 2, 7, 8, 9, 16, 32])
@pytest.mark.parametrize("D", [384, 7168, 16384])
def test_routed_rows(D, k):
    check(make(4, D, k, 100 * k + D, spread=False), "fp8")


@pytest.mark.parametrize("absent", [("residual",), ("delta",), ("residual", "delta"), ("gamma",), ("residual", "delta", "gamma")])
def test_absent_inputs(absent):
    d = make(4, 640, 3, 7)
    for n in absent:
        d[n] = None
    check(d, "mxfp8")


def test_positions_outside_add_nothing():
    d = make(6, 256, 4, 8, spread=False)
    d["pos"][0] = -1
    d["pos"][1, 2] = d["y"].shape[0]
    d["pos"][2, 0] = -(2**31)
    d["pos"][3] = 2**31 - 1
    d["residual"][3] = d["delta"][3] = 0.0  # nothing is left of this token
    got = check(d, "fp8")
    assert not host(got[1])[3].any() and not host(got[2])[3].any()


def test_same_row_for_several_picks():
    d = make(3, 256, 4, 9, spread=False)
    d["pos"][:] = 5
    check(d, "fp8")


@pytest.mark.parametrize("quant", ["fp8", "fp8_p2", "mxfp8"])
def test_zero_and_tiny_rows(quant):
    d = make(5, 256, 0, 10, spread=False)
    d["residual"][0] = d["delta"][0] = 0.0
    d["residual"][1, :128] = d["delta"][1, :128] = 0.0
    d["delta"][2:] = 0.0
    d["residual"][2] = 2.0**-126          # the smallest normal
    d["residual"][3] = 2.0**-133          # the smallest BF16 subnormal
    d["residual"][4] = 2.0**100
    check(d, quant)
    d["gamma"] = None
    check(d, quant)


def test_in_place_and_no_outputs():
    d = make(4, 512, 0, 11)
    t = device(d)
    want = check(d, "fp8")
    res, out, q, s = add_rmsnorm_quant(eps=EPS, inplace=True, want_out=False, **t)
    assert res.data_ptr() == t["residual"].data_ptr() and out is None
    for a, b in ((res, want[0]), (q, want[2]), (s, want[3])):
        assert torch.equal(a, b)
    res, out, q, s = add_rmsnorm_quant(eps=EPS, want_residual=False, quant=None, **device(d))
    assert res is None and q is None and torch.equal(out, want[1])


def test_empty():
    e = torch.empty((0, 256), dtype=torch.bfloat16, device=DEV)
    res, out, q, s = add_rmsnorm_quant(e, torch.ones(256, dtype=torch.bfloat16, device=DEV))
    assert res.shape == out.shape == q.shape == (0, 256) and s.shape == (0, 2)


def test_most_tokens():
    """The longest call there is, in the narrowest rows."""
    x = torch.randn(1048576, 8, generator=torch.Generator(device=DEV).manual_seed(42), device=DEV).to(torch.bfloat16)
    res, out, _, _ = add_rmsnorm_quant(x, None, EPS, quant=None)
    assert torch.equal(res, x) and torch.equal(out, x)


@pytest.mark.parametrize("quant", ["fp8", "mxfp8"])
def test_nan_and_infinity(quant):
    """A NaN or infinite value spoils its row (through rstd) and no other;
    without normalisation a NaN code stands in its place alone, and its block's
    scale is that of the others."""
    d = make(4, 512, 0, 12, spread=False)
    d["delta"][:] = 0.0
    clean = check(d, quant)
    d["residual"][1, 200] = np.nan
    d["residual"][2, 300] = np.inf
    t = device(d)
    res, out, q, s = add_rmsnorm_quant(eps=EPS, quant=quant, **t)
    for got, want in zip((res, out, q, s), clean):
        assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])
    assert torch.isnan(out[1]).all() and torch.isnan(res[1, 200]) and torch.isnan(out[2, 300])
    assert ((q[1] & 0x7F) == 0x7F).all()
    assert torch.isinf(res[2, 300]) and not out[2, :300].any()
    t["gamma"] = None
    _, out, q, s = add_rmsnorm_quant(eps=EPS, quant=quant, **t)
    assert (int(q[1, 200]) & 0x7F) == 0x7F
    v = d["residual"].copy()
    v[1, 200] = 0.0
    v[2, 300] = 0.0
    wq, ws = ref.quantize_rows(v, quant)
    keep = np.ones_like(wq, bool)
    keep[1, 200] = False
    block = 128 if quant == "fp8" else 32
    keep[2, 300 // block * block : (300 // block + 1) * block] = False  # the block of the infinity has an infinite scale
    assert np.array_equal(host(q)[keep], wq[keep])
    sk = np.ones_like(ws, bool)
    sk[2, 300 // block] = False
    assert np.array_equal(host(s)[sk], ws[sk])


def test_same_bits_alone_and_in_a_batch():
    d = make(64, 1024, 3, 13)
    whole = add_rmsnorm_quant(eps=EPS, **device(d))
    one = {n: (v[40:41] if n in ("residual", "delta", "pos", "weights") else v) for n, v in d.items()}
    for a, b in zip(add_rmsnorm_quant(eps=EPS, **device(one)), whole):
        assert torch.equal(a[0], b[40])


# plain rows of more than 512 tokens have narrower workgroups, up to four chunks a lane
@pytest.mark.parametrize("quant", ["fp8", "fp8_p2", "mxfp8"])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths_of_many_tokens(D, quant):
    check(make(513, D, 0, D + 1), quant)


@pytest.mark.parametrize("D,quant", [(8, None), (2056, None), (4104, None), (4096 + 96, "mxfp8"), (8192 + 32, "mxfp8"), (16376, None)])
def test_narrow_units_of_many_tokens(D, quant):
    check(make(600, D, 0, D + 2), quant)


@pytest.mark.parametrize("D", [2176, 7168])
@pytest.mark.parametrize("T", [512, 513, 4096])
def test_tokens_around_the_narrow_workgroups(T, D):
    check(make(T, D, 0, T + D), "fp8")


def test_order_of_a_cancelling_sum():
    """Terms 2^54 and more above what is left of them: residual, addend, then the
    picks as they come, each addition rounded to FP64 (the products of a weight and
    a value are exact there)."""
    d = make(40, 256, 4, 14, spread=False)
    rng = np.random.default_rng(15)
    big = 2.0 ** rng.integers(54, 70, size=(40, 256))
    y = d["y"].copy()
    for a, b in ((0, 2), (1, 3), (3, 0)):
        at = slice(0, 20) if (a, b) == (0, 2) else slice(20, 30) if (a, b) == (1, 3) else slice(30, 40)
        y[d["pos"][at, a]], y[d["pos"][at, b]] = big[at], -big[at]
        d["weights"][at, b] = d["weights"][at, a]
    d["y"] = y
    h = d["residual"].astype(np.float64) + d["delta"]
    for j in range(4):
        h = h + d["weights"][:, j : j + 1].astype(np.float64) * y[d["pos"][:, j]]
    res, _, _, _ = add_rmsnorm_quant(eps=EPS, quant=None, want_out=False, **device(d))
    assert np.array_equal(host(res), bf16_round(h.astype(np.float32).astype(np.float64)))
    back = d["residual"].astype(np.float64) + d["delta"]
    for j in range(3, -1, -1):
        back = back + d["weights"][:, j : j + 1].astype(np.float64) * y[d["pos"][:, j]]
    assert (back != h).any()  # another order is another sum
