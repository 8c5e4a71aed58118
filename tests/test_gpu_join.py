"""moe_join_rmsnorm_quant on the GPU against oracle/block.py.

The sums and the statistics are FP64 on both sides and every other step is one
binary32 operation, so residual, rows, codes and scales have to be bit-equal,
but for values next to a rounding border: an rstd (FP64 sums of at most 16,384
terms in different orders differ by less than 2^-38 of their magnitude: one row
in 2^13 at most), a sum of weighted rows (the order of its terms is the same on
both sides but NumPy's: within 2^-47, one in 2^22) and the sum that gives the
residual's row (rounded once on the GPU, by way of float64 in NumPy: one in
2^28). The inputs are seeded, so a pass stays a pass."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from fp8_block_scaled_moe_amd import add_rmsnorm_quant, join_rmsnorm_quant
from oracle import block as ref
from oracle.codecs import bf16_round
from oracle.rows import quantize_rows

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-5
TENSORS = ("residual", "delta", "gamma", "y", "post_gamma")


def bf16(v):
    return torch.from_numpy(np.asarray(v, np.float32)).to(torch.bfloat16).to(DEV)


def host(t):
    return t.cpu().numpy() if t.dtype in (torch.uint8, torch.int32) else t.float().cpu().numpy().astype(np.float64)


def make(T, D, k, seed, gate=None, post=True, spread=True, gate_dtype="fp32"):
    rng = np.random.default_rng(seed)
    size = 2.0 ** rng.integers(-20, 20, size=(T, 1)) if spread else 1.0
    d = {"residual": bf16_round(rng.standard_normal((T, D)) * (size if not post else 1.0)), "delta": bf16_round(rng.standard_normal((T, D)) * size),
         "gamma": bf16_round(rng.uniform(0.5, 1.5, D)), "y": None, "pos": None, "weights": None, "gate": None,
         "post_gamma": bf16_round(rng.uniform(0.5, 1.5, D)) if post else None}
    if k:
        R = T * k + 3
        d["y"] = bf16_round(rng.standard_normal((R, D)))
        d["pos"] = rng.permutation(R)[: T * k].reshape(T, k).astype(np.int32)
        d["weights"] = rng.uniform(0.0, 1.0, (T, k)).astype(np.float32)
    if gate:
        g = rng.uniform(-1.0, 2.0, {"row": (T, 1), "column": (1, D), "full": (T, D)}[gate]).astype(np.float32)
        d["gate"] = g if gate == "row" and gate_dtype == "fp32" else bf16_round(g).astype(np.float32)
        d["gate_bf16"] = not (gate == "row" and gate_dtype == "fp32")
    return d


def device(d):
    t = {n: None if d[n] is None else bf16(d[n]) for n in TENSORS}
    for n in ("pos", "weights", "gate"):
        t[n] = None if d[n] is None else torch.from_numpy(d[n]).to(DEV)
    if d["gate"] is not None and d["gate_bf16"]:
        t["gate"] = t["gate"].to(torch.bfloat16)
    return t


def check(d, quant, residual_scale=1.0, gamma_offset=0.0, post_eps=None, **kw):
    t = device(d)
    got = join_rmsnorm_quant(eps=EPS, quant=quant, residual_scale=residual_scale, gamma_offset=gamma_offset, post_eps=post_eps, **t, **kw)
    torch.cuda.synchronize()
    h, v = ref.join_rows(d["residual"], d["delta"], d["y"], d["pos"], d["weights"], gamma=d["gamma"], eps=EPS, post_gamma=d["post_gamma"],
                         post_eps=post_eps, gate=d["gate"], residual_scale=residual_scale, gamma_offset=gamma_offset)
    res, out, q, s = got
    assert np.array_equal(host(res), bf16_round(h))
    assert np.array_equal(host(out), bf16_round(v))
    if quant is None:
        assert q is None and s is None
    else:
        wq, ws = quantize_rows(v, quant)
        assert np.array_equal(host(s), ws), f"{np.sum(host(s) != ws)} scales differ"
        assert np.array_equal(host(q), wq), f"{np.sum(host(q) != wq)} codes differ"
    return got


# every width at which another number of chunks or of threads begins, the narrowest and the widest, odd ones
WIDTHS = [128, 256, 1408, 2048, 2048 + 128, 4096, 4096 + 128, 7168, 8192, 8192 + 128, 16384 - 128, 16384]


@pytest.mark.parametrize("quant", ["fp8", "fp8_p2", "mxfp8"])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(D, quant):
    check(make(3, D, 0, D, gate="row"), quant)
    check(make(2, D, 3, D + 1, gate="full", spread=False), quant, residual_scale=0.5)


@pytest.mark.parametrize("D,quant", [(8, None), (24, None), (2056, None), (32, "mxfp8"), (96, "mxfp8"), (4096 + 96, "mxfp8"),
                                     (8192 + 32, "mxfp8"), (16376, None)])
def test_narrow_units(D, quant):
    check(make(5, D, 0, D, gate="column"), quant, gamma_offset=1.0)


@pytest.mark.parametrize("T", [1, 2, 255, 257, 1000])
def test_tokens(T):
    check(make(T, 256, 2, T, gate="row"), "fp8")


@pytest.mark.parametrize("D", [640, 2176, 4224, 8320])
def test_more_tokens_than_the_wide_form_takes(D):
    """Plain rows beyond 512 tokens have workgroups of one, two and four chunks a lane."""
    check(make(600, D, 0, D, gate="full"), "mxfp8", residual_scale=-2.0)


@pytest.mark.parametrize("k", [1, 2, 7, 8, 9, 16, 32])
@pytest.mark.parametrize("D", [384, 7168, 16384])
def test_routed_rows(D, k):
    check(make(4, D, k, 100 * k + D, gate="row", spread=False), "fp8")


@pytest.mark.parametrize("gate", [None, "row", "column", "full"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("k", [0, 3])
def test_gates(gate, post, k):
    for dtype in ("fp32", "bf16"):
        check(make(6, 640, k, 5, gate=gate, post=post, spread=False, gate_dtype=dtype), "fp8", residual_scale=0.25, gamma_offset=0.5, post_eps=0.125)


def test_a_gate_for_one_token_and_flat_gates():
    d = make(1, 256, 0, 1, gate="full")
    check(d, "fp8")
    for gate in ("row", "column"):
        d = make(5, 256, 0, 2, gate=gate)
        want = check(d, "fp8")
        t = device(d)
        t["gate"] = t["gate"].flatten()
        for a, b in zip(want, join_rmsnorm_quant(eps=EPS, **t)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("absent", [("residual",), ("delta",), ("residual", "delta"), ("gamma",), ("post_gamma",), ("gamma", "post_gamma"),
                                    ("residual", "gamma", "post_gamma"), ("y", "pos", "weights")])
def test_absent_inputs(absent):
    d = make(4, 640, 3, 7, gate="row", spread=False)
    for n in absent:
        d[n] = None
    check(d, "mxfp8")


def test_as_the_norm():
    """Without the second norm, gate and scale: add_rmsnorm_quant of the same rows, bit by bit."""
    for T, D, k in ((3, 7168, 0), (700, 2176, 0), (5, 640, 4)):
        t = device(make(T, D, k, 9, post=False, spread=False))
        del t["gate"], t["post_gamma"]
        if k:  # the sum begins with the residual there
            t["residual"] = torch.zeros_like(t["residual"])
        for a, b in zip(add_rmsnorm_quant(eps=EPS, **t), join_rmsnorm_quant(eps=EPS, **t)):
            assert torch.equal(a, b)


def test_positions_outside_add_nothing():
    d = make(6, 256, 4, 8, spread=False)
    d["pos"][0] = -1
    d["pos"][1, 2] = d["y"].shape[0]
    d["pos"][2] = 2**31 - 1
    d["pos"][3, 0] = -(2**31)
    check(d, "fp8")


def test_zero_rows():
    """A block's output of zeros stays zero behind its norm."""
    d = make(4, 256, 0, 3, gate="row")
    d["delta"][:2] = 0.0
    d["residual"][0] = 0.0
    res, out, q, s = check(d, "fp8")
    assert (res[0] == 0).all() and (out[0] == 0).all() and torch.equal(res[1], bf16(d["residual"][1]))
    check(d, "mxfp8")


def test_bad_values_stay_in_their_row():
    d = make(6, 256, 2, 4, gate="row", spread=False)
    want = join_rmsnorm_quant(eps=EPS, **device(d))
    for what, value in (("delta", np.nan), ("delta", np.inf), ("residual", np.nan), ("residual", -np.inf)):
        e = {n: None if v is None else (v.copy() if isinstance(v, np.ndarray) else v) for n, v in d.items()}
        e[what][2, 17] = value
        got = join_rmsnorm_quant(eps=EPS, **device(e))
        keep = torch.tensor([0, 1, 3, 4, 5], device=DEV)
        for a, b in zip(want, got):
            assert torch.equal(a[keep], b[keep])
        assert not got[0][2, 17].isfinite()
    e = {n: None if v is None else (v.copy() if isinstance(v, np.ndarray) else v) for n, v in d.items()}
    e["gate"][3] = np.nan
    got = join_rmsnorm_quant(eps=EPS, **device(e))
    assert got[0][3].isnan().all() and torch.equal(got[0][4:], want[0][4:])


def test_outputs_wanted_and_in_place():
    d = make(9, 512, 2, 6, gate="full", spread=False)
    t = device(d)
    want = join_rmsnorm_quant(eps=EPS, **t)
    res, out, q, s = join_rmsnorm_quant(eps=EPS, want_residual=False, quant=None, **t)
    assert res is None and q is None and s is None and torch.equal(out, want[1])
    res, out, q, s = join_rmsnorm_quant(eps=EPS, want_out=False, **t)
    assert out is None and torch.equal(q, want[2]) and torch.equal(s, want[3])
    got = join_rmsnorm_quant(eps=EPS, inplace=True, **t)
    assert got[0] is t["residual"]
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_empty_batch():
    z = torch.zeros(0, 256, dtype=torch.bfloat16, device=DEV)
    g = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    res, out, q, s = join_rmsnorm_quant(z, g, delta=z, post_gamma=g)
    assert res.shape == out.shape == q.shape == (0, 256) and s.shape == (0, 2)


@pytest.mark.parametrize("T,k", [(1, 0), (600, 0), (70, 4)])
def test_captured_streams_and_again(T, k):
    t = device(make(T, 768, k, 12, gate="row", spread=False))
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for _ in range(2):
            join_rmsnorm_quant(eps=EPS, **t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = join_rmsnorm_quant(eps=EPS, **t)
    for seed in (1, 2, 3):
        t["delta"].copy_(device(make(T, 768, k, seed, gate="row", spread=False))["delta"])
        graph.replay()
        eager = join_rmsnorm_quant(eps=EPS, **t)
        torch.cuda.synchronize()
        other = join_rmsnorm_quant(eps=EPS, **t, stream=stream)
        torch.cuda.synchronize()
        for a, c, d in zip(captured, eager, other):
            assert torch.equal(a, c) and torch.equal(a, d)


def test_rows_past_32_bits():
    """Gated rows whose elements lie past 2^31: the last ones against a call of their own."""
    T, D = 150000, 14400
    z = torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
    some = device(make(4, D, 0, 3, gate="full", spread=False))
    z[-4:] = some["delta"]
    full = torch.empty_like(z)
    full[-4:] = some["gate"]
    kw = dict(post_gamma=some["post_gamma"], quant=None, eps=EPS)
    res, out, _, _ = join_rmsnorm_quant(None, some["gamma"], delta=z, gate=full, **kw)
    small = join_rmsnorm_quant(None, some["gamma"], delta=some["delta"], gate=some["gate"], **kw)
    assert T * D > 2**31 and torch.equal(res[-4:], small[0])
    # another workgroup size may round an rstd the other way: a step of BF16 at most
    assert ((out[-4:].float() - small[1].float()).abs() <= 2.0**-7 * small[1].float().abs()).all()
