"""The calls around the experts together with those of the experts, as a
serving program makes them for a layer with a dense expert beside the routed
ones and norms on both sides of the block: join (the block before) -> router
logits -> routing by groups -> grouped SwiGLU -> grouped product, dense expert
up and down -> join. Against float64 step by step, in a replayed graph, on
another stream and with two runs at once."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import synth
from fp8_block_scaled_moe_amd import dense_gemm, grouped_gemm, grouped_swiglu, join_rmsnorm_quant, route_rows_scored
from oracle import block as ref
from oracle.codecs import bf16_round
from oracle.rows import quantize_rows
from tests.helpers import bf16_step, host

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
SHAPE = synth.CONFIGS["tiny"].with_(M=1, hidden=512, inter=256, experts=24, top_k=4)
EPS = 1e-5
ROUTE = dict(top_k=4, routed_scale=2.5, scores="softmax", groups=6, top_groups=3)


class Layer:
    def __init__(self, T, seed):
        s = SHAPE
        self.inp = synth.make_inputs(s.with_(M=T), seed=seed, device=DEV)
        g = torch.Generator(device=DEV).manual_seed(seed)
        new = lambda *n, by=1.0, add=0.0: (torch.randn(*n, generator=g, device=DEV) * by + add).to(BF)  # noqa: E731
        self.residual, self.delta = new(T, s.hidden), new(T, s.hidden, by=3.0)
        self.gammas = [new(s.hidden, by=0.1, add=1.0) for _ in range(4)]
        self.router = new(s.experts, s.hidden, by=s.hidden**-0.5)
        self.gate = new(1, s.hidden, by=s.hidden**-0.5)
        self.up, self.up_bias = new(s.inter, s.hidden, by=s.hidden**-0.5), new(s.inter, by=0.1)
        self.down = new(s.hidden, s.inter, by=s.inter**-0.5)
        self.bias = torch.randn(s.experts, generator=g, device=DEV) * 0.02

    def __call__(self):
        a, b, c, d = self.gammas
        inp = self.inp
        h, x, q, qs = join_rmsnorm_quant(self.residual, b, EPS, delta=self.delta, post_gamma=a, residual_scale=0.5)
        logits = dense_gemm(x, self.router, out_dtype=torch.float32)
        r = route_rows_scored(logits, self.bias, **ROUTE)
        hid, hs = grouped_swiglu(q, qs, inp.w13, inp.w13_scale, r.offsets, limit=SHAPE.limit, rows=r.rows)
        y = grouped_gemm(hid, hs, inp.w2, inp.w2_scale, r.offsets)
        gate = dense_gemm(x, self.gate, act="sigmoid", out_dtype=torch.float32)
        dense = dense_gemm(x, self.up, bias=self.up_bias, act="gelu_tanh")
        dense = dense_gemm(dense, self.down, residual=x)
        out = join_rmsnorm_quant(h, d, EPS, delta=dense, y=y, pos=r.pos, weights=r.weights, post_gamma=c, gate=gate)
        return dict(h=h, x=x, q=q, qs=qs, logits=logits, ids=r.ids, weights=r.weights, pos=r.pos, y=y, gate=gate, dense=dense, out=out)


def close_bf16(got, want, by=0.0):
    """Within half a step of BF16 and `by`."""
    g = host(got)
    assert (np.abs(g - want) <= bf16_step(np.maximum(np.abs(g), np.abs(want))) / 2 * (1 + 2.0**-7) + by).all()


@pytest.mark.parametrize("T", [1, 5, 90, 700])
def test_every_step_against_float64(T):
    """Each step from the GPU's own inputs to it, so that an error is met where it is made."""
    layer = Layer(T, 41)
    r = layer()
    torch.cuda.synchronize()
    a, b, c, d = (host(g) for g in layer.gammas)
    h, v = ref.join_rows(host(layer.residual), host(layer.delta), None, None, None, gamma=b, eps=EPS, post_gamma=a, residual_scale=0.5)
    assert np.array_equal(host(r["h"]), bf16_round(h)) and np.array_equal(host(r["x"]), bf16_round(v))
    q, s = quantize_rows(v, "fp8")
    assert np.array_equal(host(r["q"]), q) and np.array_equal(host(r["qs"]), s)
    x = host(r["x"])
    sums = lambda x, w: (w.shape[1] / 16 + 64) * 2.0**-23 * (np.abs(x) @ np.abs(w).T)  # noqa: E731  FP32 sums of exact products
    w = host(layer.router)
    assert (np.abs(host(r["logits"]) - x @ w.T) <= sums(x, w)).all()
    ids, weights, _ = ref.route_scored(host(r["logits"]), host(layer.bias), 4, 2.5, kind="softmax", groups=6, top_groups=3, group_best=2)
    assert np.array_equal(r["ids"].cpu().numpy(), ids)
    np.testing.assert_allclose(host(r["weights"]), weights, rtol=1e-6)
    w = host(layer.gate)
    np.testing.assert_allclose(host(r["gate"]), ref.dense(x, w, act="sigmoid")[0], atol=float(sums(x, w).max()) / 4 + 2.0**-21)
    up = ref.dense(x, host(layer.up), host(layer.up_bias), "gelu_tanh")[0]
    steps = bf16_step(np.abs(up)) / 2 + 1.13 * sums(x, host(layer.up)) + 2.0**-19  # of the hidden, as the down product meets them
    down = host(layer.down)
    close_bf16(r["dense"], ref.dense(bf16_round(up), down, residual=x)[0], (2 * steps) @ np.abs(down).T + sums(up, down))
    h2, v2 = ref.join_rows(host(r["h"]), host(r["dense"]), host(r["y"]), r["pos"].cpu().numpy(), host(r["weights"]), gamma=d, eps=EPS, post_gamma=c,
                           gate=host(r["gate"]))
    assert np.array_equal(host(r["out"][0]), bf16_round(h2)) and np.array_equal(host(r["out"][1]), bf16_round(v2))


def flat(r):
    return [t for v in r.values() for t in (v if isinstance(v, tuple) else (v,))]


@pytest.mark.parametrize("T", [1, 90, 700])
def test_replayed_graph(T):
    layer = Layer(T, 42)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for _ in range(2):
            layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer()
    for seed in (1, 2, 3):
        other = Layer(T, seed)
        layer.residual.copy_(other.residual)
        layer.delta.copy_(other.delta)
        graph.replay()
        eager = layer()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(flat(captured), flat(eager)))


def test_two_runs_at_once():
    one, two = Layer(90, 43), Layer(300, 44)
    want = flat(one()), flat(two())
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            got.append((want[0], flat(one())))
        with torch.cuda.stream(s2):
            got.append((want[1], flat(two())))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, g in got for a, b in zip(w, g))


def test_padded_batch():
    """Tokens of a padded batch have the rows of the batch without padding: every step but the products'
    last FP32 bits is a row's own, so ids agree and the rows lie within a step of BF16."""
    layer = Layer(64, 45)
    full = layer()
    for n in ("residual", "delta"):
        setattr(layer, n, torch.cat([getattr(layer, n), torch.zeros(36, SHAPE.hidden, dtype=BF, device=DEV)]))
    padded = layer()
    assert torch.equal(padded["ids"][:64], full["ids"]) and torch.equal(padded["h"][:64], full["h"])
    a, b = host(padded["out"][0][:64]), host(full["out"][0])
    assert (np.abs(a - b) <= 2 * bf16_step(np.maximum(np.abs(a), np.abs(b))) + 2.0**-8).all()
    assert all(t.isfinite().all() for t in flat(padded) if t.is_floating_point())
