"""The calls over any number of tokens together, as a serving program makes
them: norm -> routing -> grouped SwiGLU (gathering token rows) -> grouped
product -> norm with the routed rows weighted and added. Against the layer's
oracle, against moe_decode_run, in a replayed graph, on another stream, and
with two runs at once."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import synth
from fp8_block_scaled_moe_amd import MoeDecode, add_rmsnorm_quant, grouped_gemm, grouped_swiglu, route_rows
from tests.helpers import ROW_RTOL, WEIGHT_RTOL, bf16_step, host, oracle_layer

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
SHAPE = synth.CONFIGS["tiny"].with_(M=90, hidden=512, inter=256, experts=24, top_k=4)


def quantise(x, quant="fp8"):
    _, _, q, s = add_rmsnorm_quant(x, None, quant=quant, want_out=False, want_residual=False)
    return q, s


def layer(inp, quant="fp8"):
    """(combined BF16, y, routed): the routed step of x without a residual."""
    s = inp.shape
    q, xs = quantise(inp.x, quant)
    r = route_rows(inp.logits, inp.bias, top_k=s.top_k, routed_scale=s.routed_scale)
    h, hs = grouped_swiglu(q, xs, inp.w13, inp.w13_scale, r.offsets, limit=s.limit, rows=r.rows)
    y = grouped_gemm(h, hs, inp.w2, inp.w2_scale, r.offsets)
    combined, _, _, _ = add_rmsnorm_quant(None, None, y=y, pos=r.pos, weights=r.weights, quant=None, want_out=False)
    return combined, y, r


def check_rows(got, ref, more=0.0, what="rows"):
    """Within 2e-2 of the row's RMS, the layer's bar, beyond one BF16 step:
    two values that differ by less than a step before their rounding can round
    to neighbouring BF16 numbers, which lie a step apart (up to 2^-7 of the
    value: 0.031 of the RMS for an element of four times the RMS). `more`: what
    the roundings of the terms of a sum may add."""
    rms = np.sqrt((ref * ref).mean(axis=1, keepdims=True))
    allowed = ROW_RTOL * rms + bf16_step(np.maximum(np.abs(got), np.abs(ref))) + more
    bad = np.abs(got - ref) > allowed
    assert not bad.any(), f"{what}: {int(bad.sum())} values outside"


def check_layer(slots, weights, combined, ref_slots, ref_combined, what=""):
    """Slots, and their weighted sums: a sum moves by its terms' steps too."""
    s = host(slots)
    check_rows(s, ref_slots, what="slots" + what)
    w = host(weights)
    steps = bf16_step(np.maximum(np.abs(s), np.abs(ref_slots))).reshape(w.shape + (-1,))
    check_rows(host(combined), ref_combined, (w[..., None] * steps).sum(axis=1), "combined" + what)


@pytest.mark.parametrize("M", [1, 3, 90, 256])
def test_matches_the_oracle_and_the_decode_call(M):
    inp = synth.make_inputs(SHAPE.with_(M=M), seed=31, device=DEV)
    combined, y, r = layer(inp)
    ref = oracle_layer(inp)
    assert np.array_equal(r.ids.cpu().numpy(), ref["ids"])
    np.testing.assert_allclose(host(r.weights), ref["weights"], rtol=WEIGHT_RTOL, atol=0)
    slots = y[r.pos.flatten().long()]
    check_layer(slots, r.weights, combined, ref["slots"], ref["combined"])
    moe = MoeDecode(inp.w13, inp.w13_scale, inp.w2, inp.w2_scale, top_k=SHAPE.top_k, limit=SHAPE.limit,
                    routed_scale=SHAPE.routed_scale, max_tokens=M, logits_dtype=inp.logits.dtype)
    slots2, ids2, weights2, combined2 = moe(inp.x, inp.logits, inp.bias)
    assert torch.equal(ids2, r.ids) and torch.equal(weights2, r.weights)
    check_layer(slots, r.weights, combined, host(slots2), host(combined2), " against the decode call")


def test_x_codes_are_the_decode_calls():
    inp = synth.make_inputs(SHAPE, seed=32, device=DEV)
    moe = MoeDecode(inp.w13, inp.w13_scale, inp.w2, inp.w2_scale, top_k=SHAPE.top_k, limit=SHAPE.limit,
                    routed_scale=SHAPE.routed_scale, max_tokens=SHAPE.M, logits_dtype=inp.logits.dtype)
    moe(inp.x, inp.logits, inp.bias)
    q, s = quantise(inp.x)
    assert torch.equal(moe.stage("x_q", torch.empty_like(q)), q)
    assert torch.equal(moe.stage("x_s", torch.empty_like(s)), s)


def test_prompt_of_many_tokens():
    """More tokens than one decode call takes: every token against the oracle."""
    inp = synth.make_inputs(SHAPE.with_(M=1500), seed=33, device=DEV)
    combined, y, r = layer(inp)
    ref = oracle_layer(inp)
    assert np.array_equal(r.ids.cpu().numpy(), ref["ids"])
    check_layer(y[r.pos.flatten().long()], r.weights, combined, ref["slots"], ref["combined"])


def test_local_shares_add_up():
    """Two GPUs' shares of the experts, one after the other: the same slots,
    bit for bit (an expert's products do not depend on the others), and
    partial sums that add up to the whole: each part is rounded to BF16 and the
    whole once, half a step each."""
    inp = synth.make_inputs(SHAPE, seed=34, device=DEV)
    whole, y0, r0 = layer(inp)
    q, xs = quantise(inp.x)
    parts = []
    for lb, lc in ((0, 10), (10, 14)):
        r = route_rows(inp.logits, inp.bias, top_k=SHAPE.top_k, routed_scale=SHAPE.routed_scale, local_begin=lb, local_experts=lc)
        sl = slice(lb, lb + lc)
        h, hs = grouped_swiglu(q, xs, inp.w13[sl].contiguous(), inp.w13_scale[sl].contiguous(), r.offsets, limit=SHAPE.limit,
                               rows=r.rows)
        y = grouped_gemm(h, hs, inp.w2[sl].contiguous(), inp.w2_scale[sl].contiguous(), r.offsets)
        mine = (r.pos >= 0).flatten()
        assert torch.equal(y[r.pos.flatten()[mine].long()], y0[r0.pos.flatten()[mine].long()])
        parts.append(host(add_rmsnorm_quant(None, None, y=y, pos=r.pos, weights=r.weights, quant=None, want_out=False)[0]))
    half = sum(bf16_step(v) / 2 for v in parts + [host(whole)])
    assert (np.abs(parts[0] + parts[1] - host(whole)) <= half * (1 + 2.0**-10)).all()


class Block:
    """Two layers' worth of calls on fixed input buffers: residual add and
    norm, the experts, and the next norm, which adds their rows."""

    def __init__(self, seed, M=SHAPE.M, quant="fp8"):
        self.inp = synth.make_inputs(SHAPE.with_(M=M), seed=seed, device=DEV)
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.residual = torch.randn(M, SHAPE.hidden, generator=gen, device=DEV).to(torch.bfloat16)
        self.delta = torch.randn(M, SHAPE.hidden, generator=gen, device=DEV).to(torch.bfloat16)
        self.g1 = (1 + 0.1 * torch.randn(SHAPE.hidden, generator=gen, device=DEV)).to(torch.bfloat16)
        self.g2 = (1 + 0.1 * torch.randn(SHAPE.hidden, generator=gen, device=DEV)).to(torch.bfloat16)
        self.quant = quant

    def run(self, stream=None):
        s, kw = self.inp.shape, dict(stream=stream)
        res, _, q, xs = add_rmsnorm_quant(self.residual, self.g1, delta=self.delta, quant=self.quant, want_out=False, **kw)
        r = route_rows(self.inp.logits, self.inp.bias, top_k=s.top_k, routed_scale=s.routed_scale, **kw)
        h, hs = grouped_swiglu(q, xs, self.inp.w13, self.inp.w13_scale, r.offsets, limit=s.limit, rows=r.rows, **kw)
        y = grouped_gemm(h, hs, self.inp.w2, self.inp.w2_scale, r.offsets, **kw)
        return add_rmsnorm_quant(res, self.g2, y=y, pos=r.pos, weights=r.weights, quant="fp8", **kw) + (r.ids,)


def bits(ts):
    return [t.clone() for t in ts]


def same(a, b):
    return all(torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x, y.view(torch.int16) if y.dtype == torch.bfloat16 else y)
               for x, y in zip(a, b))


@pytest.mark.parametrize("M,quant", [(1, "fp8"), (50, "mxfp8"), (200, "fp8")])
def test_graph_replay_equals_eager(M, quant):
    blk = Block(41, M, quant)
    blk.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = blk.run()
    gen = torch.Generator(device=DEV).manual_seed(42)
    seen = set()
    for _ in range(4):
        blk.inp.logits.copy_(torch.randn(blk.inp.logits.shape, generator=gen, device=DEV) * 2)
        blk.residual.copy_(torch.randn(blk.residual.shape, generator=gen, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        replayed = bits(out)
        eager = blk.run()
        torch.cuda.synchronize()
        assert same(replayed, eager)
        seen.add(tuple(eager[-1].flatten().tolist()))
    assert len(seen) == 4


def test_two_graphs_replayed_at_once():
    """Two captured runs of their own inputs, replayed on two streams."""
    a, b = Block(43, 200), Block(44, 130)
    want = bits(a.run()), bits(b.run())
    torch.cuda.synchronize()
    graphs = []
    for blk in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = blk.run()
        graphs.append((g, out))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        for s, (g, _) in zip((s1, s2), graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert same(graphs[0][1], want[0]) and same(graphs[1][1], want[1])
        torch.zeros(1 << 20, device=DEV).add_(1)  # the program's own work in between
        torch.cuda.synchronize()


@pytest.mark.parametrize("how", ["argument", "context", "raw"])
def test_on_another_stream(how):
    blk = Block(45)
    want = bits(blk.run())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    if how == "context":
        with torch.cuda.stream(s):
            got = blk.run()
    else:
        got = blk.run(s if how == "argument" else s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    assert same(got, want)
    torch.cuda.synchronize()


def test_eager_runs_at_once_on_two_streams():
    a, b = Block(46, 250), Block(47, 250)
    want = bits(a.run()), bits(b.run())
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got = a.run(s1), b.run(s2)
        torch.cuda.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1])


def test_padded_batch():
    """Tokens behind the real ones (any finite values) change nothing of the
    real ones' rows."""
    blk = Block(48, 100)
    want = bits(blk.run())
    pad = Block(49, 140)
    for n in ("x", "logits"):
        getattr(pad.inp, n)[:100].copy_(getattr(blk.inp, n))
    for n in ("w13", "w13_scale", "w2", "w2_scale", "bias"):
        setattr(pad.inp, n, getattr(blk.inp, n))
    for n in ("residual", "delta"):
        getattr(pad, n)[:100].copy_(getattr(blk, n))
    pad.g1, pad.g2 = blk.g1, blk.g2
    got = [t[:100] for t in pad.run()]
    assert same([t.contiguous() for t in got], want)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_inputs_let_go_while_another_stream_needs_them(raw):
    """Inputs that the caller drops right after a call on a stream that has not
    begun with it keep their memory until that stream is through."""
    blk = Block(50, 60)
    inp, sh = blk.inp, SHAPE
    q, xs = quantise(inp.x)
    r = route_rows(inp.logits, inp.bias, top_k=sh.top_k, routed_scale=sh.routed_scale)
    h, hs = grouped_swiglu(q, xs, inp.w13, inp.w13_scale, r.offsets, limit=sh.limit, rows=r.rows)
    y = grouped_gemm(h, hs, inp.w2, inp.w2_scale, r.offsets)
    calls = [
        (add_rmsnorm_quant, (blk.residual, blk.g1), dict(delta=blk.delta)),
        (add_rmsnorm_quant, (blk.residual, blk.g2), dict(y=y, pos=r.pos, weights=r.weights)),
        (route_rows, (inp.logits, inp.bias), dict(top_k=sh.top_k, routed_scale=sh.routed_scale)),
        (grouped_swiglu, (q, xs, inp.w13, inp.w13_scale, r.offsets), dict(limit=sh.limit, rows=r.rows)),
        (grouped_gemm, (h, hs, inp.w2, inp.w2_scale, r.offsets), {}),
    ]
    copy = lambda v: v.clone() if isinstance(v, torch.Tensor) else v  # noqa: E731
    flat = lambda out: list(out) if isinstance(out, tuple) else [out]  # noqa: E731
    for call, args, kw in calls:
        want = bits(flat(call(*args, **kw)))
        s = torch.cuda.Stream()
        mine, mkw = [copy(v) for v in args], {n: copy(v) for n, v in kw.items()}
        like = [v for v in (*mine, *mkw.values()) if isinstance(v, torch.Tensor)]
        at = {v.data_ptr() for v in like}
        shapes = [(v.shape, v.dtype) for v in like]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = flat(call(*mine, **mkw, stream=s.cuda_stream if raw else s))
        del mine, mkw, like
        new = [torch.empty(n, dtype=d, device=DEV) for n, d in shapes]
        for t in new:
            t.view(torch.uint8).fill_(0x11)
        assert not at & {t.data_ptr() for t in new}
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_captured_with_the_stream_given():
    """A capture on a stream that the calls are given too."""
    blk = Block(51, 70)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    blk.run(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = blk.run(s)
    for seed in range(3):
        blk.residual.copy_(torch.randn(blk.residual.shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        replayed = bits(out)
        assert same(replayed, blk.run())
        torch.cuda.synchronize()
