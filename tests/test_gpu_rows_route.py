"""moe_route_rows on the GPU: picks and weights against the oracle's routing
(ids bit-exact, weights to 1e-6 relative, the layer's bar), the grouping
against oracle/rows.py's, exactly, and both against moe_decode_run's ids."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import synth
from fp8_block_scaled_moe_amd import MoeDecode, route_rows
from oracle import rows as ref
from tests.helpers import WEIGHT_RTOL

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def make(T, E, seed, dtype=torch.float32, ties=False):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E)) * 2.0
    if ties:
        z = np.round(z)
    return torch.from_numpy(z.astype(np.float32)).to(dtype).to(DEV), torch.from_numpy(
        (np.zeros(E) if ties else rng.standard_normal(E) * 0.1).astype(np.float32)).to(DEV)


def check(logits, bias, k, scale=2.5, **local):
    r = route_rows(logits, bias, top_k=k, routed_scale=scale, **local)
    torch.cuda.synchronize()
    T, E = logits.shape
    lb = local.get("local_begin", 0)
    lc = local.get("local_experts") or E - lb
    ids, weights, _ = oracle.route(logits.float().cpu().numpy().astype(np.float64), bias.cpu().numpy().astype(np.float64), k, scale)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    np.testing.assert_allclose(r.weights.cpu().numpy(), weights, rtol=WEIGHT_RTOL, atol=0)
    offsets, rows, pos = ref.group_routes(ids, lb, lc)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy()[: len(rows)], rows)
    assert np.array_equal(r.pos.cpu().numpy(), pos)
    return r


# tokens around the one-workgroup form (32) and the ends of chunks; experts around each number per lane
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 512, 513])
@pytest.mark.parametrize("E,k", [(8, 2), (256, 8)])
def test_tokens(T, E, k):
    check(*make(T, E, T + E), k)


@pytest.mark.parametrize("T", [5, 130])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (7, 7), (63, 5), (64, 32), (65, 6), (128, 8), (129, 9), (257, 6), (512, 32), (513, 4),
                                 (896, 16), (1024, 32)])
def test_experts(T, E, k):
    check(*make(T, E, 3 * T + E), k)


@pytest.mark.parametrize("T", [32, 300])
def test_bf16_logits(T):
    check(*make(T, 200, 5, torch.bfloat16), 6, scale=1.0)


@pytest.mark.parametrize("T", [25, 150])
@pytest.mark.parametrize("E,k", [(64, 8), (600, 16)])
def test_equal_scores_go_to_the_lower_expert(T, E, k):
    check(*make(T, E, 6, ties=True), k)


@pytest.mark.parametrize("T", [30, 33, 150])
@pytest.mark.parametrize("lb,lc", [(0, 8), (8, 24), (63, 1), (0, 64), (32, None)])
def test_local_experts(T, lb, lc):
    r = check(*make(T, 64, 7), 4, local_begin=lb, local_experts=lc)
    assert r.offsets.shape[0] == (32 if lc is None else lc) + 1


@pytest.mark.parametrize("T", [32, 200])
def test_one_expert_takes_all_and_one_none(T):
    logits, bias = make(T, 16, 8)
    bias[3], bias[5] = 50.0, -50.0
    r = check(logits, bias, 2)
    n = (r.offsets[1:] - r.offsets[:-1]).tolist()
    assert n[3] == T and n[5] == 0


def test_infinite_logits():
    logits, bias = make(70, 32, 9)
    logits[0, 4], logits[1, :] = float("inf"), float("-inf")
    logits[2, 7] = float("-inf")
    r = route_rows(logits, bias, top_k=3, routed_scale=1.0)
    key = torch.sigmoid(logits.double()).float() + bias
    want = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :3].int()
    assert torch.equal(r.ids, want)


@pytest.mark.parametrize("mask", [float("-inf"), torch.finfo(torch.float32).min], ids=["infinity", "lowest"])
@pytest.mark.parametrize("T", [25, 150])
def test_masked_experts(T, mask):
    """Experts switched off by their bias are not picked while k others are
    there, and are picked in their order where not."""
    logits, bias = make(T, 100, 41)
    bias[3:60] = mask
    r = check(logits, bias, 8)
    assert not ((r.ids >= 3) & (r.ids < 60)).any()
    bias[5:] = mask
    check(logits, bias, 8)
    bias[:] = mask
    check(logits, bias, 8)


@pytest.mark.parametrize("T", [20, 200])
def test_nan_logits_give_valid_places(T):
    """Whatever a NaN is routed to, every place is a row of the batch."""
    logits, bias = make(T, 32, 10)
    logits[1, :] = float("nan")
    logits[3, 5] = float("nan")
    r = route_rows(logits, bias, top_k=4, routed_scale=1.0)
    ids = r.ids.cpu().numpy()
    assert ids.min() >= 0 and ids.max() < 32 and all(len(set(row)) == 4 for row in ids)
    offsets, rows, pos = ref.group_routes(ids, 0, 32)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets) and np.array_equal(r.pos.cpu().numpy(), pos)
    assert np.array_equal(r.rows.cpu().numpy(), rows)


def test_no_tokens():
    r = route_rows(torch.empty((0, 16), device=DEV), torch.zeros(16, device=DEV), top_k=2, routed_scale=1.0)
    assert r.ids.shape == (0, 2) and r.rows.shape == (0,) and r.offsets.tolist() == [0] * 17


@pytest.mark.parametrize("E,lb,lc", [(1, 0, 1), (16, 4, 8), (1024, 0, 1024)])
def test_no_tokens_needs_the_offsets_alone(E, lb, lc):
    """An empty batch of a C caller: every pointer but offsets is NULL."""
    import ctypes
    from fp8_block_scaled_moe_amd import _rows, lib

    buf = torch.full((lc + 3,), -7, dtype=torch.int32, device=DEV)
    a = _rows.RouteArgs(T=0, E=E, k=1, local_begin=lb, local_experts=lc, routed_scale=1.0, offsets=buf[1:].data_ptr())
    assert lib().moe_route_rows(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    assert buf.tolist() == [-7] + [0] * (lc + 1) + [-7]


def test_rows_behind_the_last_stay(T=100):
    """Entries of rows from offsets[-1] on are not written."""
    import ctypes
    from fp8_block_scaled_moe_amd import _rows, lib

    logits, bias = make(T, 64, 11)
    k, lc = 4, 8
    i32 = dict(dtype=torch.int32, device=DEV)
    ids, pos, weights = torch.empty(T, k, **i32), torch.empty(T, k, **i32), torch.empty(T, k, device=DEV)
    offsets, rows = torch.empty(lc + 1, **i32), torch.full((T * k,), -7, **i32)
    ws = torch.empty(lib().moe_route_rows_workspace(T, lc), dtype=torch.uint8, device=DEV)
    a = _rows.RouteArgs(T, 64, k, 0, 8, lc, 1.0, logits.data_ptr(), bias.data_ptr(), ids.data_ptr(), weights.data_ptr(),
                        offsets.data_ptr(), rows.data_ptr(), pos.data_ptr(), ws.data_ptr(), ws.numel())
    assert lib().moe_route_rows(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    n = int(offsets[-1])
    assert 0 < n < T * k and (rows[n:] == -7).all() and (rows[:n] >= 0).all()


@pytest.mark.parametrize("T,E,k", [(8192, 64, 4), (8193, 40, 3), (16385, 256, 8), (65537, 72, 2), (70001, 16, 1)])
def test_long_prompts_against_plain_operations(T, E, k):
    """Around the sizes where a chunk's tokens change: sorted by stable
    library sorts."""
    logits, bias = make(T, E, 12)
    r = route_rows(logits, bias, top_k=k, routed_scale=2.5)
    key = (1.0 / (1.0 + torch.exp(-logits.double()))).float() + bias
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.ids.long(), ids)
    flat, order = torch.sort(ids.flatten(), stable=True)
    assert torch.equal(r.rows.long(), order // k)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device=DEV)
    assert torch.equal(r.pos.long().flatten(), pos)
    assert torch.equal(r.offsets.long(), torch.searchsorted(flat, torch.arange(E + 1, device=DEV)))


def test_ids_and_weights_are_the_layers():
    shape = synth.CONFIGS["tiny"].with_(M=100, hidden=256, inter=128, experts=96, top_k=6)
    inp = synth.make_inputs(shape, seed=13, device=DEV)
    moe = MoeDecode(inp.w13, inp.w13_scale, inp.w2, inp.w2_scale, top_k=6, limit=shape.limit, routed_scale=shape.routed_scale,
                    max_tokens=100, logits_dtype=inp.logits.dtype)
    _, ids, weights, _ = moe(inp.x, inp.logits, inp.bias)
    r = route_rows(inp.logits, inp.bias, top_k=6, routed_scale=shape.routed_scale)
    assert torch.equal(r.ids, ids) and torch.equal(r.weights, weights)
