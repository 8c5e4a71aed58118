"""How near the activations of moe_dense_gemm are to their values: the products are
zeros, so that the bias, in FP32, is what the activation gets."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from fp8_block_scaled_moe_amd import dense_gemm

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16


def activation(v, act):
    v = v.astype(np.float64)
    return (v if act == "silu" else 1.0) / (1.0 + np.exp(-v))


def run(v, act, dtype, T):
    x, w = torch.zeros(T, 16, dtype=BF, device=DEV), torch.zeros(len(v), 16, dtype=BF, device=DEV)
    got = dense_gemm(x, w, bias=torch.from_numpy(v).to(DEV), act=act, out_dtype=dtype)
    assert torch.equal(got, got[:1].expand_as(got))
    return got[0].cpu().to(torch.float64).numpy()


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("T", [1, 300])
@pytest.mark.parametrize("low,high", [(-87.0, -80.0), (-80.0, -40.0), (-40.0, -8.0), (-8.0, 20.0)])
def test_fp32_outputs_are_as_near_as_stated(low, high, T, act):
    """The exponential and the reciprocal are one step of 2^-23 off at most, the three roundings around them half of
    one each, what the argument lost 2^-40: 3.5 * 2^-23, where 4 are stated."""
    v = np.random.default_rng(int(-low)).uniform(low, high, 200000).astype(np.float32)
    want = activation(v, act)
    off = np.abs(run(v, act, torch.float32, T) - want) / np.abs(want)
    assert off.max() <= 3.5 * 2.0**-23, f"{off.max() * 2.0**23} at {v[off.argmax()]}"


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("T,odd", [(1, 0), (300, 0), (300, 1)])
@pytest.mark.parametrize("low,high", [(-80.0, -30.0), (-30.0, -10.0), (-10.0, 10.0)])
def test_bf16_outputs_are_rounded_from_values_as_near(low, high, T, odd, act):
    """Values that lie 4.5 to 12 * 2^-23 of themselves beside the middle of two BF16 values round to the right one."""
    v = np.random.default_rng(int(-low) + odd).uniform(low, high, 4000000).astype(np.float32)
    want = activation(v, act)
    below = (np.abs(want).astype(np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32).astype(np.float64)
    middle = below + np.ldexp(1.0, np.frexp(below)[1] - 9)
    off = (np.abs(want) - middle) / middle
    keep = np.flatnonzero((np.abs(off) >= 4.5 * 2.0**-23) & (np.abs(off) <= 12 * 2.0**-23))[: 1200 + odd]
    right = np.sign(want) * np.where(off > 0, 2 * middle - below, below)
    got = run(v[keep], act, BF, T)
    wrong = got != right[keep]
    assert len(keep) >= 500 and not wrong.any(), f"{int(wrong.sum())} of {len(keep)} values, the first at {v[keep][wrong][0]}"
