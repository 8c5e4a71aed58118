"""Groups of moe_route_rows_scored whose two largest keys are far apart: biases of
+B and -B in a group, so that its value is of size 1 and its keys, with their
roundings, of size B. Everything is compared exactly with oracle/block.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from fp8_block_scaled_moe_amd import route_rows_scored
from oracle import block as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
G = 8


def sigmoid32(z):
    return (1.0 / (1.0 + np.exp(-z.astype(np.float64)))).astype(np.float32)


def logit32(s):
    return np.log(s / (1.0 - s)).astype(np.float32)


def pairs(rng, shape, B, total):
    """Logits (z1, z2) whose keys with biases +B and -B add up to about `total`, the first one's score within some 2^-24
    of a value at which its key turns."""
    step = float(np.spacing(np.float32(B)))  # of the keys from B on
    steps = int(0.9 / step)
    n = rng.integers(int(0.1 * steps), max(int(0.8 * steps), int(0.1 * steps) + 1), size=shape)
    z1 = logit32(np.clip((n + 0.5) * step, 0.02, 0.98))
    key1 = sigmoid32(z1) + np.float32(B)
    s2 = total - (key1.astype(np.float64) - B)
    return z1, logit32(np.clip(s2, 0.02, 0.98))


def check(z, bias, k, top):
    r = route_rows_scored(torch.from_numpy(z).to(DEV), torch.from_numpy(bias).to(DEV), top_k=k, groups=G, top_groups=top, group_best=2)
    ids, weights, _ = ref.route_scored(z, bias, k, 1.0, groups=G, top_groups=top, group_best=2)
    wrong = np.flatnonzero((r.ids.cpu().numpy() != ids).any(axis=1))
    assert not len(wrong), f"{len(wrong)} of {len(z)} tokens, the first {wrong[0]}: {r.ids[wrong[0]].tolist()}, not {ids[wrong[0]].tolist()}"
    np.testing.assert_allclose(r.weights.cpu().numpy(), weights, rtol=1e-6)


@pytest.mark.parametrize("T", [20, 700])
@pytest.mark.parametrize("size", [2, 32])
@pytest.mark.parametrize("B", [64.0, 1024.0, 4096.0, 8192.0, 2.0**16, 2.0**20])
def test_opposite_biases_in_every_group(B, size, T):
    """Groups that tie or are one step apart, whichever side the first key turns to."""
    rng = np.random.default_rng(int(B) + size)
    z = np.zeros((T, G, size), np.float32)
    z[..., 0], z[..., 1] = pairs(rng, (T, G), B, 1.0)
    bias = np.full((G, size), -np.inf, np.float32)
    bias[:, 0], bias[:, 1] = B, -B
    check(z.reshape(T, -1), bias.reshape(-1), 6, 4)


@pytest.mark.parametrize("size", [2, 32])
@pytest.mark.parametrize("B", [1024.0, 4096.0, 2.0**14])
def test_opposite_biases_beside_plain_groups(B, size):
    """Every other group has no bias and a value between the steps of the others'."""
    rng = np.random.default_rng(int(B) + 3)
    T, step = 700, float(np.spacing(np.float32(B)))
    z = np.full((T, G, size), -30.0, np.float32)
    z[:, 1::2, 0], z[:, 1::2, 1] = pairs(rng, (T, G // 2), B, 1.0)
    first = rng.uniform(0.3, 0.7, (T, G // 2))
    z[:, ::2, 0], z[:, ::2, 1] = logit32(first), logit32(1.0 + step * rng.choice([-0.4, 0.4], (T, G // 2)) - first)
    bias = np.zeros((G, size), np.float32)
    bias[1::2] = -np.inf
    bias[1::2, 0], bias[1::2, 1] = B, -B
    check(z.reshape(T, -1), bias.reshape(-1), 6, 4)
