"""Where moe_join_rmsnorm_quant rounds, from the definition written out here.

Without the second norm the FP8 scales show the largest FP32 values of the row
h bit by bit: scale = FP32(max |h| / 448). h is rounded once from
residual_scale residual + gate n, whose products FP64 holds exactly (24 by 24
bits; a sum that float64 rounds onto the middle of two FP32 values is one in
2^28), where n is the block's output or its norm (b rstd) (post_gamma +
gamma_offset), an FP32 rounding each as in moe_add_rmsnorm_quant. The scales are
bit-equal, but for an rstd next to a rounding border (FP64 sums in another order:
one row in 2^13 at most; the inputs are seeded, so a pass stays a pass)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from fp8_block_scaled_moe_amd import join_rmsnorm_quant

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
EPS = 2.0**-20


def f32(v):
    return np.asarray(v, np.float64).astype(np.float32).astype(np.float64)


def host(t):
    return t.detach().cpu().to(torch.float64).numpy()


def make(T, D, seed, gate, k=0):
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = dict(residual=normal(T, D) * 3.0, delta=normal(T, D) * torch.exp2(normal(T, 1)), post_gamma=1.0 + 0.1 * normal(D))
    t = {n: v.to(BF).to(DEV) for n, v in t.items()}
    if gate:
        u = torch.rand({"row": (T, 1), "column": (1, D), "full": (T, D)}[gate], generator=g) + 0.01
        t["gate"] = (u if gate == "row" else u.to(BF)).to(DEV)
    if k:
        t["y"] = normal(T * k, D).to(BF).to(DEV)
        t["pos"] = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k).to(DEV)
        t["weights"] = (torch.rand(T, k, generator=g) + 0.05).to(DEV)
    return t


def row_of(t, residual_scale, gamma_offset):
    """h in FP32, from float64 sums and products."""
    b = host(t["delta"])
    if "y" in t:
        b = b + (host(t["weights"])[..., None] * host(t["y"])[host(t["pos"]).astype(np.int64)]).sum(1)
    n = b = f32(b)
    if "post_gamma" in t:
        rstd = f32(1.0 / np.sqrt((b * b).mean(1, keepdims=True) + EPS))
        n = f32(f32(b * rstd) * f32(host(t["post_gamma"]) + gamma_offset))
    n = n * (host(t["gate"]) if "gate" in t else 1.0)
    return f32(n + host(t["residual"]) * float(np.float32(residual_scale)))


@pytest.mark.parametrize("k", [0, 3])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "row", "column", "full"])
@pytest.mark.parametrize("T,D", [(64, 7168), (600, 640), (600, 4224), (40, 16384)])
def test_the_residual_row_is_rounded_once(T, D, gate, post, k):
    t = make(T, D, T + D, gate, k)
    if not post:
        del t["post_gamma"]
    for residual_scale, gamma_offset in ((1.0, 0.0), (0.3, 1.0), (-32767 * 2.0**-15, 0.5), (1.5, 0.0)):
        h = row_of(t, residual_scale, gamma_offset)
        res, out, q, scale = join_rmsnorm_quant(gamma=None, eps=EPS, residual_scale=residual_scale, gamma_offset=gamma_offset, **t)
        largest = np.maximum(np.abs(h).reshape(T, D // 128, 128).max(-1), np.float64(np.float32(1e-10)))
        want = f32(largest / 448.0)
        assert np.array_equal(host(scale), want), f"{int((host(scale) != want).sum())} of {want.size} scales differ"
        assert np.array_equal(host(res), host(torch.from_numpy(h).to(torch.float32).to(BF))) and torch.equal(out, res)
