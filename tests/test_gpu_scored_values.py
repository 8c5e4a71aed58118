"""The last bits of moe_route_rows_scored's softmax scores."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from fp8_block_scaled_moe_amd import route_rows_scored

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def next_to_borders(count, seed):
    """Pairs of FP32 logits (about 0 and -d) whose second softmax score, in 64-bit
    mantissas, lies 2^-50 to 2^-49.2 of itself beside the middle of two FP32 values, and
    that score rounded. d is close to an odd multiple of ln 2 / 64, as far from the
    multiples of ln 2 / 32 as an argument can be."""
    L = np.longdouble
    rng = np.random.default_rng(seed)
    z1, z2, want = [], [], []
    for _ in range(20):  # some thousand of each draw are kept
        n = rng.integers(32 * 3, 32 * 18, size=40000)
        d = (L(1.0) * n + L(0.5) + rng.uniform(-0.01, 0.01, n.size)) * np.log(L(2.0)) / 32
        below = (np.exp(-d) / (1 + np.exp(-d))).astype(np.float64).astype(np.float32)
        middle = (L(1.0) * below + L(1.0) * np.nextafter(below, np.float32(1.0))) / 2
        target = np.log((1 - middle) / middle)  # d of the middle: b, and a for what is left
        b = target.astype(np.float64).astype(np.float32)
        a = (target - b).astype(np.float64).astype(np.float32)
        # the definition's difference of the logits, in float64, is their difference
        whole = L(1.0) * (a.astype(np.float64) + b.astype(np.float64)) == L(1.0) * a + L(1.0) * b
        e = np.exp(-(L(1.0) * a + L(1.0) * b))
        off = (e / (1 + e) - middle) / middle
        keep = whole & (np.abs(off) > L(2.0) ** -50) & (np.abs(off) < L(2.0) ** L(-49.2))
        z1.extend(a[keep])
        z2.extend(-b[keep])
        want.extend(np.where(off > 0, np.nextafter(below, np.float32(1.0)), below)[keep])
        if len(want) >= count:
            break
    return np.array(z1[:count]), np.array(z2[:count]), np.array(want[:count])


@pytest.mark.parametrize("E,at", [(2, (0, 1)), (70, (3, 67)), (896, (1, 890))])
def test_softmax_scores_next_to_rounding_borders(E, at):
    """A score is the FP32 rounding of a value that is off by a few roundings of FP64: 2^-53 each for the polynomial's
    last sum, the table's entry, their product, the sum and its reciprocal, less than 2^-50 in all."""
    z1, z2, want = next_to_borders(400, E)
    z = np.full((len(want), E), -np.inf, np.float32)
    z[:, at[0]], z[:, at[1]] = z1, z2
    r = route_rows_scored(torch.from_numpy(z).to(DEV), top_k=2, scores="softmax", renormalise=False)
    assert (r.ids.cpu().numpy() == np.array(at)).all()
    got = r.weights.cpu().numpy()[:, 1]
    assert np.array_equal(got, want), f"{int((got != want).sum())} of {len(want)} scores differ"
