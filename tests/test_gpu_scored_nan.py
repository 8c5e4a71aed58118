"""A NaN among the logits of moe_route_rows_scored."""

from __future__ import annotations

import pytest
import torch

from fp8_block_scaled_moe_amd import route_rows_scored

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def nan_of(bits):
    return torch.tensor([bits], dtype=torch.int64).to(torch.int32).view(torch.float32).to(DEV)


@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bits", [0x7FC00000, 0xFFC00000 - 2**32, -1, 0x7F800001])
@pytest.mark.parametrize("T,E,k,groups,top", [(9, 32, 4, 4, 2), (100, 32, 4, 1, 1), (40, 600, 32, 4, 2), (40, 60, 5, 6, 3)])
def test_a_nan_shows_in_every_weight_of_its_token(T, E, k, groups, top, bits, scores, renormalise):
    """... whatever its sign, its place and whether its expert could be picked; the other tokens stay as they are."""
    g = torch.Generator().manual_seed(E)
    z = (torch.randn(T, E, generator=g) * 2.0).to(DEV)
    kw = dict(top_k=k, scores=scores, groups=groups, top_groups=top, renormalise=renormalise)
    want = route_rows_scored(z, **kw)
    bad = {1: 0, 3: E - 1, T - 1: E // 2}
    for t, e in bad.items():
        z[t, e] = nan_of(bits)[0]
    assert int(z.isnan().sum()) == len(bad)
    r = route_rows_scored(z, **kw)
    others = torch.tensor([t for t in range(T) if t not in bad], device=DEV)
    assert torch.equal(r.ids[others], want.ids[others]) and torch.equal(r.weights[others], want.weights[others])
    for t in bad:
        assert r.weights[t].isnan().all(), r.weights[t]
        assert len(set(r.ids[t].tolist())) == k and 0 <= int(r.ids[t].min()) and int(r.ids[t].max()) < E


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_a_bf16_nan_of_either_sign(scores):
    z = torch.randn(3, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    z.view(torch.int16)[1, 5], z.view(torch.int16)[2, 5] = 0x7FC0, -0x40
    r = route_rows_scored(z.to(DEV), top_k=4, scores=scores)
    assert not r.weights[0].isnan().any() and r.weights[1:].isnan().all()


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_a_nan_in_the_bias(scores):
    z, b = torch.randn(5, 64, generator=torch.Generator().manual_seed(2)).to(DEV), torch.zeros(64, device=DEV)
    b[9] = -float("nan")
    assert route_rows_scored(z, b, top_k=4, scores=scores, groups=4, top_groups=2).weights.isnan().all()


def test_plus_infinity():
    """A sigmoid of 1; a softmax has no value."""
    z = torch.zeros(3, 64, device=DEV)
    z[1, 40] = float("inf")
    r = route_rows_scored(z, top_k=4, renormalise=False)
    assert r.ids[1].tolist() == [40, 0, 1, 2] and r.weights[1].tolist() == [1.0, 0.5, 0.5, 0.5]
    r = route_rows_scored(z, top_k=4, scores="softmax")
    assert r.weights[1].isnan().all() and not r.weights[::2].isnan().any() and len(set(r.ids[1].tolist())) == 4
