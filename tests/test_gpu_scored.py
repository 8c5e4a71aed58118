"""moe_route_rows_scored on the GPU against oracle/block.py: ids, offsets, rows
and positions exactly, weights to 1e-6 relative (a score is one rounding of a
float64 value that both sides have to some 2^-50, so both differ by at most one
step of 2^-23; the sum of up to 32 and two more operations add as much again:
under 4 * 2^-23 = 5e-7).

Where a float64 score lies within 2^-50 of the border between two binary32
values the sides may round it apart, one score in 2^26; that can change a pick
only next to an equal key. The inputs are seeded, so a pass stays a pass."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from fp8_block_scaled_moe_amd import route_rows, route_rows_scored
from oracle import block as ref
from oracle import rows

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def make(T, E, seed, dtype=torch.float32, ties=False, bias=0.1):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E)) * 2.0
    if ties:
        z = np.round(z)
    b = None if bias is None else torch.from_numpy((np.round(rng.standard_normal(E)) * 0.5 if ties else rng.standard_normal(E) * bias)
                                                   .astype(np.float32)).to(DEV)
    return torch.from_numpy(z.astype(np.float32)).to(dtype).to(DEV), b


def check(logits, bias, k, *, scale=2.5, local_begin=0, local_experts=None, **kw):
    r = route_rows_scored(logits, bias, top_k=k, routed_scale=scale, local_begin=local_begin, local_experts=local_experts, **kw)
    torch.cuda.synchronize()
    E = logits.shape[1]
    groups = kw.get("groups", 1)
    best = kw.get("group_best") or min(2, E // groups)
    ids, weights, _ = ref.route_scored(logits.double().cpu().numpy(), None if bias is None else bias.double().cpu().numpy(), k, scale,
                                       kind=kw.get("scores", "sigmoid"), groups=groups, top_groups=kw.get("top_groups") or groups,
                                       group_best=best, renormalise=kw.get("renormalise", True))
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    np.testing.assert_allclose(r.weights.cpu().numpy(), weights, rtol=1e-6, atol=1e-44)
    offsets, of, pos = rows.group_routes(ids, local_begin, E - local_begin if local_experts is None else local_experts)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy()[: len(of)], of)
    assert np.array_equal(r.pos.cpu().numpy(), pos)
    return r


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 129, 513])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,groups,top", [(8, 2, 4, 2), (256, 8, 8, 4), (256, 6, 1, 1)])
def test_tokens(T, scores, E, k, groups, top):
    check(*make(T, E, T + E), k, scores=scores, groups=groups, top_groups=top)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (7, 7), (63, 5), (64, 32), (65, 6), (128, 8), (129, 9), (257, 6), (512, 32), (513, 4),
                                 (896, 16), (1024, 32)])
def test_experts(E, k, scores, renormalise):
    check(*make(40, E, E), k, scores=scores, renormalise=renormalise)
    check(make(5, E, E + 1)[0], None, k, scores=scores, renormalise=renormalise)


# groups of one expert to 512, a number of groups that is no power of two, one to all of them
GROUPS = [(8, 8, 3), (12, 3, 2), (60, 4, 1), (60, 60, 20), (64, 64, 40), (96, 6, 5), (130, 13, 4), (160, 8, 3), (160, 5, 5), (256, 8, 1),
          (256, 64, 33), (384, 6, 2), (576, 9, 4), (896, 8, 4), (896, 56, 30), (1000, 40, 7), (1024, 2, 1), (1024, 64, 64), (1024, 16, 2)]


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("E,groups,top", GROUPS)
def test_groups(E, groups, top, best, scores):
    if best > E // groups:
        best = 1
    k = min(top * (E // groups), 32)  # where they just fit: every expert of the groups
    for take in {k, max(1, k // 3)}:
        check(*make(35, E, E + groups), take, scores=scores, groups=groups, top_groups=top, group_best=best)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,groups,top", [(256, 8, 8, 4), (896, 16, 7, 2), (64, 20, 4, 2), (40, 4, 1, 1)])
def test_equal_scores(E, k, groups, top, scores):
    """Rounded logits and biases: many equal keys and equal groups, the lower index first."""
    check(*make(70, E, 1, ties=True), k, scores=scores, groups=groups, top_groups=top)
    z = torch.zeros(3, E, device=DEV)
    r = check(z, None, k, scores=scores, groups=groups, top_groups=top)
    assert torch.equal(r.ids, torch.arange(k, device=DEV, dtype=torch.int32).expand(3, k))


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [1, 40, 1000])
def test_bf16_logits(T, scores):
    check(*make(T, 896, T, dtype=torch.bfloat16), 16, scores=scores, groups=8, top_groups=4)
    check(make(T, 896, T + 1, dtype=torch.bfloat16)[0], None, 16, scores=scores, renormalise=False)


@pytest.mark.parametrize("seed", range(30))
def test_drawn(seed):
    rng = np.random.default_rng(seed)
    E = int(round(np.exp(rng.uniform(0, np.log(1024)))))
    groups = int(rng.choice([g for g in range(1, 65) if E % g == 0]))
    top = int(rng.integers(1, groups + 1))
    k = int(rng.integers(1, min(top * (E // groups), 32) + 1))
    T = int(round(np.exp(rng.uniform(0, np.log(600)))))
    check(*make(T, E, seed, bias=(None, 0.1)[int(rng.integers(2))], dtype=(torch.float32, torch.bfloat16)[int(rng.integers(2))]), k,
          scores=("sigmoid", "softmax")[int(rng.integers(2))], groups=groups, top_groups=top, group_best=int(rng.integers(1, min(2, E // groups) + 1)),
          renormalise=bool(rng.integers(2)), scale=float(rng.uniform(0.1, 3.0)))


def test_many_tokens():
    """Every form of the grouping, at sizes where the picks can be checked token by token on the CPU for some."""
    for T in (8193, 65537):
        z, b = make(T, 64, T)
        r = route_rows_scored(z, b, top_k=4, routed_scale=1.0, scores="softmax", groups=8, top_groups=3)
        some = np.unique(np.linspace(0, T - 1, 500).astype(int))
        ids, _, _ = ref.route_scored(z[some].double().cpu().numpy(), b.double().cpu().numpy(), 4, 1.0, kind="softmax", groups=8, top_groups=3, group_best=2)
        assert np.array_equal(r.ids[some].cpu().numpy(), ids)
        flat, order = torch.sort(r.ids.flatten(), stable=True)
        assert torch.equal(r.rows, (order // 4).to(torch.int32))
        assert torch.equal(r.offsets.long(), torch.searchsorted(flat, torch.arange(65, device=DEV, dtype=torch.int32)))
        assert torch.equal(r.rows[r.pos.long()], torch.arange(T, device=DEV, dtype=torch.int32)[:, None].expand(T, 4))


@pytest.mark.parametrize("T", [9, 300])
@pytest.mark.parametrize("begin,count", [(0, 8), (8, 24), (31, 1), (0, 32)])
def test_local_share(T, begin, count):
    """One GPU's share: rows behind the last local route are left as they were."""
    check(*make(T, 32, T), 4, groups=4, top_groups=2, local_begin=begin, local_experts=count)


def test_as_route_rows():
    """Sigmoid scores with a bias over all experts: the picks, weights and places of route_rows, bit by bit."""
    for T, E, k in ((1, 256, 8), (700, 256, 8), (300, 896, 16), (50, 40, 3)):
        z, b = make(T, E, T + 5)
        for a, c in zip(route_rows(z, b, top_k=k, routed_scale=2.5), route_rows_scored(z, b, top_k=k, routed_scale=2.5, groups=4, top_groups=4)):
            assert torch.equal(a, c)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_experts_switched_off(scores):
    """Logits of minus infinity score 0; a bias of minus infinity keeps an expert out; groups of such go last."""
    z, b = make(50, 64, 3)
    z[:, 5:40] = -float("inf")
    check(z, b, 6, scores=scores)
    check(z, None, 30, scores=scores, groups=8, top_groups=8)  # more picks than live experts
    z, b = make(50, 64, 4)
    b[8:16] = -float("inf")
    check(z, b, 6, scores=scores, groups=8, top_groups=7)
    b[:] = -float("inf")  # nothing but equal keys
    check(z, b, 6, scores=scores, groups=8, top_groups=2)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_groups_with_one_expert_left(scores):
    """A group's two largest keys add up to minus infinity where all but one of its experts are kept out: such groups go
    by their index, and what the one expert's key is does not matter."""
    z, b = make(40, 32, 5)
    b[8:] = -float("inf")
    b[20] = 4.0
    r = check(z, b, 4, scores=scores, groups=4, top_groups=2)
    assert (r.ids != 20).all()
    check(z, b, 9, scores=scores, groups=4, top_groups=3)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("E", [32, 256])
def test_masks_of_the_lowest_value(E, best, scores):
    """Experts kept out by the lowest finite bias are picked all the same where too few others are there, but those of
    groups that do not take part are not."""
    z, b = make(40, E, 6)
    lowest = torch.finfo(torch.float32).min
    b[:] = lowest
    b[E // 2 + 1] = b[3 * E // 4 + 1] = 0.5
    r = check(z, b, 4, scores=scores, groups=4, top_groups=2, group_best=1)
    assert (r.ids >= E // 2).all()
    check(z, b, 4, scores=scores, groups=4, top_groups=2, group_best=best)
    check(z, b, 4, scores=scores)
    z[:, 3:] = lowest  # the same in the logits: scores of 0
    check(z, None, 5, scores=scores, groups=4, top_groups=2, group_best=best)


def test_rows_of_minus_infinities():
    """A softmax over nothing has scores and weights of 0, and picks all the same."""
    z = torch.full((40, 32), -float("inf"), device=DEV)
    z[7] = 1.0
    r = check(z, None, 4, scores="softmax", groups=4, top_groups=2)
    assert (r.weights[:7] == 0).all() and (r.weights[7] > 0).all()
    check(z, None, 4, scores="sigmoid")


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_large_logits(scores):
    """Exponentials far beyond FP32's range, and scores that round to 0."""
    z, b = make(60, 100, 9)
    check(z * 500.0, b, 8, scores=scores, groups=4, top_groups=2)
    check(z * 60.0, None, 8, scores=scores, renormalise=False)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("nan")])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k", [(32, 4), (600, 32)])
def test_bad_logits_pick_distinct_experts(bad, scores, E, k):
    """... and leave the other tokens alone."""
    z, b = make(40, E, 2)
    want = route_rows_scored(z, b, top_k=k, scores=scores, groups=4, top_groups=2)
    z[3] = bad
    z[4, 7] = bad
    if bad != bad:
        z[5] = torch.full((E,), -1, dtype=torch.int32, device=DEV).view(torch.float32)  # a NaN with every bit set
    r = route_rows_scored(z, b, top_k=k, scores=scores, groups=4, top_groups=2)
    for t in (3, 4, 5):
        assert len(set(r.ids[t].tolist())) == k and 0 <= int(r.ids[t].min()) and int(r.ids[t].max()) < E
    others = torch.tensor([t for t in range(40) if t not in (3, 4, 5)], device=DEV)
    assert torch.equal(r.ids[others], want.ids[others]) and torch.equal(r.weights[others], want.weights[others])
    assert sorted(r.pos.flatten().tolist()) == list(range(40 * k))


def test_empty_batch():
    r = route_rows_scored(torch.zeros(0, 16, device=DEV), top_k=2, groups=4, top_groups=1)
    assert r.ids.shape == (0, 2) and r.offsets.tolist() == [0] * 17


def test_captured_streams_and_again():
    for T in (1, 600):
        z, b = make(T, 256, 21)
        kw = dict(top_k=8, routed_scale=2.5, scores="softmax", groups=8, top_groups=4)
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(2):
                route_rows_scored(z, b, **kw)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = route_rows_scored(z, b, **kw)
        for seed in (1, 2, 3):
            z.copy_(make(T, 256, seed)[0])
            graph.replay()
            eager = route_rows_scored(z, b, **kw)
            torch.cuda.synchronize()
            other = route_rows_scored(z, b, **kw, stream=stream)
            torch.cuda.synchronize()
            for a, c, d in zip(captured, eager, other):
                assert torch.equal(a, c) and torch.equal(a, d)
