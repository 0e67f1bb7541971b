"""GPU tests of the routing with biases that force an expert or take it out,
on every way a row can be decided: the list of candidates, the near ties
among them, one expert after another, and the whole row in 64 bits."""
import math

import pytest
import torch

from routed_moe_decode_router_gb300 import ops
from tests import ops_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def randn(*shape, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(3000 + seed)
    return torch.randn(*shape, generator=g, device="cuda") * std


def want(logits, top_k, bias, scoring, groups, group_limit, group_score):
    """(ids, weights) by the definition, in 64 bits: an expert whose logit or
    biased score is -inf or NaN is out."""
    x = logits.double()
    t, e = x.shape
    dead = ~(x > -math.inf)
    if scoring == "softmax":
        p = torch.softmax(x.masked_fill(dead, -math.inf), 1)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    p = p.masked_fill(dead, 0.0)
    key = p + bias.double()
    key = key.masked_fill(dead | ~(key > -math.inf), -math.inf)
    best = key.unflatten(1, (groups, -1)).sort(dim=2, descending=True).values
    score = best[:, :, 0]
    if group_score == "top2" and best.shape[2] > 1:
        score = score + best[:, :, 1].masked_fill(best[:, :, 1] == -math.inf, 0.0)
    rank = score.sort(dim=1, descending=True, stable=True).indices.argsort(1)
    key = key.masked_fill((rank >= group_limit).repeat_interleave(e // groups, 1), -math.inf)
    key, ids = key.sort(dim=1, descending=True, stable=True)
    key, ids = key[:, :top_k], ids[:, :top_k]
    w = p.gather(1, ids).masked_fill(key == -math.inf, 0.0)
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w / total, 0.0)
    return ids.masked_fill(key == -math.inf, -1).to(torch.int32), w


def check(logits, top_k, bias, scoring, groups=1, group_limit=1, group_score="max"):
    kw = dict(scoring=scoring, groups=groups, group_limit=group_limit, group_score=group_score)
    ids, w = want(logits, top_k, bias, **kw)
    got, wts = ops.route_topk(logits, top_k, bias=bias, **kw)
    assert torch.equal(got, ids), "%d rows differ" % int((got != ids).any(1).sum())
    # p: expf of a difference up to 100, the sum and the division, under 2^7 U;
    # the total and its division the same again
    assert ((wts.double() - w).abs() <= w * 2.0 ** 8 * R.U + 1e-38).all()


SCORINGS = pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])


@SCORINGS
@pytest.mark.parametrize("experts", [40, 128, 256])
@pytest.mark.parametrize("top_k,forced", [(1, 1), (1, 3), (4, 2), (4, 4), (4, 6), (8, 1), (31, 31),
                                          (32, 5), (40, 40)])
def test_forced_experts(scoring, experts, top_k, forced):
    bias = randn(experts, seed=1, std=0.1)
    bias[torch.randperm(experts, generator=torch.Generator().manual_seed(2))[:forced]] = math.inf
    check(randn(50, experts), top_k, bias, scoring)
    # beside near and exact ties
    check(randn(50, experts).round(), top_k, bias.round(), scoring)
    check(torch.zeros(3, experts, device="cuda"), top_k, bias, scoring)


@SCORINGS
@pytest.mark.parametrize("score", ["max", "top2"])
@pytest.mark.parametrize("limit", [1, 2, 3])
def test_forced_experts_in_groups(scoring, score, limit):
    for forced in ([17], [17, 18], [1, 17], [3, 17, 30], range(0, 32, 8)):
        bias = randn(32, seed=1, std=0.1)
        bias[list(forced)] = math.inf
        kw = dict(groups=4, group_limit=limit, group_score=score)
        check(randn(50, 32), 4, bias, scoring, **kw)
        # the other groups tie
        bias = torch.where(bias == math.inf, bias, 0.25)
        check(torch.zeros(3, 32, device="cuda"), 4, bias, scoring, **kw)
        check(randn(50, 8).repeat(1, 4), 4, bias, scoring, **kw)


NANS = [math.nan, -math.nan]


def test_nans_of_both_signs():
    signs = torch.tensor(NANS, device="cuda").view(torch.int32) < 0
    assert signs.tolist() == [False, True]


@SCORINGS
@pytest.mark.parametrize("value", [-math.inf] + NANS, ids=["-inf", "nan", "-nan"])
@pytest.mark.parametrize("top_k,live", [(1, 0), (4, 2), (4, 9), (8, 3), (31, 20), (32, 20), (40, 7)])
def test_experts_taken_out_by_their_bias(scoring, value, top_k, live):
    bias = randn(64, seed=1, std=0.1)
    off = torch.randperm(64, generator=torch.Generator().manual_seed(3))[live:]
    bias[off] = value
    check(randn(50, 64), top_k, bias, scoring)
    # near and exact ties: the candidates, or the row, again in 64 bits
    check(randn(50, 64).round(), top_k, bias.round(), scoring)
    check(torch.zeros(3, 64, device="cuda"), top_k, bias, scoring)
    # weights too small for fp32: the row in 64 bits
    far = randn(50, 64, seed=4) - 200.0
    far[:, off[0]] = 0.0
    check(far, top_k, bias, scoring)
    # with a logit that takes its expert out too, and one forced expert
    gone = randn(50, 64, seed=5)
    gone[::2, 7] = -math.inf
    bias[9] = math.inf
    check(gone, top_k, bias, scoring)


@SCORINGS
@pytest.mark.parametrize("value", [-math.inf] + NANS, ids=["-inf", "nan", "-nan"])
@pytest.mark.parametrize("score", ["max", "top2"])
@pytest.mark.parametrize("limit", [1, 2, 3])
def test_experts_and_groups_taken_out_by_their_bias(scoring, value, score, limit):
    for off in ([3], [0, 1, 2, 3, 4, 5, 7], list(range(8, 16)), list(range(1, 32)), list(range(32)),
                [8, 9, 10, 11, 12, 13, 14, 24, 25, 26, 27, 28, 29, 30]):
        bias = randn(32, seed=1, std=0.1)
        bias[off] = value
        kw = dict(groups=4, group_limit=limit, group_score=score)
        check(randn(50, 32), 8, bias, scoring, **kw)
        bias = torch.where(bias == bias.clamp(-9, 9), 0.25, bias)
        # groups that tie
        check(torch.zeros(3, 32, device="cuda"), 8, bias, scoring, **kw)
        check(randn(50, 8).repeat(1, 4), 8, bias, scoring, **kw)
        check(randn(50, 32) - 200.0, 8, bias, scoring, **kw)


@SCORINGS
@pytest.mark.parametrize("limit", [1, 3, 8, 31])
@pytest.mark.parametrize("big", [0.5, 8.0, 64.0, 256.0, 1000.0, 1e6])
def test_groups_whose_two_best_cancel(scoring, limit, big):
    """The score of a group is what is left of two large biased scores."""
    bias = torch.tensor([big, -big] * 32, device="cuda")
    kw = dict(groups=32, group_limit=limit, group_score="top2")
    check(randn(4096, 64), 2, bias, scoring, **kw)
    # all groups near each other: logits some steps of fp32 apart
    steps = torch.randint(-8, 9, (500, 64), generator=torch.Generator().manual_seed(6)).cuda()
    check(randn(500, 2, seed=7).repeat(1, 32) * (1 + steps * 2.0 ** -21), 2, bias, scoring, **kw)
    few = dict(groups=4, group_limit=min(limit, 3), group_score="top2")
    bias = torch.cat([randn(28, seed=8, std=0.1), bias[:4]]).view(2, 16).t().reshape(32)
    check(randn(500, 8, seed=7).repeat(1, 4) * (1 + steps[:, :32] * 2.0 ** -21), 4, bias, scoring,
          **few)


@SCORINGS
def test_group_scores_beyond_fp32(scoring):
    pairs = [(2e38, 3.3e38), (3e38, 1e38), (1.0, 2.0), (-3e38, -3e38), (-2e38, -3.3e38),
             (-math.inf, -3e38), (-math.inf, -math.inf), (3.4e38, -3.4e38)]
    bias = torch.tensor(pairs, device="cuda").flatten()
    for limit in range(1, 9):
        check(randn(20, 16), 2, bias, scoring, groups=8, group_limit=limit, group_score="top2")
