"""Infinite, lowest and NaN biases in the expert choice: an expert masked by its bias, an expert
that has to be taken, and groups of them; then the layer fed by such a choice.

The oracle is the formula in 64 bits with its infinities: -inf choices tie, a group with one among
its best sums to -inf and ties with its equals, a group with +inf comes first; ties go to the lower
index.  Choices are compared whole; weights need no tolerance of their own here (a bias does not
enter them): they have to equal the scores of the chosen to 2^-18, their fp32 error for |logit| < 8
(32 + 2 * 16 half steps of 2^-24, twice with the renormalising sum)."""
import math

import numpy as np
import pytest
import torch

import sparse_moe_layer_gb300 as moe

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


def choose(l, k, score, bias, groups, top_groups, group_top):
    E = len(l)
    if score == "softmax":
        s = np.exp(l - l.max())
        s = s / s.sum()
    else:
        s = 1.0 / (1.0 + np.exp(-l))
    c = s + np.where(np.isnan(bias), -INF, bias)
    gs = E // groups
    best = []
    for g in range(groups):
        m = sorted(c[g * gs:(g + 1) * gs], reverse=True)[:group_top]
        best.append(INF if m[0] == INF else sum(m))
    open_ = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
    order = sorted((e for e in range(E) if e // gs in open_), key=lambda e: (-c[e], e))[:k]
    idx = np.array(sorted(order))
    return idx, s[idx] / (s[idx].sum() + 1e-20)


def check(l, k, bias, score="sigmoid", groups=1, top_groups=1, group_top=1):
    bias = torch.as_tensor(bias, dtype=torch.float32)
    idx, w = moe.route_experts(l, k, score=score, bias=bias.cuda(), groups=groups, top_groups=top_groups, group_top=group_top)
    idx, w = idx.cpu().numpy(), w.double().cpu().numpy()
    for t, row in enumerate(l.double().cpu().numpy()):
        want, weight = choose(row, k, score, bias.double().numpy(), groups, top_groups, group_top)
        assert np.array_equal(idx[t], want), (t, idx[t], want)
        assert np.all(np.abs(w[t] - weight) <= 2.0 ** -18 * weight), (t, w[t], weight)


def draw(T, E, seed=0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, E), generator=g, device="cuda").clamp(-8, 8).to(dtype)


BOTH = pytest.mark.parametrize("score", ["softmax", "sigmoid"])


@BOTH
def test_every_group_has_a_masked_expert_among_its_best(score):
    """All sums tie at -inf: the first groups open, and their unmasked experts are taken."""
    bias = np.zeros(16)
    bias[1::2] = -INF
    check(draw(40, 16), 4, bias, score, 8, 4, 2)
    idx, _ = moe.route_experts(draw(3, 16), 4, score=score, bias=torch.tensor(bias).float().cuda(), groups=8, top_groups=4,
                               group_top=2)
    assert idx.tolist() == [[0, 2, 4, 6]] * 3


@BOTH
@pytest.mark.parametrize("E,groups,top_groups,k", [(64, 32, 8, 8), (64, 32, 3, 5), (16, 8, 4, 8), (256, 8, 4, 8), (60, 5, 2, 7),
                                                   (96, 32, 30, 8), (160, 8, 3, 6), (12, 3, 1, 4)])
def test_masked_groups(score, E, groups, top_groups, k):
    """From no group left whole to all but one; masks of -inf and NaN."""
    g = torch.Generator().manual_seed(E + groups)
    gs = E // groups
    for left in {0, 1, top_groups - 1, top_groups, groups - 1}:
        for mask in (-INF, math.nan):
            bias = 0.05 * torch.randn(E, generator=g).double().numpy()
            for gr in torch.randperm(groups, generator=g).tolist()[left:]:
                n = int(torch.randint(1, gs + 1, (1,), generator=g))
                for e in torch.randperm(gs, generator=g).tolist()[:n]:
                    bias[gr * gs + e] = mask
            for group_top in (1, 2):
                check(draw(24, E, E), k, bias, score, groups, top_groups, group_top)


@BOTH
def test_lowest_value_counts_as_masked(score):
    """The same call with finfo.min and with -inf gives the same experts."""
    l, low = draw(50, 64), torch.finfo(torch.float32).min
    bias = torch.zeros(64, device="cuda")
    for first in (3, 20, 40, 64):
        bias[:first:3] = low
        a = moe.route_experts(l, 8, score=score, bias=bias, groups=8, top_groups=3, group_top=2)
        b = moe.route_experts(l, 8, score=score, bias=torch.where(bias == low, -INF, bias), groups=8, top_groups=3, group_top=2)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@BOTH
@pytest.mark.parametrize("E", [2, 9, 31, 64, 128, 255, 256])
def test_fewer_unmasked_experts_than_chosen(score, E):
    for live in (0, 1, 3, 7):
        bias = np.full(E, -INF)
        bias[[(e * 37 + 1) % E for e in range(min(live, E))]] = 0.25
        check(draw(10, E, E), min(E, 8), bias, score)


@BOTH
def test_forced_experts(score):
    for E, k in ((64, 1), (64, 4), (256, 8)):
        bias = 0.05 * draw(1, E, 1)[0].double().cpu().numpy()
        bias[E // 2 + 3] = INF
        check(draw(30, E), k, bias, score)
        check(draw(30, E), k, bias, score, 8, 1, 1)
        check(draw(30, E), k, bias, score, 8, 1, 2)
        check(draw(30, E), min(k, 8), bias, score, 8, 4, 2)
        bias[E // 2 + 2] = -INF  # and its neighbour masked
        check(draw(30, E), k, bias, score, 8, 2, 2)
        bias[[1, 7, E - 1]] = INF
        check(draw(30, E), k, bias, score)
        check(draw(30, E), k, bias, score, 8, 2, 2)
    bias = np.full(32, -INF)
    bias[21] = INF  # alone in a masked group: the group opens
    check(draw(20, 32), 4, bias, score, 4, 1, 2)


@BOTH
def test_large_finite_biases(score):
    for size in (1e3, 1e6, 1e12, 1e30):
        g = torch.Generator().manual_seed(7)
        bias = size * torch.randint(-2, 3, (64,), generator=g).float()
        for groups, top, two in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
            # choices of 64 bits: below 2^-53 of the bias the scores are lost there too
            check(draw(40, 64, 5), 8, bias, score, groups, top, two)


def test_16_bit_logits_and_masks():
    bias = np.zeros(64)
    bias[::3] = -INF
    for dtype in (torch.bfloat16, torch.float16):
        check(draw(100, 64, 2, dtype), 6, bias, "sigmoid", 8, 4, 2)
        check(draw(100, 64, 2, dtype), 6, bias, "softmax", 32, 9, 2)
        check(draw(100, 64, 2, dtype), 6, bias, "softmax")


def test_gated_layer_on_masked_experts():
    """The layer gets distinct experts for every place, and their rows add up."""
    import synth
    from harness import Layer
    L = Layer(synth.config("tiny")).to_device()
    weights = (L.d_w13, L.d_s13, L.d_b13, L.d_w2, L.d_s2, L.d_b2)
    l = draw(L.T, L.E, 3)
    for bias, kw in (([0.0, -INF] * (L.E // 2), dict(groups=4, top_groups=2, group_top=2)),
                     ([-INF] * (L.E - 1) + [0.0], dict(groups=4, top_groups=2, group_top=2)),
                     ([-INF] * L.E, dict()), ([INF] + [0.0] * (L.E - 1), dict(groups=2, top_groups=1, group_top=2))):
        bias = torch.tensor(bias).cuda()
        k = 4
        ws = moe.new_workspace(L.T, L.H, L.I, L.E, k)
        ws.fill_(0xFF)
        out = moe.forward_gated(L.d_x, l, *weights, k, score="sigmoid", bias=bias, workspace=ws, **kw)
        assert moe.read_device_status(ws) == 0 and torch.all(torch.isfinite(out))
        idx, w = moe.route_experts(l, k, score="sigmoid", bias=bias, **kw)
        v = moe.workspace_views(ws, L.T, L.H, L.I, L.E, k)
        assert torch.equal(v["topk_idx"], idx) and torch.equal(v["topk_w"], w)
        assert torch.all(idx[:, 1:] > idx[:, :-1]) and int(idx.min()) >= 0 and int(idx.max()) < L.E
        assert torch.equal(v["perm"].long(), torch.sort(idx.flatten().long(), stable=True).indices)
