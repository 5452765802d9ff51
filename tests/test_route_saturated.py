"""Logits whose scores are equal in 64 bits (sigmoid above 37, softmax 745 below the largest, masks of
-inf beside large negative ones): without a bias experts, and groups by one best, go by their logits;
with a bias, and for sums of two, by the formula in 64 bits.  Indices are compared whole."""
import math

import numpy as np
import pytest
import torch

import sparse_moe_layer_gb300 as moe

pytestmark = pytest.mark.gpu
INF = math.inf
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


def choose(l, k, score, bias=None, groups=1, top_groups=1, group_top=1):
    E, gs = len(l), len(l) // groups
    with np.errstate(under="ignore", over="ignore"):
        if score == "softmax":
            s = np.exp(l - l.max()) if l.max() > -INF else np.zeros(E)
            s = s / s.sum() if s.sum() else s
        else:
            s = 1.0 / (1.0 + np.exp(-l))
    c = s if bias is None else s + bias
    rank = l if bias is None else c
    part = (rank if group_top == 1 else c).reshape(groups, gs)
    best = part.max(1) if group_top == 1 else np.sort(part, axis=1)[:, -2:].sum(1)
    open_ = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
    return sorted(sorted((e for e in range(E) if e // gs in open_), key=lambda e: (-rank[e], e))[:k])


def rows(dtype):
    g = torch.Generator().manual_seed(4)
    r = torch.randn(8, 64, generator=g)
    l = torch.zeros(64, 64)
    l[0:8] = 40 + 4 * r  # sigmoid 1.0 throughout
    l[8:16] = -900 + 20 * r  # sigmoid 0.0 throughout; softmax far apart
    l[16:24] = torch.where(torch.arange(64) % 7 == 0, r, -1000 + r)  # softmax: all but ten at 0.0
    l[24:32] = torch.where(torch.arange(64) % 9 == 0, r, torch.where(r > 0, -INF, -1e4 + 64 * r))  # two kinds of masks
    l[32:40] = torch.where(torch.arange(64) < 61, torch.full((64,), -INF), -3e4 - 64 * torch.arange(64.0))
    l[40:48] = torch.where(r > 0.5, 60.0, 40 + r)  # ties at the top, saturated
    l[48:56] = 2.0 ** -12 * r  # sigmoid of bf16 values near 0.5
    l[56:64] = 1e-20 * r if dtype != "fp16" else 2.0 ** -20 * r  # sigmoid 0.5 throughout
    return l.to(DT[dtype])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_saturated_scores(score, dtype):
    l = rows(dtype)
    for k, kw in ((1, {}), (5, {}), (8, {}), (6, dict(groups=8, top_groups=3)), (6, dict(groups=16, top_groups=4)),
                  (6, dict(groups=8, top_groups=3, group_top=2)), (6, dict(bias=True)),
                  (6, dict(bias=True, groups=8, top_groups=3, group_top=2))):
        kw = dict(kw)
        bias = torch.zeros(64) if kw.pop("bias", False) else None
        idx, w = moe.route_experts(l.cuda(), k, score=score, bias=None if bias is None else bias.cuda(), **kw)
        assert torch.all(torch.isfinite(w))
        for t, row in enumerate(l.double().numpy()):
            want = choose(row, k, score, None if bias is None else bias.double().numpy(), **kw)
            assert idx[t].tolist() == want, (t, k, kw, idx[t].tolist(), want)


def test_the_larger_of_two_logits_past_one():
    l = torch.tensor([[40.0, 48.0]], device="cuda")
    assert moe.route_experts(l, 1, score="sigmoid")[0].tolist() == [[1]]
    assert moe.route_experts(l, 1, score="sigmoid", bias=torch.zeros(2, device="cuda"))[0].tolist() == [[0]]
