"""The gated layer on prompts: several histogram chunks, more tokens than the gate's grid has warps, more
chunks than the scan stages in shared memory (24 of them at 32 experts), and the prefill GEMM tiles.

Routing has to be the operator's own, whole.  The output is the sum of the experts' outputs y_e
(each expert alone, in the same GEMM kernels) by the weights in bf16, to the two roundings of bf16
outputs: each y_e 2^-8 of its term, the sum k + 4 roundings of fp32, the output 2^-8."""
import math

import pytest
import torch

import sparse_moe_layer_gb300 as moe

pytestmark = pytest.mark.gpu
PACK = {"block128": moe.pack_weights, "mxfp8": moe.pack_weights_mx, "mxfp4": moe.pack_weights_mxfp4}


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


@pytest.mark.parametrize("fmt", ["block128", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("T", [257, 300, 6500, 9001])  # the short ones on the decode tiles, as their experts alone
def test_prompts(T, fmt):
    E, H, I, k = 32, 256, 256, 4
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = n(T, H).bfloat16()
    weights = PACK[fmt](0.1 * n(E, 2 * I, H), 0.1 * n(E, H, I))
    w13, s13, w2, s2 = weights
    args = (w13, s13, 0.1 * n(E, 2 * I).bfloat16(), w2, s2, 0.1 * n(E, H).bfloat16())
    logits = n(T, E)
    logits[:, 5] -= 8.0  # an expert with few tokens
    logits[T // 2:, 7] = -math.inf  # one that later chunks do not have
    kw = dict(score="sigmoid", bias=0.1 * n(E), groups=4, top_groups=2, group_top=2, scale=2.5)
    mx = fmt != "block128"
    for gate in (kw, dict()):
        ws = moe.new_workspace(T, H, I, E, k, mx=mx)
        ws.fill_(0xFF)
        out = moe.forward_gated(x, logits, *args, k, workspace=ws, **gate)
        assert moe.read_device_status(ws) == 0
        idx, w = moe.route_experts(logits, k, **gate)
        v = moe.workspace_views(ws, T, H, I, E, k, mx=mx)
        assert torch.equal(v["topk_idx"], idx) and torch.equal(v["topk_w"], w)
        order = torch.sort(idx.flatten().long(), stable=True).indices
        assert torch.equal(v["perm"].long(), order)
        assert torch.equal(v["inv"].long()[order], torch.arange(T * k, device="cuda"))
        counts = torch.bincount(idx.flatten().long(), minlength=E)
        assert torch.equal(v["count"].long(), counts) and torch.equal(v["offset"][1:].long(), counts.cumsum(0))
        total, size = torch.zeros(T, H, dtype=torch.float64, device="cuda"), torch.zeros(T, H, dtype=torch.float64, device="cuda")
        one = torch.full((T, E), -math.inf, device="cuda")
        for e in range(E):
            one[:, e] = 0.0
            y = moe.forward_gated(x, one, *args, 1).double()
            one[:, e] = -math.inf
            wb = (w.bfloat16().double() * (idx == e)).sum(1, keepdim=True)
            total += wb * y
            size += (wb * y).abs()
        tol = size * (2.0 ** -8 + (k + 4) * 2.0 ** -24) * (1 + 2.0 ** -8) + total.abs() * 2.0 ** -8
        assert torch.all((out.double() - total).abs() <= tol), float(((out.double() - total).abs() / tol).max())
