"""Expert choice from router logits (moe_route_experts) and the layer fed by it
(moe_forward_gated): refusals on the CPU, then on the GPU the choice against the
formula in 64 bits, row by row, where it can go wrong: odd expert counts, ties,
borders closer than fp32 resolves, masked logits, strided rows, every group
rule; and the gated layer against sums of its experts' own outputs.

Weight tolerance, counted in half-steps of fp32 (2^-24, relative to the weight):
exp of a rounded difference x - m costs |x - m| + 4 (two steps of the function),
the sum over at most 256 scores 13 additions of values >= 0, its own terms the
same |x - m| + 4, reciprocal, products, renormalising sum and division 8 more:
2 (|x - m| + 4) + 13 + 8 < 32 + 2 |x - m|.  Sigmoid and the chosen-only softmax
stay below that."""
import ctypes
import math

import numpy as np
import pytest
import torch

import sparse_moe_layer_gb300 as moe

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


def choose(l, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0):
    """One row (float64 logits) by the formula: (ascending indices, weights)."""
    E = len(l)
    if score == "softmax":
        m = l.max()
        s = np.exp(l - m) / np.exp(l - m).sum() if m > -np.inf else np.zeros(E)
    else:
        s = 1.0 / (1.0 + np.exp(-np.maximum(l, -700.0)))
    c = s + bias if bias is not None else s
    rank = c if bias is not None else l  # scores order like logits
    open_ = np.ones(E, bool)
    if groups > 1:
        gs = E // groups
        if group_top == 1:
            best = rank.reshape(groups, gs).max(1)
        else:
            best = np.sort(c.reshape(groups, gs), axis=1)[:, -2:].sum(1)
        order = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
        open_ = np.isin(np.arange(E) // gs, order)
    order = sorted(np.nonzero(open_)[0], key=lambda e: (-rank[e], e))[:k]
    idx = np.array(sorted(order))
    w = s[idx]
    if renormalize:
        w = w / (w.sum() + 1e-20)
    return idx, w * scale


def check(logits, k, **kw):
    idx, w = moe.route_experts(logits, k, **kw)
    torch.cuda.synchronize()
    assert idx.dtype == torch.int32 and w.dtype == torch.float32 and idx.shape == w.shape == (logits.shape[0], k)
    l = logits.double().cpu().numpy()
    l = np.where(np.isnan(l), -np.inf, l)
    ref = dict(kw)
    if ref.get("bias") is not None:
        ref["bias"] = ref["bias"].double().cpu().numpy()
    got_i, got_w = idx.cpu().numpy(), w.double().cpu().numpy()
    for t in range(len(l)):
        ri, rw = choose(l[t], k, **ref)
        assert np.array_equal(got_i[t], ri), (t, got_i[t], ri)
        spread = l[t].max() - l[t][ri]
        spread = np.where(np.isfinite(spread), spread, 0.0)
        tol = rw * (32 + 2 * spread) * 2.0 ** -24 + 2.0 ** -126
        if kw.get("renormalize", True):  # the sum's error is that of its terms
            tol = tol + rw * (32 + 2 * min(spread.max(), 40.0)) * 2.0 ** -24
        assert np.all(np.abs(got_w[t] - rw) <= tol), (t, got_w[t], rw)


# ------------------------------------------------------------- on the CPU ----
def test_refusals_on_the_host():
    L = moe.lib()

    def call(E=8, k=2, T=4, ld=None, dt=2, score=0, groups=1, top_groups=1, group_top=1, scale=1.0, logits=16, bias=None,
             idx=16, w=16, gate=True):
        g = moe._Gate(score, groups, top_groups, group_top, 1, scale, bias)
        return L.moe_route_experts(ctypes.byref(g) if gate else None, logits, dt, E if ld is None else ld, T, E, k, idx,
                                   w, None)

    assert call(gate=False) == 1 and call(logits=None) == 1 and call(idx=None) == 1 and call(w=None) == 1
    assert call(T=0) == 1 and call(k=0) == 1 and call(k=9, E=16) == 1 and call(k=3, E=2) == 1 and call(E=257) == 1
    assert call(ld=7) == 1 and call(score=2) == 1 and call(score=-1) == 1
    assert call(groups=3) == 1 and call(groups=0) == 1 and call(groups=64, E=64) == 1
    assert call(groups=4, top_groups=5) == 1 and call(groups=4, top_groups=0) == 1
    assert call(groups=4, top_groups=2, group_top=3) == 1 and call(groups=8, top_groups=8, group_top=2) == 1
    assert call(groups=4, top_groups=1, k=3) == 1  # one open group of 2 experts cannot give 3
    assert call(scale=math.nan) == 1
    assert call(dt=3) == 2 and call(dt=7) == 2  # no e4m3 logits
    assert call(logits=18) == 2 and call(dt=0, logits=17) == 2 and call(bias=18) == 2  # misaligned
    g = moe._Gate(0, 1, 1, 1, 1, 1.0, None)
    fake = [256] * 6
    assert L.moe_forward_gated(ctypes.byref(g), None, 2, 8, 256, 0, *fake, 4, 256, 256, 8, 2, 256, 256, 1 << 30, None) == 1
    assert L.moe_forward_gated(ctypes.byref(g), 256, 2, 8, 256, 3, *fake, 4, 256, 256, 8, 2, 256, 256, 1 << 30, None) == 1
    assert L.moe_forward_gated(ctypes.byref(g), 256, 2, 8, None, 0, *fake, 4, 256, 256, 8, 2, 256, 256, 1 << 30, None) == 1
    assert L.moe_forward_gated(ctypes.byref(g), 256, 2, 8, 256, 0, *fake, 4, 256, 256, 8, 2, 256, 256, 16, None) == 3


def test_binding_refuses_host_tensors_and_bad_shapes():
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        moe.route_experts(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        moe.forward_gated(torch.zeros(4, 256), torch.zeros(4, 8), *[None] * 6, 2)


# ------------------------------------------------------------- on the GPU ----
gpu = pytest.mark.gpu


def draw(T, E, dtype="fp32", seed=0, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (spread * torch.randn((T, E), generator=g, device="cuda")).to(DT[dtype])


@gpu
@pytest.mark.parametrize("E", [1, 2, 7, 31, 32, 33, 64, 96, 128, 160, 255, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_every_expert_count(E, dtype):
    for T, k in ((1, 1), (9, min(E, 8)), (300, min(E, 3))):
        check(draw(T, E, dtype, seed=E + T), k)
        check(draw(T, E, dtype, seed=E), k, score="sigmoid", renormalize=False, scale=2.5)


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E,groups,top_groups,k", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 4, 1, 8), (96, 32, 5, 8),
                                                   (60, 5, 2, 7), (32, 1, 1, 4), (14, 7, 7, 8), (256, 2, 1, 8)])
def test_scores_groups_and_bias(score, renormalize, E, groups, top_groups, k):
    for bias in (None, 0.05 * torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda()):
        for group_top in (1, 2):
            check(draw(65, E, "fp32", seed=groups), k, score=score, bias=bias, groups=groups, top_groups=top_groups,
                  group_top=group_top, renormalize=renormalize, scale=1.25)


@gpu
def test_equal_logits_take_the_lowest_experts():
    for E in (8, 100, 256):
        l = torch.full((5, E), 0.75, device="cuda")
        idx, w = moe.route_experts(l, 8)
        assert idx.cpu().tolist() == [list(range(8))] * 5 and torch.all(w == 0.125)
        check(l, 8, bias=torch.full((E,), 0.1, device="cuda"))
    check(draw(400, 256, "bf16", spread=0.1), 8)  # a few dozen distinct values: ties in every row
    check(draw(400, 256, "bf16", spread=0.1), 8, score="sigmoid", bias=torch.zeros(256, device="cuda"), groups=8,
          top_groups=4, group_top=2)
    z = torch.zeros(3, 16, device="cuda")
    z[:, 1::2] = -0.0
    check(z, 4)


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_borders_below_fp32_resolution_follow_64_bits(score):
    """Biases that make every choice equal up to fp32 rounding: only the 64-bit sums tell them apart."""
    T, E = 64, 64
    l = draw(1, E, "fp32", seed=3).expand(T, E).contiguous()
    l += 1e-3 * draw(T, 1, seed=4)
    s = torch.softmax(l[0].double(), 0) if score == "softmax" else torch.sigmoid(l[0].double())
    bias = (1.5 - s).float()
    check(l, 8, score=score, bias=bias)
    check(l, 8, score=score, bias=bias, groups=8, top_groups=3, group_top=2)
    check(l, 4, score=score, bias=bias, groups=4, top_groups=2, group_top=1)
    mixed = l.clone()
    mixed[::2] += draw(T // 2, E, seed=5)
    check(mixed, 8, score=score, bias=bias)


@gpu
def test_logits_and_choices_apart_in_the_last_bits():
    """fp32 logits one step apart (0 to 40 steps, shuffled), in one binade, across two, negative, and
    around zero; the same as biases of equal scores, and as whole groups."""
    g = torch.Generator().manual_seed(2)
    for E in (16, 64, 160, 256):
        steps = torch.stack([torch.randperm(E, generator=g) % 41 for _ in range(40)])
        for base in (1.0, 2.0 - 2.0 ** -22, -3.0, 0.0):
            l = (base + steps.double() * 2.0 ** (-23 if base else -140)).float().cuda()
            check(l, 8)
            check(l, 8, groups=8, top_groups=5, group_top=1)
            check(l, 8, score="sigmoid", groups=8, top_groups=4, group_top=2)
            check(torch.zeros(3, E, device="cuda"), 8, score="sigmoid", bias=l[0], groups=4, top_groups=2, group_top=2)
            check(l, 8, score="sigmoid", bias=l[0])


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_logits(score):
    l = draw(12, 40, seed=7)
    l[0, :] = -math.inf  # nothing left
    l[1, 3:] = -math.inf  # fewer left than chosen
    l[2, ::2] = torch.finfo(torch.float32).min
    l[3, 5] = math.nan
    l[4, :] = math.nan
    l[5, 10:] = -math.inf
    check(l, 6, score=score)
    check(l, 6, score=score, renormalize=False)
    check(l, 6, score=score, bias=0.01 * draw(1, 40, seed=8)[0], groups=4, top_groups=2, group_top=2)
    idx, w = moe.route_experts(l, 6, score="softmax")
    assert idx[0].tolist() == [0, 1, 2, 3, 4, 5] and torch.all(w[0] == 0) and torch.all(torch.isfinite(w))
    h = l.half()
    check(h, 6, score=score)
    top = torch.zeros(2, 9, device="cuda")
    top[:, 4] = math.inf
    idx, w = moe.route_experts(top, 1, score=score)
    assert idx.flatten().tolist() == [4, 4] and torch.all(w == 1)


@gpu
def test_strided_and_misaligned_rows():
    for E, ld in ((64, 65), (64, 80), (33, 37), (128, 129), (256, 257)):
        for dtype in ("bf16", "fp32"):
            big = draw(31, ld, dtype, seed=ld)
            check(big[:, :E], 4)
            check(big[:, ld - E:], 4)
    empty = moe.route_experts(torch.empty(0, 8, device="cuda"), 2)
    assert empty[0].shape == (0, 2) and empty[1].shape == (0, 2)


@gpu
def test_large_batch_and_repeated_calls_agree():
    l, b = draw(5000, 256, seed=11), 0.05 * draw(1, 256, seed=12)[0]
    kw = dict(score="sigmoid", bias=b, groups=8, top_groups=4, group_top=2, scale=2.5)
    a = moe.route_experts(l, 8, **kw)
    c = moe.route_experts(l, 8, **kw)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    parts = [moe.route_experts(l[i:i + 1000], 8, **kw) for i in range(0, 5000, 1000)]
    assert torch.equal(a[0], torch.cat([p[0] for p in parts])) and torch.equal(a[1], torch.cat([p[1] for p in parts]))


@gpu
def test_inside_a_graph_and_on_another_stream():
    l = draw(130, 128, seed=1)
    want = moe.route_experts(l, 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = moe.route_experts(l, 4)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx, w = moe.route_experts(l, 4)
    l.copy_(draw(130, 128, seed=2))
    g.replay()
    want = moe.route_experts(l, 4)
    torch.cuda.synchronize()
    assert torch.equal(idx, want[0]) and torch.equal(w, want[1])


# ------------------------------------------------------------ gated layer ----


@gpu
@pytest.mark.parametrize("fmt", ["block128", "mxfp8", "mxfp4"])
def test_gated_layer_sums_its_experts(fmt):
    """Expert e alone (every other logit -inf) gives y_e; a gate's output is the sum of its
    weights (bf16) times those, to the two roundings of bf16 outputs (w y_e summed in fp32)."""
    import synth
    from harness import Layer
    L = Layer(synth.config("tiny"), mx=fmt == "mxfp8", fp4=fmt == "mxfp4").to_device()
    T, E, H = L.T, L.E, L.H
    weights = (L.d_w13, L.d_s13, L.d_b13, L.d_w2, L.d_s2, L.d_b2)
    y = torch.empty(E, T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        one = torch.full((T, E), -math.inf, device="cuda")
        one[:, e] = 0.0
        y[e] = moe.forward_gated(L.d_x, one, *weights, 1).double()
    l, b = draw(T, E, seed=9), 0.1 * draw(1, E, seed=10)[0]
    for kw, k in ((dict(), 2), (dict(score="sigmoid", bias=b, groups=4, top_groups=2, group_top=2, scale=2.5), 3),
                  (dict(renormalize=False, scale=4.0), 8)):
        ws = moe.new_workspace(T, H, L.I, E, k, mx=fmt != "block128")
        out = moe.forward_gated(L.d_x, l, *weights, k, workspace=ws, **kw)
        assert moe.read_device_status(ws) == 0
        idx, w = moe.route_experts(l, k, **kw)
        v = moe.workspace_views(ws, T, H, L.I, E, k, mx=fmt != "block128")
        assert torch.equal(v["topk_idx"], idx) and torch.equal(v["topk_w"], w)
        rows = torch.sort(idx.flatten().long(), stable=True).indices
        assert torch.equal(v["perm"].long(), rows)
        counts = torch.bincount(idx.flatten().long(), minlength=E)
        assert torch.equal(v["offset"][1:].long(), counts.cumsum(0))
        wb = w.bfloat16().double()
        terms = wb[..., None] * y.permute(1, 0, 2).gather(1, idx.long()[..., None].expand(-1, -1, H))
        # each y_e was rounded to bf16 (2^-8), the output too; fp32 sums add k 2^-24
        tol = terms.abs().sum(1) * (2.0 ** -8 + (k + 4) * 2.0 ** -24) * (1 + 2.0 ** -8) + terms.sum(1).abs() * 2.0 ** -8
        assert torch.all((out.double() - terms.sum(1)).abs() <= tol)


@gpu
def test_gated_layer_equals_the_layers_own_router():
    import synth
    from harness import Layer, check_output, torch_bf16_to_np
    L = Layer(synth.config("tiny")).to_device()
    own, views, _ = L.run_gpu()
    logits = L.d_x.double() @ L.d_rw.double().t() + L.d_rb.double()
    ws = moe.new_workspace(L.T, L.H, L.I, L.E, L.k)
    out = moe.forward_gated(L.d_x, logits.float(), L.d_w13, L.d_s13, L.d_b13, L.d_w2, L.d_s2, L.d_b2, L.k, workspace=ws)
    v = moe.workspace_views(ws, L.T, L.H, L.I, L.E, L.k)
    for name in ("topk_idx", "perm", "inv", "offset", "count", "tiles1", "tiles2", "xq"):
        assert torch.equal(v[name], views[name]), name
    check_output(torch_bf16_to_np(out), torch_bf16_to_np(own))
