"""Scales of an e4m3 cache in paged attention: value = code * scale, for scales of either sign and any
spread, heads of zeros (which the append stores with the scale 1), and large scales without weight.

Tolerance of out_d, from what is rounded, token by token (W = max_t p_t |vscale_t|, A = sum_t p_t |v_td|):
  scores   e_t = (D + 8) 2^-23 scale sum|q k_t| on p_t, in the numerator and in the sum
  weights  ex2, the accumulators' factors and the fp32 sums: (L + 64) 2^-22 A
  p to fp16   2^-11 A; below fp16's normals half its smallest step, 2^-25, where the row's largest
              weight is at least 2^5, times codes of at most 448:           2^-21 L W
              (rows whose weights are all below 2^-105: 2^-116)
  out      half a step, and half of the type's smallest (2^-134 bf16, 2^-25 fp16)"""
import math

import pytest
import torch

import sparse_moe_layer_gb300 as moe
from test_paged_attention import HALF, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


def check(c, out=None, sinks=False, window=0):
    out = c.run(sinks=sinks, window=window) if out is None else out
    G, scale = c.Hq // c.Hkv, c.D ** -0.5
    for b, n in enumerate(c.lengths):
        lo = max(0, n - window) if window else 0
        L = n - lo
        if L == 0:
            assert torch.all(out[b] == 0)
            continue
        k, v = c.values(0, b, lo, n), c.values(1, b, lo, n)
        t = torch.arange(lo, n, device="cuda")
        vs = c.sc[1][c.table[b].long()[t // c.page], :, t % c.page].double().abs().t()  # [Hkv, L]
        q = c.q[b].double().view(c.Hkv, G, c.D)
        s = (q @ k.transpose(1, 2)) * scale
        e = (c.D + 8) * 2.0 ** -23 * scale * (q.abs() @ k.abs().transpose(1, 2))
        if sinks:
            s = torch.cat((s, c.sinks.double().view(c.Hkv, G, 1)), -1)
        p = torch.softmax(s, -1)[..., :L]
        some = (v != 0).any(-1)  # heads of zeros have no weight
        want, A, W = p @ v, p @ v.abs(), (p * (vs * some)[:, None]).amax(-1, keepdim=True)
        tol = ((p * e) @ v.abs() + (p * e).sum(-1, keepdim=True) * A + A * ((L + 64) * 2.0 ** -22 + 2.0 ** -11)
               + 2.0 ** -21 * L * W + 2.0 ** -116 + want.abs() * HALF[c.dtype] + (2.0 ** -134 if c.dtype == "bf16" else 2.0 ** -25))
        err = (out[b].double().view(c.Hkv, G, c.D) - want).abs()
        assert torch.all(err <= tol), (b, float((err / tol).max()))


def tokens(c, b, which):
    """Pages and places of tokens of sequence b."""
    t = torch.as_tensor(which, device="cuda")
    return c.table[b].long()[t // c.page], t % c.page


def put(c, i, b, which, x):
    """Tokens of sequence b get the keys (0) or values (1) x [tokens, Hkv, D], quantised."""
    pg, off = tokens(c, b, which)
    s = x.abs().amax(-1) / 448.0
    s = torch.where(s == 0, torch.ones_like(s), s)
    c.kv[i][pg, :, off] = (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    c.sc[i][pg, :, off] = s


SHAPES = pytest.mark.parametrize("lengths", [[1, 0, 40, 200], [3000], [150] * 90], ids=["team", "runs", "rows"])


@pytest.mark.parametrize("D", [48, 64, 128, 256])
@SHAPES
def test_negative_scales(D, lengths):
    for negative in ("k", "v", "both", "some"):
        c = Case(lengths, 8, 2, D, cache="e4m3", seed=D)
        for i, s in enumerate(c.sc):
            if negative in ("both", "kv"[i]):
                s.neg_()
            elif negative == "some":
                s[:, :, ::3] *= -1.0
        c.both(sinks=True)
        check(c, sinks=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [48, 64, 128, 256])
@SHAPES
def test_zero_heads_among_small_values(lengths, D, dtype):
    """A head of zeros has the scale 1; the others' scales are far below it and keep their bits."""
    for std in (1e-2, 3e-3, 1e-3) + ((1e-6, 1e-20) if dtype == "bf16" else ()):
        for every in (0, 3, 32):
            c = Case(lengths, 8, 2, D, dtype=dtype, cache="e4m3", seed=D)
            c.sc[1].mul_(std)
            for b, n in enumerate(lengths):
                zero = [t for t in range(n) if (t % every == every - 1 if every else t == 0)]
                if zero:
                    put(c, 1, b, zero, torch.zeros(len(zero), 2, D, device="cuda"))
                    if every == 3:  # codes of -0 are zeros as well
                        pg, off = tokens(c, b, zero)
                        c.kv[1][pg, :, off] = 0x80
            check(c)
            check(c, sinks=True, window=100)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("first", [True, False])
def test_large_scales_without_weight(D, first):
    """A token whose score is far below the others' and whose value scale far above: from a weight that
    adds nothing to one that is the output."""
    for far, size in ((28.0, 2.0 ** 20), (28.0, 2.0 ** 36), (28.0, 2.0 ** 44), (60.0, 2.0 ** 60), (11.0, 2.0 ** 13)):
        c = Case([90, 700], 2, 2, D, cache="e4m3", seed=D)
        c.sc[0].mul_(0.05)
        for b, n in enumerate(c.lengths):
            at = [0 if first else n - 1]
            q = c.q[b].float()
            put(c, 0, b, at, (-q * (far * D ** 0.5 / q.square().sum(-1, keepdim=True)))[None])
            pg, off = tokens(c, b, at)
            c.sc[1][pg, :, off] *= size
        check(c)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rising", [True, False])
def test_scales_against_scores(D, rising):
    """Scores that rise (fall) by 2^80 along the sequence, value scales that fall (rise) as much: every
    token weighs alike, while the sum belongs to the last (first) ones."""
    n = 300
    c = Case([n], 2, 2, D, cache="e4m3", seed=D)
    q = c.q[0].float()
    s = torch.linspace(-28.0, 28.0, n, device="cuda") * (1 if rising else -1)
    put(c, 0, 0, list(range(n)), q[None] * (s[:, None] * D ** 0.5 / q.square().sum(-1))[..., None])
    pg, off = tokens(c, 0, list(range(n)))
    real = (c.q[0].double()[:, None] @ c.values(0, 0, 0, n).transpose(1, 2))[:, 0] * D ** -0.5  # [Hkv, n]
    c.sc[1][pg, :, off] *= torch.exp(-real).t().float()
    check(c)


@pytest.mark.parametrize("order", [1, -1])
def test_scales_of_all_sizes(order):
    c = Case([200, 70], 8, 2, 64, cache="e4m3")
    for b, n in enumerate(c.lengths):
        pg, off = tokens(c, b, list(range(n)))
        c.sc[1][pg, :, off] = (2.0 ** (torch.arange(n, device="cuda") * order % 121 - 60.0))[:, None].expand(n, 2)
    check(c, sinks=True)


def test_zero_values_appended_beside_small_ones():
    """The same through rotate_append: padding tokens of zeros in a cache of small values."""
    B, Hkv, D, page, n = 2, 2, 64, 16, 200
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn(B * n, 3 * Hkv, D, generator=g, device="cuda")
    qkv[:, 2 * Hkv:] *= 1e-3
    qkv[::5, 2 * Hkv:] = 0.0
    qkv = qkv.bfloat16()
    pages = B * -(-n // page)
    c = Case.__new__(Case)
    c.dtype, c.cache, c.Hq, c.Hkv, c.D, c.page, c.lengths = "bf16", "e4m3", Hkv, Hkv, D, page, [n] * B
    c.table = torch.arange(pages, dtype=torch.int32, device="cuda").view(B, -1)
    c.lens = torch.tensor(c.lengths, dtype=torch.int32, device="cuda")
    c.kv = [torch.full((pages, Hkv, page, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    c.sc = [torch.full((pages, Hkv, page), math.nan, device="cuda") for _ in range(2)]
    t = torch.arange(B * n, device="cuda")
    inv = (150000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    q = moe.rotate_append(qkv[:, :Hkv], qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:], t % n,
                          t // n * (pages // B * page) + t % n, *c.kv, inv, k_scale=c.sc[0], v_scale=c.sc[1])
    assert float(c.sc[1][0, 0, 0]) == 1.0
    c.q = q.view(B, n, Hkv, D)[:, -1].contiguous()
    check(c)
