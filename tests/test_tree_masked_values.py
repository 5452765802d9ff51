"""Attention of drafted tokens where values (or their scales) of tokens that only some of a sequence's drafts see are
infinite or NaN: drafts of other branches, context tokens at a window's edge.  The drafts that do not see them get what
the formula gives; those that do, a result that is not finite in just these dims.

Tolerance: that of tests/test_tree_attention.py."""
import math

import pytest
import torch

import sparse_moe_layer_gb300 as moe
from test_tree_attention import Case

pytestmark = pytest.mark.gpu
BAD = (math.nan, math.inf, -math.inf)


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


def spoil(c, places, dims):
    """Values of tokens (b, t) become NaN, inf, -inf in turn in `dims` of all heads; e4m3: NaN codes."""
    for i, (b, t) in enumerate(places):
        pg, off = c.place(b, t)
        if c.cache == "e4m3":
            c.kv[1][pg, :, off, dims] = 0x7F if i % 2 else 0xFF
        else:
            c.kv[1][pg, :, off, dims] = BAD[i % 3]


def check(c, out, places, dims, window):
    """c has bad values in `dims` of `places`; afterwards 0."""
    for b, t in places:
        pg, off = c.place(b, t)
        c.kv[1][pg, :, off, dims] = 0
    good, out = c.run(True, window), out.clone()
    for b, n in enumerate(c.drafts):
        lo, see = int(c.starts[b]), c.seen(b, window)
        hit = torch.zeros(n, dtype=torch.bool, device="cuda")
        for at, t in places:
            if at == b:
                hit |= see[:, t]
        assert bool(hit.any()) and bool((~hit).any()) or not any(at == b for at, _ in places), b
        rows = lo + hit.nonzero()[:, 0]
        for d in dims:
            assert not torch.any(torch.isfinite(out[rows, :, d])), (b, d)
            out[rows, :, d] = good[rows, :, d]
    c.check(out, True, window)


CASES = [(8, 2, 64, 16, "bf16", "bf16"), (64, 8, 64, 16, "bf16", "bf16"), (8, 2, 64, 7, "fp16", "fp16"), (32, 2, 128, 24, "fp16", "fp16"),
         (6, 2, 256, 8, "bf16", "bf16"), (8, 8, 80, 16, "bf16", "e4m3"), (16, 2, 64, 16, "fp16", "e4m3"), (24, 2, 128, 7, "bf16", "e4m3"),
         (4, 1, 192, 32, "fp16", "e4m3")]


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype,cache", CASES)
@pytest.mark.parametrize("contexts,drafts", [([33, 100], [12, 70]), ([3000, 0, 700], [9, 40, 256]), ([64, 5], [3, 2])])
def test_values_of_other_branches(Hq, Hkv, D, page, dtype, cache, contexts, drafts):
    c = Case(contexts, drafts, Hq, Hkv, D, page, dtype, cache, kind="binary", seed=sum(drafts))
    dims = [0, 3, 9, D - 1]
    places = [(b, contexts[b] + j) for b, n in enumerate(drafts) for j in sorted({1, n // 2, n - 1}) if 0 < j < n]
    spoil(c, places, dims)
    status = moe.new_status()
    out = c.run(True, status=status)
    assert moe.read_device_status(status) == 0
    assert torch.equal(c.run(True).view(torch.int16), out.view(torch.int16))
    check(c, out, places, dims, 0)


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype,cache", CASES)
@pytest.mark.parametrize("kind", ["chain", "none", "binary"])
@pytest.mark.parametrize("window", [7, 40, 150])
def test_values_at_a_windows_edge(Hq, Hkv, D, page, dtype, cache, kind, window):
    contexts, drafts = [200, 1000, 160], [6, 5, 30]
    c = Case(contexts, drafts, Hq, Hkv, D, page, dtype, cache, kind=kind, seed=window)
    dims = list(range(D))
    # the first token that the first draft sees; and a draft, which late ones have passed or early ones not reached
    places = [(b, n - window + 1) for b, n in enumerate(contexts)] + [(2, contexts[2] + 9)]
    spoil(c, places, dims)
    check(c, c.run(True, window), places, dims, window)


@pytest.mark.parametrize("scale", [0.0, -0.3])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_scales(scale, cache):
    c = Case([40, 900], [7, 30], 8, 2, 64, cache=cache, kind="binary", seed=1)
    spoil(c, [(0, 42), (1, 910)], [5])
    out = c.run(True, scale=scale)
    for b, t in ((0, 42), (1, 910)):
        pg, off = c.place(b, t)
        c.kv[1][pg, :, off, 5] = 0
        rows = int(c.starts[b]) + c.seen(b, 0)[:, t].nonzero()[:, 0]
        assert not torch.any(torch.isfinite(out[rows, :, 5]))
        out[rows, :, 5] = c.run(True, scale=scale)[rows, :, 5]
    c.check(out, True, scale=scale)


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 64, 16), (64, 8, 64, 16), (16, 1, 128, 7), (8, 1, 256, 16), (10, 1, 64, 7)])
@pytest.mark.parametrize("bad", BAD)
def test_value_scales_of_other_branches(Hq, Hkv, D, page, bad):
    c = Case([33, 700], [12, 70], Hq, Hkv, D, page, "bf16", "e4m3", kind="binary", seed=3)
    places = [(0, 33 + 3), (1, 700 + 2), (1, 700 + 40)]
    keep = [x.clone() for x in c.sc]
    for b, t in places:
        pg, off = c.place(b, t)
        c.sc[1][pg, :, off] = bad
    out = c.run(True)
    c.sc = keep
    good = c.run(True)
    for b, n in enumerate(c.drafts):
        hit = torch.zeros(n, dtype=torch.bool, device="cuda")
        for at, t in places:
            if at == b:
                hit |= c.seen(b, 0)[:, t]
        rows = int(c.starts[b]) + hit.nonzero()[:, 0]
        assert not torch.any(torch.isfinite(out[rows])) and 0 < len(rows) < n
        out[rows] = good[rows]
    c.check(out, True)


@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("t", [100, 290, 299])
def test_values_that_all_see(cache, window, page, t):
    """Context tokens, far from the drafts and in a tile with them, beside a draft's: no row is spared the first, and no
    other sequence touched."""
    c = Case([90, 300, 64], [5, 20, 7], 8, 2, 64, page, "fp16" if cache == "fp16" else "bf16", cache, kind="binary", seed=2)
    clean = c.run(True, window)
    spoil(c, [(1, t)], [2])
    spoil(c, [(1, 300 + 7)], [40])
    out = c.run(True, window)
    see = c.seen(1, window)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[5:25, :, 2] = see[:, t][:, None]
    hit[5:25, :, 40] = see[:, 307][:, None]
    assert bool(hit[5:25, 0, 2].all()) == (window == 0 or t > 100)
    assert torch.equal(out[:5], clean[:5]) and torch.equal(out[25:], clean[25:])
    assert not torch.any(torch.isfinite(out[hit])) and torch.all(torch.isfinite(out[~hit]))
    for x, d in ((t, 2), (307, 40)):
        pg, off = c.place(1, x)
        c.kv[1][pg, :, off, d] = 0
    c.check(torch.where(hit, c.run(True, window), out), True, window)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_out_may_be_q(cache):
    """In place (no row is computed anew then): the same, without bad values."""
    c = Case([90, 300, 64], [5, 20, 7], 8, 2, 64, cache=cache, seed=2)
    want, q = c.run(True), c.q.clone()
    assert torch.equal(c.run(True, q=q, out=q), want)
