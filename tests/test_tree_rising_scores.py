"""Attention of drafted tokens where a row's largest score rises by more than the sums' slack from one part of a
tile of tokens to the next (moe_tree_attention): what the sums are about moves several times within a tile, in the
accumulators and in probabilities that are there already; for one row tile and two, keys and values copied by TMA and
by threads, 16-bit and e4m3 caches, for e4m3 also by the value scales.

Tolerance: that of tests/test_tree_attention.py."""
import pytest
import torch

import sparse_moe_layer_gb300 as moe
from test_tree_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


def climbing(drafts, Hq, Hkv, D, page, cache, step, by):
    """Scores (or, by "values", value scales) that are equal over `step` tokens and then rise, by 9 to 18 powers of two
    for the rows' different queries, value scales by 9."""
    c = Case([330, 70], [drafts, 3], Hq, Hkv, D, page, "fp16" if cache == "fp16" else "bf16", cache, seed=drafts + page)
    g = torch.Generator(device="cuda").manual_seed(page)
    c.q.mul_(0.05)
    c.q[..., 0] = 1 + torch.rand(c.q.shape[:2], generator=g, device="cuda").to(c.q.dtype)
    for b, n in enumerate(c.lengths):
        t = torch.arange(n, device="cuda")
        level = torch.clamp(t // step, max=330 // step).float()
        pg, off = c.table[b, t // page].long(), t % page
        if by == "values":
            c.sc[1][pg, :, off] = 2.0 ** (9 * level[:, None] - 100)
        elif cache == "e4m3":
            codes = torch.zeros(n, Hkv, D, dtype=torch.uint8, device="cuda")
            codes[..., 0] = 0x38  # 1
            c.kv[0][pg, :, off] = codes
            c.sc[0][pg, :, off] = 6.5 * level[:, None]
        else:
            keys = torch.zeros(n, Hkv, D, device="cuda")
            keys[..., 0] = 6.5 * level[:, None]
            c.kv[0][pg, :, off] = keys.to(c.kv[0].dtype)
    return c


# drafts x heads of a key: 512 rows (two row tiles up to 128 dims), 80 (one), 24 (one; e4m3: four times)
@pytest.mark.parametrize("drafts,Hq,Hkv", [(64, 16, 2), (10, 16, 2), (6, 8, 2)])
@pytest.mark.parametrize("D", [64, 128, 192])
@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("cache,by", [("bf16", "scores"), ("fp16", "scores"), ("e4m3", "scores"), ("e4m3", "values")])
@pytest.mark.parametrize("step", [16, 32, 64])
def test_scores_that_rise_within_a_tile(drafts, Hq, Hkv, D, page, cache, by, step):
    c = climbing(drafts, Hq, Hkv, D, page, cache, step, by)
    out = c.run(True, scale=1.0)
    c.check(out, True, scale=1.0)
    for _ in range(3):
        assert torch.equal(c.run(True, scale=1.0), out)
