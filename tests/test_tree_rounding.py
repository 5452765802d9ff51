"""Attention of drafted tokens: probabilities that stand beside a tile's scores are rounded to 16 bits once, also where
the sums' reference moves between two parts of the tile and they are scaled (moe_tree_attention).

The inputs are made so that a second rounding would show.  Scores (16-bit caches) rise from 0 to just below 8 powers of
two, which moves nothing, and then past 8 within the same tile: the earlier part's probabilities are still as large as
the new ones.  e4m3: scores are 0; a value scale makes weights just below a half step above a power of two, and a far
larger scale in the tile's next part moves the reference to where they are so again.

Tolerance: that of tests/test_tree_attention.py, which counts one rounding of a probability and one of the output."""
import math

import pytest
import torch

import sparse_moe_layer_gb300 as moe
from test_tree_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


def fill(c, parts):
    """Tokens [lo, hi) of the one sequence get keys, values and scales: parts of (lo, hi, k, v, ks, vs), k and v [Hkv, D]
    in the cache's type, scales [Hkv] or None."""
    for lo, hi, *what in parts:
        t = torch.arange(lo, hi, device="cuda")
        pg, off = c.table[0, t // c.page].long(), t % c.page
        for to, x in zip((*c.kv, *c.sc), what):
            if x is not None:
                to[pg, :, off] = x


# tile: its tokens; part: those taken together.  Two row tiles by TMA (192 rows), one by threads (64 rows).
@pytest.mark.parametrize("page,drafts,tile,part", [(16, 3, 128, 64), (7, 1, 64, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B0", [8.0625, 8.125, 8.25, 9.0])
def test_scores_rise_past_the_slack_within_a_tile(page, drafts, tile, part, dtype, B0):
    Hkv, D = 16, 16
    c = Case([2 * tile], [drafts], 64 * Hkv, Hkv, D, page, dtype, kind="none")
    t = c.kv[0].dtype
    c.q.zero_()
    row = torch.arange(64 * Hkv, device="cuda") % 64
    for d in range(drafts):
        c.q[d, :, 0] = (1 + row / 64 + d / 128).to(t)
    zero = torch.zeros(Hkv, D, dtype=t, device="cuda")
    a, b, v = zero.clone(), zero.clone(), zero.clone()
    a[:, 0] = 4 + torch.arange(Hkv, device="cuda") / 4
    b[:, 0] = B0
    v[:] = 1 + torch.arange(D, device="cuda") / D
    fill(c, [(0, 2 * tile + drafts, zero, zero, None, None), (tile, tile + part, a, v, None, None),
             (tile + part, 2 * tile, b, zero, None, None)])
    c.check(c.run(scale=math.log(2)), scale=math.log(2))


# Two row tiles (144 rows), one whose rows are there once (96).
@pytest.mark.parametrize("drafts,tile", [(3, 128), (2, 64)])
@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("up", [2.0 ** 11, 2.0 ** 14])
def test_a_large_scale_moves_the_weights_reference_within_a_tile(drafts, tile, page, up):
    Hkv, D, part = 32, 16, 32
    c = Case([2 * tile], [drafts], 48 * Hkv, Hkv, D, page, "fp16", "e4m3", kind="none")
    more = 1 + 0.97 * 2.0 ** -11  # just below a half step of fp16
    s0 = 2.0 ** (torch.arange(Hkv, device="cuda") / Hkv)
    one = torch.ones(Hkv, device="cuda")
    zero = torch.zeros(Hkv, D, dtype=torch.uint8, device="cuda")
    v = (0x38 + torch.arange(D, device="cuda") % 8).byte().expand(Hkv, D)
    fill(c, [(0, 2 * tile + drafts, zero, zero, one, s0 * up / more), (0, tile, zero, zero, one, s0),
             (tile, tile + part, zero, v, one, s0 * 0.5 * more)])
    c.check(c.run())
