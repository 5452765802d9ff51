"""Attention of drafted tokens over a cache whose heads are expanded (a stride of 0): one key head that stands for
several, keys, values or both, with their scales; against the formula, and its last draft against the operator for one
token."""
import pytest
import torch

import sparse_moe_layer_gb300 as moe
from test_tree_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("which", ["keys", "values", "both"])
def test_one_head_stands_for_all(cache, D, page, which):
    c = Case([70, 300, 0], [5, 40, 1], 16, 4, D, page, "fp16" if cache == "fp16" else "bf16", cache, seed=D)
    for i in ((0,) if which == "keys" else (1,) if which == "values" else (0, 1)):
        c.kv[i] = c.kv[i][:, :1].expand(c.kv[i].shape)
    if cache == "e4m3" and which == "both":
        c.sc = [s[:, :1].expand(s.shape) for s in c.sc]
    out = c.run(True)
    c.check(out, True)
    one = moe.paged_attention(c.q[-1:], *c.kv, c.table[2:], c.lens[2:], D ** -0.5, k_scale=c.sc[0], v_scale=c.sc[1],
                              sinks=c.sinks)
    c.check(torch.cat((out[:-1], one)), True, only=[2])
