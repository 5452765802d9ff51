"""Scales of an e4m3 cache that its own quantiser does not write, in paged attention: value = code *
scale for scales of either sign."""
import math

import pytest
import torch

import sparse_moe_layer_gb300 as moe
from test_paged_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


@pytest.mark.parametrize("D", [48, 64, 128, 256])
@pytest.mark.parametrize("lengths", [[1, 0, 40, 200], [3000], [150] * 90], ids=["team", "runs", "rows"])
def test_negative_scales(D, lengths):
    for negative in ("k", "v", "both", "some"):
        c = Case(lengths, 8, 2, D, cache="e4m3", seed=D)
        for i, s in enumerate(c.sc):
            if negative in ("both", "kv"[i]):
                s.neg_()
            elif negative == "some":
                s[:, :, ::3] *= -1.0
        c.both(sinks=True)
