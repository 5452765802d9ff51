"""Sinks that are not numbers, and infinite ones: a NaN sink makes its head NaN (and no other), a sink
of +inf takes all of the weight (out 0), one of -inf none."""
import math

import pytest
import torch

import sparse_moe_layer_gb300 as moe
from test_paged_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("lengths", [[1, 40, 200], [6000], [150] * 90], ids=["team", "runs", "rows"])
def test_nan_and_infinite_sinks(lengths, dtype, cache):
    c = Case(lengths, 8, 2, 64, dtype=dtype, cache=cache)
    plain = c.run(sinks=True)
    c.sinks[1], c.sinks[4], c.sinks[6] = math.nan, math.inf, -math.inf
    out = c.run(sinks=True)
    assert torch.all(torch.isnan(out[:, 1])) and torch.all(out[:, 4] == 0)
    for h in (0, 2, 3, 5, 7):
        assert torch.equal(out[:, h], plain[:, h])
    assert torch.equal(out[:, 6], c.run()[:, 6])
