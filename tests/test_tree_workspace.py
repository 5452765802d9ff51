"""A workspace for tree_attention made for N drafts of B sequences serves every call of at most so many drafts,
sequences and tokens, with windows or without."""
import pytest
import torch

import sparse_moe_layer_gb300 as moe
from test_tree_attention import Case

NB = [(1, 1), (6, 1), (16, 1), (17, 1), (64, 1), (64, 4), (256, 1), (256, 64), (512, 8), (512, 64), (2000, 40), (2000, 2000)]


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (4, 4), (256, 1), (4096, 1)])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 192, 256])
def test_a_size_serves_smaller_calls(Hq, Hkv, D):
    size = moe.lib().moe_tree_attention_workspace_size
    for tokens in (100, 240, 241, 500, 752, 753, 100000):
        for N, B in NB:
            most = size(N, B, Hq, Hkv, D, 0, tokens)
            assert most > 0
            for n, b in NB:
                for t in (100, 241, 500, 100000):
                    if n <= N and b <= B and t <= tokens:
                        assert size(n, b, Hq, Hkv, D, 0, t) <= most, (N, B, n, b, tokens, t)


# per sequence: contexts, drafts; the first is the largest call
CALLS = [([700] * 8, [32] * 8), ([700], [200]), ([700] * 8, [2] * 8), ([650, 3], [256, 0]), ([100] * 3, [5, 80, 9]), ([40], [1])]


@pytest.mark.gpu
@pytest.mark.parametrize("D,cache", [(64, "bf16"), (128, "bf16"), (64, "e4m3"), (128, "fp16"), (256, "bf16")])
@pytest.mark.parametrize("page", [16, 7])
def test_one_workspace_for_calls_of_many_sizes(D, cache, page):
    most = max(max(a + b for a, b in zip(*call)) for call in CALLS) + page
    ws = moe.tree_attention_workspace(256, 8, 16, 2, D, most)
    for i, (contexts, drafts) in enumerate(CALLS):
        c = Case(contexts, drafts, 16, 2, D, page, "fp16" if cache == "fp16" else "bf16", cache, seed=i)
        for window in (0, 300):
            out = c.run(True, window, workspace=ws.fill_(255))
            c.check(out, True, window)
            assert torch.equal(out, c.run(True, window))
