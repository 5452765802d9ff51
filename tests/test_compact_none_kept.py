"""compact_drafts with no draft kept of any sequence: kept [B, 0], which moves nothing and returns the contexts."""
import pytest
import torch

import sparse_moe_layer_gb300 as moe
from test_cache_pages import Drafts, caches, clones, equal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,layers", [("bf16", 0), ("e4m3", 3)])
@pytest.mark.parametrize("view", [False, True])
def test_no_draft_is_kept(kind, layers, view):
    moe.build()
    d = Drafts([5, 0, 30], [8, 3, 0], [[], [], []], page=4)
    c = caches(layers, d.pages, 2, 4, 64, kind)
    got, status = clones(c), moe.new_status()
    kept = torch.zeros(3, 7, dtype=torch.int32, device="cuda")[:, :0] if view else d.kept_t.new_empty(3, 0)
    out = d.run(got, kept=kept, status=status)
    assert out.tolist() == [5, 0, 30] and moe.read_device_status(status) == 0
    equal(got, c)
    # a sequence that does not fit is reported all the same
    out = d.run(got, kept=kept, status=status, lens=torch.tensor([7, 3, 30], dtype=torch.int32, device="cuda"))
    assert out.tolist() == [7, 0, 30] and moe.read_device_status(status) == 6
    equal(got, c)
