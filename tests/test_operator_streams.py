"""Operators given a stream that is not the current one: what they allocate belongs to that
stream, so that memory dropped early is not handed to work that runs before it."""
import pytest
import torch

import sparse_moe_layer_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


def calls():
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    logits = n(300, 32)
    q, k, v = n(300, 8, 64), n(300, 2, 64), n(300, 2, 64)
    cache = [n(400, 2, 16, 64), n(400, 2, 16, 64)]
    pos = torch.arange(300, device="cuda")
    freq = (1e4 ** -torch.arange(32, device="cuda", dtype=torch.float64).div(32))
    table = torch.arange(400, device="cuda", dtype=torch.int32).view(2, 200)
    lens = torch.tensor([3200, 1500], dtype=torch.int32, device="cuda")
    return {
        "route_experts": lambda s: moe.route_experts(logits, 4, stream=s)[1],
        "rotate_append": lambda s: moe.rotate_append(q, k, v, pos, pos, *[c.clone() for c in cache], freq, stream=s),
        "paged_attention": lambda s: moe.paged_attention(q[:2], *cache, table, lens, 0.125, stream=s),
    }


@pytest.mark.parametrize("name", ["route_experts", "rotate_append", "paged_attention"])
def test_dropped_results_are_not_written_over_other_memory(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    want = call(None)
    call(side)  # first use of the stream
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # ~10 ms: the call is still waiting when its result is dropped
    got = call(side)
    shape, dtype = got.shape, got.dtype
    del got
    mine = [torch.full(shape, 7.0, dtype=dtype, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.all(m == 7.0) for m in mine)
    got = call(side)
    side.synchronize()
    assert torch.equal(got, want)
