"""Rotation by positions with several axes where one row stands for all of them, as for tokens of text: positions
[N] expanded to [A, N]; the same as that row written out, and as the one-axis call, bit for bit."""
import pytest
import torch

import sparse_moe_layer_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 2, 300])
@pytest.mark.parametrize("A", [1, 3, 16])
def test_expanded_positions(N, A):
    moe.build()
    g = torch.Generator(device="cuda").manual_seed(N)
    qkv = torch.randn(N, 12, 64, generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 1 << 20, (N,), generator=g, device="cuda")
    slots = torch.randperm(320, generator=g, device="cuda")[:N]
    freq = 1e6 ** -torch.arange(32, dtype=torch.float64, device="cuda").div(32)
    axes = torch.arange(32, dtype=torch.int32, device="cuda") % A

    def run(positions, **kw):
        kv = [torch.zeros(20, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        return [moe.rotate_append(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], positions, slots, *kv, freq, **kw), *kv]

    want = run(pos)
    for positions in (pos.expand(A, N), pos.repeat(A, 1), pos[None].expand(A, -1)):
        assert all(torch.equal(x, y) for x, y in zip(run(positions, axes=axes), want))
