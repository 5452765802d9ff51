"""The decode block example past the end of its pages: the step reports it and stays inside its tensors."""
import importlib.util
import os

import pytest
import torch

import sparse_moe_layer_gb300 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = dict(H=256, I=256, E=8, top_k=2, q_heads=8, kv_heads=2, head_dim=64, page=8)


@pytest.fixture(scope="module")
def example():
    moe.build()
    spec = importlib.util.spec_from_file_location("decode_block", os.path.join(ROOT, "examples", "decode_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_slots_past_the_pages(example):
    """On the CPU: every token number up to far past the table's last column."""
    table = torch.tensor([[4, 2, 0], [1, 5, 3]], dtype=torch.int32)
    for n in range(200):
        slots = example.next_slots(table, torch.tensor([n, n + 1]), 8, 6)
        for b, t in enumerate((n, n + 1)):
            assert int(slots[b]) == (int(table[b, t // 8]) * 8 + t % 8 if t < 24 else 48)


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_steps_past_the_pages_set_the_status(example, cache):
    b = example.DecodeBlock(3, 13, 3, cache=cache, **SIZES)  # 16 places: three more tokens
    x = torch.randn(3, 256, device="cuda").bfloat16()
    static, out, graph = b.graphed(x)
    for _ in range(3):
        graph.replay()
    assert moe.read_device_status(b.status) == 0
    full = b.k.clone(), b.v.clone()
    for _ in range(20):
        graph.replay()
        assert moe.read_device_status(b.status) == 6
        assert torch.equal(b.k, full[0]) and torch.equal(b.v, full[1]) and torch.all(torch.isfinite(out))
    b.step(x)
    assert moe.read_device_status(b.status) == 6
