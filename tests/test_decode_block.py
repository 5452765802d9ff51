"""The decode step of one block (examples/decode_block.py): rotate_append,
paged_attention and forward_gated together, eager and as a CUDA graph."""
import importlib.util
import os

import pytest
import torch

import sparse_moe_layer_gb300 as moe

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = dict(H=256, I=256, E=8, top_k=2, q_heads=8, kv_heads=2, head_dim=64, page=8)
GATES = [dict(), dict(score="sigmoid", groups=4, top_groups=2, group_top=2, scale=2.5)]


@pytest.fixture(scope="module")
def example():
    moe.build()
    spec = importlib.util.spec_from_file_location("decode_block", os.path.join(ROOT, "examples", "decode_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 16])
def test_attention_half_against_64_bits(example, cache, window):
    """Attention over what the cache then holds: two roundings of bf16 (probabilities, output; fp16
    probabilities in an e4m3 cache are finer) and the fp32 score error, far below them here."""
    b = example.DecodeBlock(5, 37, 8, cache=cache, window=window, **SIZES)
    x = torch.randn(5, 256, device="cuda").bfloat16()
    for step in range(4):
        q, out = b.attention(x)
        n = 37 + step + 1
        assert b.lengths.tolist() == [n] * 5
        lo = max(0, n - window) if window else 0
        t = torch.arange(lo, n, device="cuda")
        pg, off = b.table[:, t // 8].long(), t % 8
        kv = []
        for c, s in ((b.k, b.ks), (b.v, b.vs)):
            y = c[pg, :, off].double() if cache == "bf16" else (c[pg, :, off].view(torch.float8_e4m3fn).double()
                                                                * s[pg, :, off].double()[..., None])
            kv.append(y.permute(0, 2, 1, 3).repeat_interleave(4, 1))
        a = (q.double()[:, :, None] @ kv[0].transpose(2, 3)) * 64 ** -0.5
        p = torch.softmax(torch.cat((a, b.sinks.double().view(1, 8, 1, 1).expand(5, 8, 1, 1)), -1), -1)[..., :-1]
        want = (p @ kv[1])[:, :, 0]
        tol = (p @ kv[1].abs())[:, :, 0] * 2.0 ** -8 * 1.02 + want.abs() * 2.0 ** -8
        assert torch.all((out.double() - want).abs() <= tol)
    assert moe.read_device_status(b.status) == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("gate", GATES, ids=["softmax", "sigmoid_groups"])
def test_graphed_steps_equal_eager_steps(example, cache, gate):
    a = example.DecodeBlock(6, 100, 8, cache=cache, gate=gate, **SIZES)
    b = example.DecodeBlock(6, 100, 8, cache=cache, gate=gate, **SIZES)
    x = torch.randn(6, 256, device="cuda").bfloat16()
    static, out, graph = b.graphed(x)
    assert b.lengths.tolist() == [100] * 6
    for _ in range(5):
        want = a.step(x)
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.all(torch.isfinite(want))
        assert torch.equal(a.k, b.k) and torch.equal(a.lengths, b.lengths)
        x = example.norm(want)
    for blk in (a, b):
        assert moe.read_device_status(blk.status) == 0 and moe.read_device_status(blk.moe_ws) == 0


def test_command(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["decode_block.py", "--batch", "3", "--context", "70", "--steps", "2"])
    example.main()
    assert "tokens/s" in capsys.readouterr().out
