"""forward_gated takes the tensors of one device and runs on it."""
import pytest
import torch

import sparse_moe_layer_gb300 as moe


def test_tensors_of_a_call_share_a_device(monkeypatch):
    """On the CPU, with the meta device as the other one: each argument in turn."""
    cpu, other = torch.zeros(1), torch.zeros(1, device="meta")
    moe._same_device(cpu, x=cpu, bias=None, out=cpu)
    for name in ("x", "bias", "w13", "workspace"):
        with pytest.raises(ValueError, match=f"{name} is on another device"):
            moe._same_device(cpu, x0=cpu, **{name: other})


@pytest.mark.gpu
def test_every_argument_is_compared_and_the_device_is_set(monkeypatch):
    import synth
    from harness import Layer
    moe.build()
    L = Layer(synth.config("tiny")).to_device()
    names = ("w13", "s13", "b13", "w2", "s2", "b2")
    kw = dict(x=L.d_x, logits=torch.zeros(L.T, L.E, device="cuda"), top_k=2, bias=torch.zeros(L.E, device="cuda"),
              out=torch.empty(L.T, L.H, dtype=torch.bfloat16, device="cuda"),
              workspace=moe.new_workspace(L.T, L.H, L.I, L.E, 2), **{n: getattr(L, "d_" + n) for n in names})
    want = moe.forward_gated(**kw).clone()
    for name in ("x", "out", "workspace", *names):
        with pytest.raises(ValueError, match="another device"):
            moe.forward_gated(**{**kw, name: kw[name].cpu()})
    used = []
    guard = torch.cuda.device

    class Device(guard):
        def __init__(self, d):
            used.append(torch.device(d))
            super().__init__(d)

    monkeypatch.setattr(torch.cuda, "device", Device)
    assert torch.equal(moe.forward_gated(**kw), want) and L.d_x.device in used
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.forward_gated(**{**kw, "out": None, "workspace": None}, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
