"""Paged attention over one peak and a long flat tail: tokens each far below the peak that together
weigh as much, or carry values far larger.

Tolerance of out_d, token by token (A = sum_t p_t |v_td|, L tokens):
  scores   e_t = (D + 8) 2^-23 scale sum|q k_t| on p_t, in the numerator and in the sum
  weights  ex2 and the fp32 sums: (L + 64) 2^-22 A
  p to 16 bit   half a step of the product's type, 2^-8 bf16, 2^-11 fp16, of A, twice (16-bit caches sum
           the rounded); fp16 below its normals half its smallest step, 2^-25, where the largest is at
           least 2^7 (e4m3: with the value's scale, 2^5, codes up to 448):
                                  2^-32 (sum_t |v_td| + L A)      e4m3: 2^-21 L max_t p_t |vscale_t|
  out      half a step, and half of the type's smallest (2^-134 bf16, 2^-25 fp16)"""
import math

import pytest
import torch

import sparse_moe_layer_gb300 as moe
from test_paged_attention import DT, HALF, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


def put(c, i, x):
    """Keys (0) or values (1) x [n, Hkv, D] of the one sequence."""
    t = torch.arange(x.shape[0], device="cuda")
    pg, off = c.table[0].long()[t // c.page], t % c.page
    if c.cache != "e4m3":
        c.kv[i][pg, :, off] = x.to(DT[c.cache])
        return
    s = x.abs().amax(-1) / 448.0
    s = torch.where(s == 0, torch.ones_like(s), s)
    c.kv[i][pg, :, off] = (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    c.sc[i][pg, :, off] = s


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("fp16", "e4m3")])
@pytest.mark.parametrize("n", [900, 60000])
@pytest.mark.parametrize("bits", [16, 23, 25, 26, 28])
@pytest.mark.parametrize("D", [64, 128])
def test_tail(dtype, cache, n, bits, D):
    H = 2
    c = Case([n], H, H, D, page=64, dtype=dtype, cache=cache)
    g = torch.Generator(device="cuda").manual_seed(bits)
    q = c.q[0].float()
    k = torch.zeros(n, H, D, device="cuda")
    k[n // 3] = q * (bits * math.log(2.0) * D ** 0.5 / q.square().sum(-1, keepdim=True))
    v = 1.0 + 0.25 * torch.randn(n, H, D, generator=g, device="cuda")
    v[n // 3] = 2.0 ** -10 * torch.randn(H, D, generator=g, device="cuda")
    put(c, 0, k)
    put(c, 1, v)
    out = c.run()
    kd, vd = c.values(0, 0, 0, n), c.values(1, 0, 0, n)
    qd = c.q[0].double()[:, None]
    s = (qd @ kd.transpose(1, 2)) * D ** -0.5
    e = (D + 8) * 2.0 ** -23 * D ** -0.5 * (qd.abs() @ kd.abs().transpose(1, 2))
    p = torch.softmax(s, -1)
    want, A = p @ vd, p @ vd.abs()
    tol = ((p * e) @ vd.abs() + (p * e).sum(-1, keepdim=True) * A + A * (n + 64) * 2.0 ** -22
           + want.abs() * HALF[dtype] + (2.0 ** -134 if dtype == "bf16" else 2.0 ** -25))
    if cache == "e4m3":
        t = torch.arange(n, device="cuda")
        vs = c.sc[1][c.table[0].long()[t // c.page], :, t % c.page].double().t()
        tol = tol + A * 2.0 ** -11 + 2.0 ** -21 * n * (p * vs[:, None]).amax(-1, keepdim=True)
    else:
        tol = tol + 2 * A * HALF[cache]
        if cache == "fp16":
            tol = tol + 2.0 ** -32 * (vd.abs().sum(1, keepdim=True) + n * A)
    err = (out[0].double()[:, None] - want).abs()
    assert torch.all(err <= tol), float((err / tol).max())
