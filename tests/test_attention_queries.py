"""Queries of a wide range over an e4m3 cache: the dims that matter lie far below the row's largest value.

One dim of each query is 2^range times the others, and the keys are 0 there; the keys' scales bring the
scores back to a few units.  Tolerance: that of the scores with exact queries, token by token
(e_t = (D + 8) 2^-23 scale sum|q k_t| on p_t, in the numerator and in the sum), weights in fp16
(2^-11 A, and 2^-21 L max_t p_t |vscale_t| below its normals), fp32 sums (L + 64) 2^-22 A, out half a step."""
import pytest
import torch

import sparse_moe_layer_gb300 as moe
from test_paged_attention import HALF, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()


@pytest.mark.parametrize("dtype,far", [("bf16", 10), ("bf16", 20), ("bf16", 27), ("bf16", -27), ("fp16", 14), ("fp16", 20)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_dims_beside_a_large_one(dtype, far, D):
    c = Case([5, 90, 1500], 8, 2, D, dtype=dtype, cache="e4m3", seed=D)
    small = 2.0 ** -(abs(far) // 2) if dtype == "fp16" else 2.0 ** (-far if far < 0 else -13)
    q = c.q.float() * small
    q[..., 3] = small * 2.0 ** abs(far)
    c.q = q.to(c.q.dtype)
    c.kv[0][..., 3] = 0
    c.sc[0].mul_(1.0 / small)
    out = c.run()
    for b, n in enumerate(c.lengths):
        k, v = c.values(0, b, 0, n), c.values(1, b, 0, n)
        t = torch.arange(n, device="cuda")
        vs = c.sc[1][c.table[b].long()[t // c.page], :, t % c.page].double().t()
        qb = c.q[b].double().view(2, 4, D)
        s = (qb @ k.transpose(1, 2)) * D ** -0.5
        e = (D + 8) * 2.0 ** -23 * D ** -0.5 * (qb.abs() @ k.abs().transpose(1, 2))
        p = torch.softmax(s, -1)
        want, A = p @ v, p @ v.abs()
        tol = ((p * e) @ v.abs() + (p * e).sum(-1, keepdim=True) * A + A * ((n + 64) * 2.0 ** -22 + 2.0 ** -11)
               + 2.0 ** -21 * n * (p * vs[:, None]).amax(-1, keepdim=True) + want.abs() * HALF[dtype] + 2.0 ** -25)
        err = (out[b].double().view(2, 4, D) - want).abs()
        assert torch.all(err <= tol), (b, float((err / tol).max()))
