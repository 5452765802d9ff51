"""One decoder block's decode step on random weights: the sparse MoE layer behind
the operators that stand before it.

  x -> norm -> q, k, v -> rotate_append (paged cache) -> paged_attention -> + x
    -> norm -> router logits -> forward_gated (experts) -> + x

Norms and the dense projections are plain torch; the cache is bf16 or e4m3.  The
step runs as one CUDA graph: lengths, slots and positions live in device tensors
that advance inside it.

  python examples/decode_block.py [--batch 64] [--context 4096] [--steps 32] [--cache bf16|e4m3] [--window 0]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_moe_layer_gb300 as moe  # noqa: E402


def norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-5)).bfloat16()


def next_slots(table, at, page, num_pages):
    """Cache slots of tokens number `at` [B] of the sequences of a page table [B, pages].  A sequence whose
    pages are full gets the slot past the last page: rotate_append appends nothing and reports it."""
    column = (at // page).clamp(max=table.shape[1] - 1)
    slots = table.gather(1, column[:, None])[:, 0].long() * page + at % page
    return torch.where(at < table.shape[1] * page, slots, num_pages * page)


class DecodeBlock:
    """Weights, the paged cache of `batch` sequences of `context` tokens already in it, and the state of
    the next step.  There are pages for `room` tokens more (rounded up to whole pages); steps past them set
    `status`.  `gate`: keyword arguments of the expert choice (route_experts)."""

    def __init__(self, batch, context, room, H=2880, I=2880, E=32, top_k=4, q_heads=64, kv_heads=8, head_dim=64,
                 page=16, cache="bf16", window=0, gate=None, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=1.0):
            return std * torch.randn(shape, generator=g, device="cuda")

        self.B, self.Hq, self.Hkv, self.D, self.page = batch, q_heads, kv_heads, head_dim, page
        self.top_k, self.window, self.gate = top_k, window, gate or {}
        rows = (q_heads + 2 * kv_heads) * head_dim
        self.w_qkv = normal(H, rows, std=H ** -0.5).bfloat16()
        self.b_qkv = normal(rows, std=0.1).bfloat16()
        self.w_o = normal(q_heads * head_dim, H, std=(q_heads * head_dim) ** -0.5).bfloat16()
        self.sinks = normal(q_heads)
        self.w_router, self.b_router = normal(H, E, std=H ** -0.5), normal(E, std=0.1)
        self.experts = moe.pack_weights(normal(E, 2 * I, H, std=0.02), normal(E, H, I, std=0.02))
        self.b13, self.b2 = normal(E, 2 * I, std=0.1).bfloat16(), normal(E, H, std=0.1).bfloat16()
        self.inv_freq = 150000.0 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64, device="cuda") / head_dim)

        pages = -(-(context + room) // page)
        shape = (batch * pages, kv_heads, page)
        if cache == "e4m3":
            self.k, self.v = (torch.randint(0, 120, (*shape, head_dim), dtype=torch.uint8, device="cuda", generator=g)
                              for _ in range(2))
            self.ks, self.vs = (torch.full(shape, 2.0 ** -7, device="cuda") for _ in range(2))
        else:
            self.k, self.v = (normal(*shape, head_dim).bfloat16() for _ in range(2))
            self.ks = self.vs = None
        order = torch.randperm(batch * pages, generator=g, device="cuda")
        self.table = order.int().view(batch, pages)
        self.lengths = torch.full((batch,), context, dtype=torch.int32, device="cuda")
        most = window if 0 < window < pages * page else pages * page
        self.att_ws = moe.attention_workspace(batch, q_heads, kv_heads, head_dim, most, self.k.dtype)
        self.moe_ws = moe.new_workspace(batch, H, I, E, top_k)
        self.status = moe.new_status()

    def attention(self, x):
        """x [B, H] -> (rotated q, attention output before w_o); the batch's keys and values are appended."""
        B, Hq, Hkv, D = self.B, self.Hq, self.Hkv, self.D
        qkv = torch.addmm(self.b_qkv, norm(x), self.w_qkv).view(B, Hq + 2 * Hkv, D)
        at = self.lengths.long()
        slots = next_slots(self.table, at, self.page, self.k.shape[0])
        q = moe.rotate_append(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], at, slots, self.k, self.v, self.inv_freq,
                              k_scale=self.ks, v_scale=self.vs, status=self.status)
        self.lengths += 1
        return q, moe.paged_attention(q, self.k, self.v, self.table, self.lengths, D ** -0.5, k_scale=self.ks,
                                      v_scale=self.vs, sinks=self.sinks, window=self.window, workspace=self.att_ws,
                                      status=self.status)

    def mlp(self, x):
        y = norm(x)
        logits = torch.addmm(self.b_router, y.float(), self.w_router)
        w13, s13, w2, s2 = self.experts
        return moe.forward_gated(y, logits, w13, s13, self.b13, w2, s2, self.b2, self.top_k, workspace=self.moe_ws,
                                 **self.gate)

    def step(self, x):
        x = x + self.attention(x)[1].reshape(self.B, -1) @ self.w_o
        return x + self.mlp(x)

    def graphed(self, x):
        """A step captured once: returns (static input, static output, graph).  Capturing runs no step."""
        keep = self.lengths.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step(x)  # library handles and kernel attributes are set up outside the capture
        torch.cuda.current_stream().wait_stream(side)
        self.lengths.copy_(keep)
        static = x.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = self.step(static)
        return static, out, graph


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--context", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--cache", choices=["bf16", "e4m3"], default="bf16")
    ap.add_argument("--window", type=int, default=0)
    a = ap.parse_args()
    block = DecodeBlock(a.batch, a.context, a.steps + 2, cache=a.cache, window=a.window)
    x = torch.randn(a.batch, 2880, device="cuda").bfloat16()
    static, out, graph = block.graphed(x)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
        static.copy_(norm(out))  # the next step's input: here the block's own output, renormalised
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / a.steps
    for word in (block.status, block.moe_ws):
        if moe.read_device_status(word) != 0:
            raise SystemExit("a device error word is set")
    print(f"batch {a.batch}, context {a.context} + {a.steps}, {a.cache} cache, window {a.window}: {t * 1e6:.1f} us a step "
          f"of one block, {a.batch / t:.0f} tokens/s")


if __name__ == "__main__":
    main()
