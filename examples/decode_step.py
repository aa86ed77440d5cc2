"""One decode step of a mixture-of-experts block, built from the package's
operators: norm, paged attention over the cached keys and the new one, norm
with an 8-bit copy, router, the whole expert layer.

The dense projections around them (queries, keys and values, output, router)
are plain matrix products.  A step changes the cache in place and keeps all of
its shapes, so it can be captured in a CUDA graph once and replayed; the first
call outside of a capture allocates the library's workspaces.

    python examples/decode_step.py
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_token_dispatch_persistent_gb300 as mk  # noqa: E402


@dataclass
class Sizes:
    H: int = 4096        # model width
    Hq: int = 32         # query heads
    Hkv: int = 8         # key-value heads
    D: int = 128         # columns of a head
    F: int = 1536        # width of an expert
    E: int = 128         # experts
    k: int = 8           # experts per token
    page: int = 64       # keys per page
    fp8: bool = True     # 8-bit experts


def quantize_blocks(w):
    """e4m3 weights and a scale per 128 x 128 block of w[E,rows,cols]."""
    E, r, c = w.shape
    g = w.view(E, r // 128, 128, c // 128, 128)
    s = g.abs().amax((2, 4)).clamp(min=1e-30) / 448
    return (g / s[:, :, None, :, None]).view(E, r, c).to(torch.float8_e4m3fn), s


class Block:
    def __init__(self, z: Sizes, batch: int, max_len: int, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.z, self.batch = z, batch
        self.w_in, self.w_post = ((1 + 0.1 * rand(z.H)).bfloat16() for _ in range(2))
        self.w_qkv = (rand(z.H, (z.Hq + 2 * z.Hkv) * z.D) * z.H ** -0.5).bfloat16()
        self.w_o = (rand(z.Hq * z.D, z.H) * (z.Hq * z.D) ** -0.5).bfloat16()
        self.w_router = rand(z.H, z.E) * z.H ** -0.5
        self.experts = {}
        for name, r, c in (("W1", z.H, z.F), ("W3", z.H, z.F), ("W2", z.F, z.H)):
            w = rand(z.E, r, c) * r ** -0.5
            if z.fp8:
                self.experts[name], self.experts[name + "_scale"] = quantize_blocks(w)
            else:
                self.experts[name] = w.bfloat16()
        per = -(-max_len // z.page)
        self.cache = torch.zeros((batch * per, 2, z.page, z.Hkv, z.D), dtype=torch.bfloat16, device="cuda")
        order = torch.randperm(batch * per, generator=gen, device="cuda")
        self.table = order.view(batch, per).to(torch.int32).contiguous()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def step(self, x, residual):
        """x [batch,H] bf16, the block's input, joins the residual stream;
        returns the block's output and the new stream."""
        z, B = self.z, self.batch
        o = mk.add_rmsnorm(x, self.w_in, residual=residual, check=False)
        stream = o["residual"]
        qkv = o["out"] @ self.w_qkv
        q = qkv[:, :z.Hq * z.D].unflatten(1, (z.Hq, z.D))
        kv = qkv[:, z.Hq * z.D:].unflatten(1, (2, z.Hkv, z.D))
        at = self.lens.long()
        self.cache[torch.gather(self.table, 1, (at // z.page)[:, None])[:, 0].long(), :, at % z.page] = kv
        self.lens += 1
        a = mk.paged_attention(q, self.cache[:, 0], self.cache[:, 1], self.table, self.lens, check=False)
        y = a["out"].view(B, z.Hq * z.D) @ self.w_o
        o = mk.add_rmsnorm(y, self.w_post, residual=stream, e4m3=z.fp8, check=False)
        logits = o["out"].float() @ self.w_router
        xe, scale = (o["out8"], {"x_scale": o["scale"]}) if z.fp8 else (o["out"], {})
        e = mk.moe_ffn_decode(xe, logits, k=z.k, check=False, **self.experts, **scale)
        return e["out"], o["residual"]


def capture(block, x, residual):
    """The step as a CUDA graph over fixed x and residual; returns the graph and its outputs."""
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        lens = block.lens.clone()
        block.step(x, residual)  # allocates what the library keeps for this stream
        block.lens.copy_(lens)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = block.step(x, residual)
    torch.cuda.current_stream().wait_stream(stream)
    return graph, out


def main():
    z, batch, length, steps = Sizes(), 32, 4096, 50
    block = Block(z, batch, length + 2 * steps)
    block.cache.normal_()
    block.lens.fill_(length)
    x = torch.randn(batch, z.H, device="cuda").bfloat16()
    residual = torch.randn(batch, z.H, device="cuda").bfloat16()
    graph, _ = capture(block, x, residual)
    for _ in range(3):
        graph.replay()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(steps):
        graph.replay()
    b.record()
    torch.cuda.synchronize()
    if mk.mk_get_status() != mk.MK_OK:
        raise SystemExit("a kernel reported an error")
    us = a.elapsed_time(b) * 1e3 / steps
    print(f"{batch} sequences of {length} keys, {z.E} experts of {z.H} x {z.F} in 8 bits, top {z.k}: {us:.0f} us a step, "
          f"{batch / us * 1e6:.0f} tokens/s through the block")


if __name__ == "__main__":
    main()
