"""Completions that share their prompts' pages, built from the package's cache
operators: room for a step's tokens, head norms with rotation into the pages
(bf16 or 4 bits), attention, forks of a prompt, pages given back, compaction.

The pool's state stays on the device and every step keeps its shapes, so a step
can be captured in a CUDA graph.  The dense projections around the attention are
plain matrix products.

    python examples/shared_prompts.py
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
    H: int = 4096          # model width
    Hq: int = 32           # query heads
    Hkv: int = 8           # key-value heads
    D: int = 128           # columns of a head
    page: int = 64         # keys per page
    pages: int = 4096      # pages of the pool
    rows: int = 64         # sequences at a time
    longest: int = 8192    # keys of a sequence
    fp4: bool = True       # 4-bit cache
    theta: float = 10000.0


class Attention:
    """The attention of one block for `rows` sequences, some of them idle."""

    def __init__(self, z: Sizes, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.z = z
        self.w_qkv = (rand(z.H, (z.Hq + 2 * z.Hkv) * z.D) * z.H ** -0.5).bfloat16()
        self.w_o = (rand(z.Hq * z.D, z.H) * (z.Hq * z.D) ** -0.5).bfloat16()
        self.q_weight, self.k_weight = ((1 + 0.1 * rand(z.D)).bfloat16() for _ in range(2))
        self.inv_freq = torch.tensor([z.theta ** (-2 * i / z.D) for i in range(z.D // 2)], dtype=torch.float32, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((z.rows, -(-z.longest // z.page)), -1, **i32)
        self.lens, self.refs = torch.zeros(z.rows, **i32), torch.zeros(z.pages, **i32)
        self.all = torch.arange(z.rows, **i32)
        if z.fp4:
            self.cache = mk.fp4_cache(z.pages, z.page, z.Hkv, z.D)
        else:
            kv = torch.zeros((2, z.pages, z.page, z.Hkv, z.D), dtype=torch.bfloat16, device="cuda")
            self.cache = dict(k_cache=kv[0], v_cache=kv[1])

    def step(self, x, live):
        """One token x[row] of each sequence; ``live[row]`` 1, or 0 for an idle row,
        whose output is zeros if it holds nothing."""
        z = self.z
        positions = self.lens.clone()
        slots = mk.extend_sequences(self.table, self.lens, self.refs, self.all, live, 1, list(self.cache.values()), z.page,
                                    check=False)
        qkv = x @ self.w_qkv
        q, k, v = (t.unflatten(1, (-1, z.D)) for t in qkv.split([z.Hq * z.D, z.Hkv * z.D, z.Hkv * z.D], 1))
        o = mk.qk_norm_rope(q, k, positions, self.inv_freq, q_weight=self.q_weight, k_weight=self.k_weight, v=v,
                            slots=slots.view(-1), check=False, **self.cache)
        attention = mk.paged_attention_fp4 if z.fp4 else mk.paged_attention
        a = attention(o["q"], block_table=self.table, seq_lens=self.lens, check=False, **self.cache)
        return a["out"].view(z.rows, z.Hq * z.D) @ self.w_o

    def fork(self, parents, children):
        mk.fork_sequences(self.table, self.lens, self.refs, parents, children, self.z.page, check=False)

    def free(self, rows):
        mk.free_sequences(self.table, self.lens, self.refs, rows, self.z.page, check=False)

    def compact(self):
        mk.compact_pages(self.table, self.lens, self.refs, list(self.cache.values()), self.z.page, table_out=self.table,
                         refs_out=self.refs, check=False)


def main():
    z, prompts, steps = Sizes(), 8, 32
    i32 = dict(dtype=torch.int32, device="cuda")
    for z.fp4 in (False, True):
        att = Attention(z)
        live = (torch.arange(z.rows, device="cuda") < prompts).to(torch.int32)
        x = torch.randn(z.rows, z.H, device="cuda").bfloat16()
        for _ in range(100):  # the prompts, a token at a time
            att.step(x, live)
        children = torch.arange(prompts, z.rows, **i32)
        att.fork(children % prompts, children)
        live.fill_(1)
        att.step(x, live)  # every child writes: the prompts' last pages are copied
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            att.step(x, live)  # allocates what the library keeps for this stream
            stream.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                att.step(x, live)
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(steps):
            graph.replay()
        b.record()
        torch.cuda.synchronize()
        held = int((att.refs > 0).sum())
        att.free(torch.arange(0, z.rows, 2, **i32))
        att.compact()
        if mk.mk_get_status() != mk.MK_OK:
            raise SystemExit("a kernel reported an error")
        print(f"{z.rows} completions of {prompts} prompts, {'4-bit' if z.fp4 else 'bf16'} cache: "
              f"{a.elapsed_time(b) * 1e3 / steps:.0f} us a step, {held} pages held, {int(att.lens.sum())} tokens left in "
              f"{int((att.refs > 0).sum())} pages after the compaction")


if __name__ == "__main__":
    main()
