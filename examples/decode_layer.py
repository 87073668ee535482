"""One decoder layer with 4-bit weights, token by token, on libwq alone.

    python examples/decode_layer.py [--batch 4] [--steps 64] [--prompt 500]

Random weights of a mixture-of-experts layer (hidden 4096, 32 query and 8 KV heads of 128,
eight experts of 14336, two for each token).  A prompt's keys and values are written to a paged
cache by the rotary append; then each step runs

    residual add and RMS norm, QKV product, rotary append, paged attention, output product,
    residual add and RMS norm, mixture-of-experts layer

for one new token per sequence, first call by call and then as one captured graph, and the two
are compared."""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from weight_only_quantized_gemm_amd import decode, torch_ops  # noqa: E402


def random_weight(g, k: int, n: int, group: int = 128) -> dict:
    """Random 4-bit codes with scales that keep a product's output near its input's size."""
    words = torch.randint(-2 ** 31, 2 ** 31, (k // 8, n), generator=g, device=g.device,
                          dtype=torch.int64).to(torch.int32)
    scales = (torch.rand((k // group, n), generator=g, device=g.device) + 0.5) / (4.6 * k ** 0.5)
    return dict(qweight=words, scales=scales.half(), group_size=group)


class DecoderLayer:
    """Weights, cache and plans of one layer for a fixed batch (at most 16 sequences)."""

    def __init__(self, g, batch: int, max_len: int, *, hidden: int = 4096, q_heads: int = 32,
                 kv_heads: int = 8, head_dim: int = 128, inter: int = 14336, experts: int = 8,
                 top_k: int = 2, page_size: int = 16):
        dev = g.device
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.page_size = page_size
        qkv = (q_heads + 2 * kv_heads) * head_dim

        def packed(k, n):
            w = random_weight(g, k, n)
            return torch_ops.PackedWeight(w["qweight"], w["scales"], device=dev)

        self.w_qkv, self.w_out = packed(hidden, qkv), packed(q_heads * head_dim, hidden)
        self.bufs = [torch_ops.GemmBuffers(w, batch, True) for w in (self.w_qkv, self.w_out)]
        self.norms = [torch.ones(hidden, dtype=torch.float16, device=dev) for _ in range(2)]
        gate_up = torch_ops.ExpertBank([dict(gate=random_weight(g, hidden, inter),
                                             up=random_weight(g, hidden, inter))
                                        for _ in range(experts)], device=dev)
        down = torch_ops.ExpertBank([random_weight(g, inter, hidden) for _ in range(experts)],
                                    device=dev)
        router = (torch.randn((experts, hidden), generator=g, device=dev) / hidden ** 0.5).half()
        self.moe = decode.MoELayer(gate_up, down, router, top_k, max_tokens=batch)

        pages = -(-max_len // page_size)
        self.cache = decode.PagedCache.empty(batch * pages, page_size, kv_heads, head_dim,
                                             torch.float16, dev)
        order = torch.randperm(batch * pages, generator=g, device=dev)
        self.table = order.view(batch, pages).to(torch.int32)
        self.attn = decode.PagedAttention(self.cache, batch, q_heads, max_len,
                                          dtype=torch.float16)
        half = head_dim // 2
        self.inv_freq = (500000.0 ** (-torch.arange(half, device=dev).double() / half)).float()
        self.lens = torch.zeros(batch, dtype=torch.int32, device=dev)

    def slots_of(self, sequence: torch.Tensor, position: torch.Tensor) -> torch.Tensor:
        page = self.table[sequence, position // self.page_size].long()
        return page * self.page_size + position % self.page_size

    def split(self, qkv: torch.Tensor):
        d = self.head_dim
        parts = qkv.split([self.q_heads * d, self.kv_heads * d, self.kv_heads * d], dim=1)
        return [x.unflatten(1, (-1, d)) for x in parts]

    def prompt(self, x: torch.Tensor, sequence: int) -> None:
        """Writes the keys and values of a prompt's layer inputs [tokens][hidden]."""
        y, _ = decode.add_rms_norm(x, self.norms[0])
        _, k, v = self.split(torch_ops.gemm(y, self.w_qkv))
        at = torch.arange(x.shape[0], device=x.device)
        decode.rope_append(None, k, v, self.cache, self.slots_of(sequence, at),
                           positions=at.to(torch.int32), inv_freq=self.inv_freq)
        self.lens[sequence] = x.shape[0]

    def step(self, x: torch.Tensor, delta: torch.Tensor) -> torch.Tensor:
        """The layer's output for one new token of every sequence, whose input is x + delta."""
        y, s = decode.add_rms_norm(x, self.norms[0], delta=delta)
        qkv = torch_ops.gemm(y, self.w_qkv, fp32_reduce=True, buffers=self.bufs[0])
        q, k, v = self.split(qkv)
        slots = self.slots_of(torch.arange(x.shape[0], device=x.device), self.lens.long())
        q = decode.rope_append(q, k, v, self.cache, slots, positions=self.lens,
                               inv_freq=self.inv_freq)
        self.lens += 1
        o = self.attn(q, self.table, self.lens).flatten(1)
        o = torch_ops.gemm(o, self.w_out, fp32_reduce=True, buffers=self.bufs[1])
        y, s = decode.add_rms_norm(s, self.norms[1], delta=o)
        return self.moe(y, residual=s)


def run(batch: int = 4, steps: int = 64, prompt: int = 500, seed: int = 0, **shape) -> dict:
    """Steps eagerly and as a graph from the same state; the outputs of both, and their times."""
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    layer = DecoderLayer(g, batch, prompt + steps + 2, **shape)
    hidden = layer.w_qkv.k
    for i in range(batch):
        n = max(1, prompt - 37 * i)  # prompts of different lengths
        layer.prompt(torch.randn((n, hidden), generator=g, device=dev).half(), i)
    x = torch.randn((batch, hidden), generator=g, device=dev).half()
    delta = torch.randn((batch, hidden), generator=g, device=dev).half()
    start = layer.lens.clone()

    def timed(step):
        layer.lens.copy_(start)
        outs = []
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(steps):
            outs.append(step())
        torch.cuda.synchronize()
        return torch.stack(outs), (time.perf_counter() - t) / steps * 1e6

    layer.step(x, delta)  # warm-up, also of what a capture must not load
    eager, eager_us = timed(lambda: layer.step(x, delta))
    graph = torch.cuda.CUDAGraph()
    layer.lens.copy_(start)
    with torch.cuda.graph(graph):
        out = layer.step(x, delta)

    def replay():
        graph.replay()
        return out.clone()

    replayed, graph_us = timed(replay)
    return dict(eager=eager, graph=replayed, eager_us=eager_us, graph_us=graph_us, layer=layer,
                x=x, delta=delta, start=start)


def main() -> None:
    p = argparse.ArgumentParser()
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--prompt", type=int, default=500)
    a = p.parse_args()
    r = run(a.batch, a.steps, a.prompt)
    same = torch.equal(r["eager"], r["graph"])
    print(f"{a.steps} steps of {a.batch} sequences after prompts of up to {a.prompt}: "
          f"{r['eager_us']:.0f} us a step call by call, {r['graph_us']:.0f} us as a graph; "
          f"outputs {'the same' if same else 'DIFFER'}")
    if not same:
        sys.exit(1)


if __name__ == "__main__":
    main()
