"""One decoder layer with 4-bit weights, token by token, on libwq alone.

    python examples/decode_layer.py [--batch 4] [--steps 64] [--prompt 500]
                                    [--cache4] [--qk-norm] [--vocab 32000]

Random weights of a mixture-of-experts layer (hidden 4096, 32 query and 8 KV heads of 128,
eight experts of 14336, two for each token).  A prompt's keys and values are written to a paged
cache by the rotary append; then each step runs

    residual add and RMS norm, QKV product, rotary append, paged attention, output product,
    residual add and RMS norm, mixture-of-experts layer

for one new token per sequence, first call by call and then as one captured graph, and the two
are compared.  --cache4 keeps keys and values as 4-bit codes, --qk-norm norms the heads of queries
and keys, and --vocab makes tokens of the steps: a token's embedding is the layer's input, and the
next one is drawn from the logits of its output."""

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
                 top_k: int = 2, page_size: int = 16, cache4: bool = False,
                 qk_norm: bool = False, vocab: int = 0):
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
        kind = decode.PagedCache4 if cache4 else decode.PagedCache
        self.cache = kind.empty(batch * pages, page_size, kv_heads, head_dim, torch.float16, dev)
        order = torch.randperm(batch * pages, generator=g, device=dev)
        self.table = order.view(batch, pages).to(torch.int32)
        self.attn = decode.PagedAttention(self.cache, batch, q_heads, max_len,
                                          dtype=torch.float16)
        half = head_dim // 2
        self.inv_freq = (500000.0 ** (-torch.arange(half, device=dev).double() / half)).float()
        self.lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.q_norm = self.k_norm = None
        if qk_norm:
            self.q_norm, self.k_norm = (
                (1 + 0.1 * torch.randn(head_dim, generator=g, device=dev)).half() for _ in range(2))
        if vocab:
            self.embedding = torch.randn((vocab, hidden), generator=g, device=dev).half()
            self.w_head = packed(hidden, vocab)
            self.head_bufs = torch_ops.GemmBuffers(self.w_head, batch, True)
            self.sampler = decode.Sampler(batch, vocab, dtype=torch.float16, device=dev)
            self.temperature = torch.full((batch,), 0.8, device=dev)
            self.top_k = torch.full((batch,), 40, dtype=torch.int32, device=dev)
            self.top_p = torch.full((batch,), 0.95, device=dev)
            self.ids = torch.zeros(batch, dtype=torch.int32, device=dev)

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
                           positions=at.to(torch.int32), inv_freq=self.inv_freq,
                           k_norm=self.k_norm)
        self.lens[sequence] = x.shape[0]

    def step(self, x: torch.Tensor, delta: torch.Tensor) -> torch.Tensor:
        """The layer's output for one new token of every sequence, whose input is x + delta."""
        y, s = decode.add_rms_norm(x, self.norms[0], delta=delta)
        qkv = torch_ops.gemm(y, self.w_qkv, fp32_reduce=True, buffers=self.bufs[0])
        q, k, v = self.split(qkv)
        slots = self.slots_of(torch.arange(x.shape[0], device=x.device), self.lens.long())
        q = decode.rope_append(q, k, v, self.cache, slots, positions=self.lens,
                               inv_freq=self.inv_freq, q_norm=self.q_norm, k_norm=self.k_norm)
        self.lens += 1
        o = self.attn(q, self.table, self.lens).flatten(1)
        o = torch_ops.gemm(o, self.w_out, fp32_reduce=True, buffers=self.bufs[1])
        y, s = decode.add_rms_norm(s, self.norms[1], delta=o)
        return self.moe(y, residual=s)

    def token_step(self, u: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
        """The next token of every sequence, which becomes the next step's input, and the log of its
        share, by the random numbers u [batch]."""
        x = self.embedding[self.ids.long()]
        y, _ = decode.add_rms_norm(self.step(x, torch.zeros_like(x)), self.norms[0])
        self.logits = torch_ops.gemm(y, self.w_head, fp32_reduce=True, buffers=self.head_bufs)
        return self.sampler(self.logits, u, temperature=self.temperature, top_k=self.top_k,
                            top_p=self.top_p, ids=self.ids, logprob=True)


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


def generate(batch: int = 4, steps: int = 64, prompt: int = 500, vocab: int = 32000, seed: int = 0,
             **shape) -> dict:
    """Tokens and the logs of their shares [steps][batch], drawn step by step, eagerly and as a
    graph, from the same state and the same random numbers; and the times of a step."""
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    layer = DecoderLayer(g, batch, prompt + steps + 2, vocab=vocab, **shape)
    for i in range(batch):
        n = max(1, prompt - 37 * i)
        layer.prompt(torch.randn((n, layer.w_qkv.k), generator=g, device=dev).half(), i)
    start = layer.lens.clone()
    u = torch.rand((steps, batch), generator=g, device=dev)
    now = u[0].clone()

    def timed(step):
        layer.lens.copy_(start)
        layer.ids.zero_()
        outs = []
        torch.cuda.synchronize()
        t = time.perf_counter()
        for i in range(steps):
            now.copy_(u[i])
            outs.append([x.clone() for x in step()])
        torch.cuda.synchronize()
        us = (time.perf_counter() - t) / steps * 1e6
        return [torch.stack(x) for x in zip(*outs)], us

    layer.token_step(now)  # warm-up, also of what a capture must not load
    eager, eager_us = timed(lambda: layer.token_step(now))
    graph = torch.cuda.CUDAGraph()
    layer.lens.copy_(start)
    with torch.cuda.graph(graph):
        out = layer.token_step(now)

    def replay():
        graph.replay()
        return out

    replayed, graph_us = timed(replay)
    return dict(eager=eager, graph=replayed, eager_us=eager_us, graph_us=graph_us, layer=layer,
                u=u)


def main() -> None:
    p = argparse.ArgumentParser()
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--prompt", type=int, default=500)
    p.add_argument("--cache4", action="store_true")
    p.add_argument("--qk-norm", action="store_true")
    p.add_argument("--vocab", type=int, default=0)
    a = p.parse_args()
    shape = dict(cache4=a.cache4, qk_norm=a.qk_norm)
    if a.vocab:
        r = generate(a.batch, a.steps, a.prompt, a.vocab, **shape)
        same = all(torch.equal(x, y) for x, y in zip(r["eager"], r["graph"]))
        what = "tokens"
    else:
        r = run(a.batch, a.steps, a.prompt, **shape)
        same, what = torch.equal(r["eager"], r["graph"]), "outputs"
    print(f"{a.steps} steps of {a.batch} sequences after prompts of up to {a.prompt}: "
          f"{r['eager_us']:.0f} us a step call by call, {r['graph_us']:.0f} us as a graph; "
          f"{what} {'the same' if same else 'DIFFER'}")
    if not same:
        sys.exit(1)


if __name__ == "__main__":
    main()
