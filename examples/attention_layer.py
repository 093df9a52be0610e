"""A quantised attention layer serving uneven sequences, start to finish.

The qkv and output projections are searched, packed and repacked to 4 bits; prompts of different
lengths go through them, the rotation and the 8-bit paged cache in one call each; then every
sequence takes tokens one by one, the whole step captured in a HIP graph.  Printed at the end:
how far the layer is from the same weights with an unquantised cache in 64 bits, and the time of a
step.

    python examples/attention_layer.py
"""

from __future__ import annotations

import sys
import time
from pathlib import Path

import torch

ROOT = Path(__file__).resolve().parents[1]
if str(ROOT) not in sys.path:
    sys.path.insert(0, str(ROOT))

import post_weight_quantization_act_amd as awq  # noqa: E402

BITS, GROUP = 4, 128


class LowBitLinear:
    """y = x W^T with W packed to 4 bits by the activation-aware search on calibration inputs."""

    def __init__(self, weight: torch.Tensor, inputs: torch.Tensor):
        res = awq.awq_search_scales(weight, inputs, awq.awq_act_stats(inputs), BITS, GROUP,
                                    [i / 8 for i in range(8)])
        self.s = res["s_best"]
        codes, steps, zeros = awq.awq_quantize_pack(weight, self.s, BITS, GROUP)
        self.codes, self.meta = awq.awq_lowbit_repack(codes, steps, zeros, weight.shape[1], BITS, GROUP)
        self.dequantised = awq.awq_fake_quant(weight, self.s, BITS, GROUP)[0]     # for the comparison

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        return awq.awq_lowbit_gemv((x / self.s).to(x.dtype), self.codes, self.meta, BITS, GROUP)


class Attention:
    def __init__(self, hidden: int, heads: int, kv_heads: int, page: int, pages: int, longest: int,
                 seed: int = 0, dtype=torch.float16):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

        self.heads, self.kv_heads, self.dim = heads, kv_heads, hidden // heads
        self.dtype = dtype
        self.qkv = LowBitLinear(normal((heads + 2 * kv_heads) * self.dim, hidden, std=hidden ** -0.5),
                                normal(512, hidden))
        self.o = LowBitLinear(normal(hidden, heads * self.dim, std=hidden ** -0.5),
                              normal(512, heads * self.dim))
        self.cache = awq.KvCache.empty(pages, kv_heads, page, self.dim)
        # twice the length that the frequencies were made for: the slow ones are slowed
        self.table = awq.awq_rope_table(longest, self.dim, scaling="turns", factor=2.0,
                                        original=longest / 2)

    def __call__(self, x, lens, table, starts=None, max_new=None, max_len=None):
        """x [T, hidden]: the new tokens of every sequence, one after another -> [T, hidden]."""
        T, h, kv = x.shape[0], self.heads, self.kv_heads
        qkv = self.qkv(x).view(T, h + 2 * kv, self.dim)            # fp32, queries, keys, values
        q = awq.awq_kv_append(self.cache, qkv[:, h: h + kv], qkv[:, h + kv:], lens, table,
                              starts=starts, max_new=max_new, table=self.table, q=qkv[:, :h],
                              q_dtype=self.dtype)
        out = awq.awq_kv_attention(self.cache, q, lens, table, starts=starts, max_new=max_new,
                                   max_len=max_len)
        return self.o(out.view(T, h * self.dim))

    def reference(self, x: torch.Tensor) -> torch.Tensor:
        """One sequence in 64 bits: the packed weights' values, no cache."""
        n, h, kv, d = x.shape[0], self.heads, self.kv_heads, self.dim
        qkv = (x.double() @ self.qkv.dequantised.double().T).view(n, h + 2 * kv, d)
        c, s = self.table[:n].double().unbind(-1)
        c, s = c[:, None], s[:, None]
        q, k, v = qkv.split((h, kv, kv), 1)

        def turn(t):
            a, b = t.chunk(2, -1)
            return torch.cat((a * c - b * s, b * c + a * s), -1)

        q, k = turn(q), turn(k).repeat_interleave(h // kv, 1)
        v = v.repeat_interleave(h // kv, 1)
        scores = (q.transpose(0, 1) @ k.permute(1, 2, 0).contiguous()) * d ** -0.5
        hidden = torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1)
        p = scores.masked_fill(hidden, float("-inf")).softmax(-1)
        out = (p @ v.transpose(0, 1).contiguous()).transpose(0, 1).reshape(n, h * d)
        return out @ self.o.dequantised.double().T


def main(hidden=2048, heads=16, kv_heads=4, page=64, prompts=(700, 33, 1, 256), steps=24, seed=0,
         verbose=True):
    """Returns (relative error of all outputs, outputs of the graph's steps equal to eager ones)."""
    B, longest = len(prompts), max(prompts) + steps
    per_seq = -(-longest // page)
    layer = Attention(hidden, heads, kv_heads, page, B * per_seq, longest, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    xs = [torch.randn((n + steps, hidden), generator=gen, device="cuda").to(layer.dtype) for n in prompts]
    order = torch.randperm(B * per_seq, generator=gen, device="cuda").int()
    table = order.view(B, per_seq).contiguous()                     # pages in any order
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, *prompts], device="cuda").cumsum(0).int()

    outs = [list(layer(torch.cat([x[:n] for x, n in zip(xs, prompts)]), lens, table, starts=starts,
                       max_new=max(prompts), max_len=max(prompts)).split(prompts))]
    new = torch.empty((B, hidden), dtype=layer.dtype, device="cuda")
    rows = lambda i: torch.stack([x[n + i] for x, n in zip(xs, prompts)])        # noqa: E731

    # the first steps eagerly (and to warm up), the others from a graph: lengths live on the device
    same = True
    for i in range(2):
        lens += 1
        new.copy_(rows(i))
        outs.append(layer(new, lens, table, max_len=longest))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(new, lens, table, max_len=longest)
    began = 0.0
    for i in range(2, steps):
        lens += 1
        new.copy_(rows(i))
        if i == 3:
            torch.cuda.synchronize()
            began = time.perf_counter()
        graph.replay()
        outs.append(y.clone())
    torch.cuda.synchronize()
    each = (time.perf_counter() - began) / (steps - 3)
    # the last token again, eagerly: its place in the cache is written with the same codes
    same = torch.equal(layer(new, lens, table, max_len=longest), outs[-1])

    off = norm = 0.0
    for b, (x, n) in enumerate(zip(xs, prompts)):
        want = layer.reference(x)
        got = torch.cat([outs[0][b], torch.stack([o[b] for o in outs[1:]])]).double()
        off += float((got - want).square().sum())
        norm += float(want.square().sum())
    error = (off / norm) ** 0.5
    if verbose:
        print(f"{B} sequences of {prompts} tokens and {steps} more each: relative error {error:.4f} "
              f"(8-bit cache), replayed step equal to the eager one: {same}, {each * 1e6:.1f} us a step")
    return error, same


if __name__ == "__main__":
    main()
