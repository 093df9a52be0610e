"""A quantised layer of experts, start to finish.

Every expert's gate, up and down projections are packed and repacked to 4 bits, one weight with all
experts' rows for each product.  A prompt goes through the router, the experts' products on its own
rows and the way back onto the residual stream, four calls in all; then single tokens take the same
calls, captured in a HIP graph.  Printed at the end: how far the layer is from the same
dequantised weights in 64 bits, and the time of a step.

    python examples/experts_layer.py
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

BITS, GROUP = 4, 64


class Packed:
    """The projections [experts, n, K] of all experts as one packed weight."""

    def __init__(self, weights: torch.Tensor):
        experts, n, K = weights.shape
        rows, ones = weights.reshape(experts * n, K), torch.ones(K, device=weights.device)
        codes, steps, zeros = awq.awq_quantize_pack(rows, ones, BITS, GROUP)
        self.codes, self.meta = awq.awq_lowbit_repack(codes, steps, zeros, K, BITS, GROUP)
        self.dequantised = awq.awq_fake_quant(rows, ones, BITS, GROUP)[0].reshape(experts, n, K)   # to compare with

    def __call__(self, x: torch.Tensor, routing: awq.Routing, **kw) -> torch.Tensor:
        return awq.awq_lowbit_linear(x, self.codes, self.meta, BITS, GROUP, routing=routing, **kw)


class Experts:
    """x + sum over a token's k experts of weight down(silu(gate x) up x)."""

    def __init__(self, hidden: int, inner: int, experts: int, k: int, seed: int = 0, dtype=torch.bfloat16):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(shape, generator=gen, device="cuda") * std

        self.k = k
        self.router = normal(experts, hidden, std=hidden ** -0.5)
        self.bias = normal(experts, std=0.05)            # for the choice alone, to even out the load
        self.up = Packed(normal(experts, 2 * inner, hidden, std=hidden ** -0.5).to(dtype))
        self.down = Packed(normal(experts, hidden, inner, std=inner ** -0.5).to(dtype))

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        routing = awq.awq_moe_route(x.float() @ self.router.T, self.k, score="sigmoid", bias=self.bias)
        h = self.up(x, routing, gather=True, activation="silu", gated=True)
        return awq.awq_moe_combine(self.down(h, routing), routing, routing.weights, residual=x)

    def in_64_bits(self, x: torch.Tensor, routing: awq.Routing) -> torch.Tensor:
        y, up, down = x.double(), self.up.dequantised.double(), self.down.dequantised.double()
        for e in range(up.shape[0]):
            t, j = (routing.experts == e).nonzero(as_tuple=True)
            gate, lift = (x[t].double() @ up[e].T).chunk(2, dim=-1)
            y.index_add_(0, t, routing.weights[t, j].double()[:, None]
                         * ((torch.nn.functional.silu(gate) * lift) @ down[e].T))
        return y


@torch.no_grad()
def main(hidden: int = 512, inner: int = 256, experts: int = 16, k: int = 4, tokens: int = 300, steps: int = 20,
         seed: int = 0, verbose: bool = True) -> tuple[float, bool]:
    """-> (error relative to 64 bits, whether replays gave what eager calls give)."""
    layer = Experts(hidden, inner, experts, k, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn((tokens, hidden), generator=gen, device="cuda").bfloat16()
    y = layer(x)
    routing = awq.awq_moe_route(x.float() @ layer.router.T, k, score="sigmoid", bias=layer.bias)
    want = layer.in_64_bits(x, routing)
    error = float((y.double() - want).norm() / (want - x.double()).norm())

    token = x[:1].clone()
    layer(token)                                         # loads what a capture may not
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(token)
    same = True
    for i in range(steps):
        token.copy_(x[i % tokens][None])
        graph.replay()
        same &= bool(torch.equal(out, layer(token)))
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(100):
        graph.replay()
    torch.cuda.synchronize()
    if verbose:
        print(f"{tokens} tokens, {experts} experts of {hidden} x {inner}, {k} a token: error {error:.2e} of the experts' "
              f"share; a captured token {(time.perf_counter() - t0) * 1e4:.1f} us")
    return error, same


if __name__ == "__main__":
    main()
