"""A mixture-of-experts layer in fp8, as a served step, on one GPU.

    python examples/moe_layer.py [--tokens M] [--hidden H] [--inner I] [--experts E] [--top T] [--layers L] [--steps N]

The weights (synthetic here) are laid out once: e4m3 codes with one scale for each 128 x 128 tile of each expert's
weights.  A layer takes the layer before's output and the residual of M tokens and

    adds the residual, norms and quantizes in one pass,
    multiplies the norm's e4m3 codes by the router's weights, also in e4m3, so that a token's logits have the same bits in
    any batch (a router that is to see the norm itself takes it from the same call with norm=True, and its own product),
    chooses each token's experts and lists the rows of each expert,
    multiplies those rows by their experts' gate and up weights, applies SwiGLU and quantizes,
    multiplies by the down weights, and adds up each token's outputs with the router's weights.

The step is run eagerly and replayed from a HIP graph, whose routing may differ in every replay; both give the same
bits, and a token's result has the same bits whatever it is batched with.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from exact_int8_gemm_amd import prism  # noqa: E402


def quantize_experts(w):
    """w [E][N][K] of any of the library's types on the GPU -> codes [E][N][K], scales [E][ceil(N/128)][ceil(K/128)]."""
    e, n, k = w.shape
    q = torch.empty((e, n, k), dtype=prism.FP8, device=w.device)
    scale = torch.empty((e, -(-n // 128), -(-k // 128)), device=w.device)
    for i in range(e):
        prism.quantize_tiles_fp8(w[i], q=q[i], scale=scale[i])
    return q, scale


class Layer:
    """One layer's frozen weights."""

    def __init__(self, gain, router, gate_up, down, top, eps=1e-6):
        """gain [H], router [E][H] fp32, gate_up [E][2 I][H], down [E][H][I]."""
        self.gain, self.eps, self.top = gain, eps, top
        # fp8 with an fp32 result: a product whose rows do not depend on the batch
        self.router = prism.quantize_tiles_fp8(router)
        self.gate_up, self.down = quantize_experts(gate_up), quantize_experts(down)
        self.inner = down.shape[2]

    def __call__(self, x, residual):
        """x [M][H] bf16, residual [M][H] fp32 -> (this layer's output bf16, the residual with x added)."""
        h = prism.add_rmsnorm_quantize_fp8(x, self.gain, self.eps, residual=residual)
        r = prism.route_experts(prism.gemm_fp8_blockscale(h.q, h.scale, *self.router), self.top)
        gu = prism.gemm_fp8_grouped(h.q, h.scale, *self.gate_up, r.offsets, rows=r.rows, out_dtype=torch.bfloat16)
        q, s = prism.swiglu_quantize_fp8(gu[:, :self.inner], gu[:, self.inner:])
        y = prism.gemm_fp8_grouped(q, s, *self.down, r.offsets, out_dtype=torch.bfloat16)
        return prism.combine_experts(y, r.weights, r.slots), h.residual


def synthetic(hidden, inner, experts, top, device, seed=0):
    g = torch.Generator(device=device).manual_seed(seed)

    def w(*shape):
        return torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5
    return Layer(1 + 0.1 * w(hidden), 2 * w(experts, hidden), w(experts, 2 * inner, hidden), w(experts, hidden, inner), top)


def run(layers, x, residual):
    for layer in layers:
        x, residual = layer(x, residual)
    return x, residual


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=2560)
    ap.add_argument("--inner", type=int, default=1280)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top", type=int, default=8)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    layers = [synthetic(a.hidden, a.inner, a.experts, a.top, dev, i) for i in range(a.layers)]
    x = torch.randn((a.tokens, a.hidden), device=dev).bfloat16()
    residual = torch.randn((a.tokens, a.hidden), device=dev)

    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        run(layers, x, residual)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(layers, x, residual)
    same = True
    for _ in range(3):
        x.normal_()  # other tokens, other experts
        graph.replay()
        eager = run(layers, x, residual)
        torch.cuda.synchronize()
        same = same and all(torch.equal(u, v) for u, v in zip(captured, eager))
    alone = run(layers, x[:1].contiguous(), residual[:1].contiguous())
    same_alone = all(torch.equal(u[0], v[0]) for u, v in zip(alone, eager))

    t0 = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    us = (time.perf_counter() - t0) / a.steps * 1e6
    print("replayed step of %d layers, %d tokens: %.1f us; replay same bits: %s; token 0 alone same bits: %s"
          % (a.layers, a.tokens, us, same, same_alone))
    return 0 if same and same_alone else 1


if __name__ == "__main__":
    sys.exit(main())
