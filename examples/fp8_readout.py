"""An fp8 gated MLP, the vocabulary head behind it, and typed answers off its logits, on one GPU.

    python examples/fp8_readout.py [--rows M] [--hidden H] [--inner I] [--vocab V] [--steps N]

The weights (synthetic here) are laid out once: e4m3 codes with one scale for each 128 x 128 tile.  A step takes the
hidden states of M requests and

    quantizes them, multiplies by the gate and up weights in one product, applies SwiGLU and quantizes,
    multiplies by the down weights, adds the hidden states, quantizes, multiplies by the vocabulary head,
    and reads off the logits: the log probabilities of the answers' tokens, the entropy and the best alternatives.

A choice is the answer with the largest log probability, a score the mean of the answers' indices under their
renormalized probabilities.  The step is run eagerly and replayed from a HIP graph, as a server of short steps does;
both give the same bits, and a request's row has the same bits whatever it is batched with.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from exact_int8_gemm_amd import prism  # noqa: E402


class Readout:
    """The frozen weights and one step over them."""

    def __init__(self, gate_up, down, head):
        """gate_up [2 I][H], down [H][I], head [V][H]: tensors of any of the library's types on the GPU."""
        self.gate_up, self.down, self.head = (prism.quantize_tiles_fp8(w) for w in (gate_up, down, head))
        self.inner = down.shape[1]

    def logits(self, x):
        """x [M][H] fp32 -> [M][V] fp32."""
        h = prism.gemm_fp8_blockscale(*prism.quantize_blocks_fp8(x), *self.gate_up, out_dtype=torch.bfloat16)
        q, s = prism.swiglu_quantize_fp8(h[:, :self.inner], h[:, self.inner:])
        x = x + prism.gemm_fp8_blockscale(q, s, *self.down)
        return prism.gemm_fp8_blockscale(*prism.quantize_blocks_fp8(x), *self.head)

    def __call__(self, x, answers, top=8):
        """answers [M][T] int64 token ids -> (choice [M], score [M], the read-out of each row)."""
        r = prism.token_logprobs(self.logits(x), answers, top=top)
        p = torch.softmax(r.logprobs, 1)
        score = (p * torch.arange(p.shape[1], device=p.device)).sum(1)
        return r.logprobs.argmax(1), score, r


def synthetic(hidden, inner, vocab, device, seed=0):
    g = torch.Generator(device=device).manual_seed(seed)

    def w(n, k):
        return torch.randn((n, k), generator=g, device=device) * k ** -0.5
    return Readout(w(2 * inner, hidden), w(hidden, inner), w(vocab, hidden) * 4)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--rows", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=2560)
    ap.add_argument("--inner", type=int, default=9728)
    ap.add_argument("--vocab", type=int, default=100003)
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    model = synthetic(a.hidden, a.inner, a.vocab, dev)
    x = torch.randn((a.rows, a.hidden), device=dev)
    answers = torch.randint(0, a.vocab, (a.rows, 5), device=dev)

    choice, score, r = model(x, answers)
    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        model(x, answers)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = model(x, answers)
    graph.replay()
    torch.cuda.synchronize()
    same = torch.equal(captured[2].logprobs, r.logprobs) and torch.equal(captured[2].top_ids, r.top_ids)
    alone = model(x[:1].contiguous(), answers[:1])[2]
    same_alone = torch.equal(alone.logprobs[0], r.logprobs[0]) and torch.equal(alone.top_ids[0], r.top_ids[0])

    t0 = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    us = (time.perf_counter() - t0) / a.steps * 1e6
    for i in range(min(a.rows, 4)):
        print("row %d: choice %d of 5, score %.3f, entropy %.3f, best token %d at %.3f"
              % (i, int(choice[i]), float(score[i]), float(r.entropy[i]), int(r.top_ids[i, 0]),
                 float(r.top_logprobs[i, 0])))
    print("replayed step: %.1f us; replay same bits: %s; row 0 alone same bits: %s" % (us, same, same_alone))
    return 0 if same and same_alone else 1


if __name__ == "__main__":
    sys.exit(main())
