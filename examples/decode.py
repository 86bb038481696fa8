"""A few decode steps through three pre-norm sublayers as a server would run
them: an MLP with biases, a SwiGLU MLP on 4-bit weights, then a mixture of
experts, its experts first in 16 bits and then in 4.  Each sublayer's sum is left
to the next one's norm.  Random weights; prints the time per token and how far the
4-bit experts are from the 16-bit ones.

    python examples/decode.py [--hidden 2048] [--steps 64] [--streams 1]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from backward_tcgen05_tma_gb300.block import LayerNorm, MLP, MLPBlock  # noqa: E402
from backward_tcgen05_tma_gb300.module import SwiGLUMLP  # noqa: E402
from backward_tcgen05_tma_gb300.serving import MoESwiGLU, W4SwiGLUMLP  # noqa: E402


def step(blocks, norm, x):
    delta = None
    for block in blocks:
        x, delta = block(x, delta, join=False)
    return norm(delta, x)[0]


def decode(blocks, norm, x, steps):
    """Microseconds of a step: one is captured as a CUDA graph and replayed."""
    x = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):  # what a first call sets up is not captured
            x.copy_(step(blocks, norm, x))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(step(blocks, norm, x))
    graph.replay()
    beg, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    beg.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    end.synchronize()
    return beg.elapsed_time(end) / steps * 1e3


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--streams", type=int, default=1)
    a = p.parse_args()
    torch.manual_seed(0)
    D = a.hidden
    with torch.no_grad():
        H = 11 * D // 4 // 8 * 8
        mlp = W4SwiGLUMLP(SwiGLUMLP(D, H, device="cuda"), group=128)
        moe = MoESwiGLU(D, D // 2, 64, 8, device="cuda")
        blocks = [MLPBlock(m, hidden_size=D, device="cuda") for m in (MLP(D, H, device="cuda"), mlp, moe)]
        norm = LayerNorm(D, device="cuda")
        x = torch.randn(a.streams, D, dtype=torch.bfloat16, device="cuda")
        first = {}
        for bits in (16, 4):
            if bits == 4:
                moe.quantize(group=128)
            first[bits] = moe(x).float()
            print("%2d-bit experts: %.1f us a step of %d token(s)"
                  % (bits, decode(blocks, norm, x, a.steps), a.streams))
        off = (first[4] - first[16]).norm() / first[16].norm()
        print("4-bit against 16-bit experts, one layer: %.1f%% apart" % (100 * off))


if __name__ == "__main__":
    main()
