"""The end of a verify step on random weights: five columns of one request,
under a grammar, with penalties over its history.

    python examples/verify_step.py [--vocab 131072] [--experts 64]

Prints the chosen tokens and the time of a step, eager and as a HIP graph."""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import quantized_moe_expert_q8_amd as moeq8  # noqa: E402
from quantized_moe_expert_q8_amd import moe_layer as ml, verify_step as vs  # noqa: E402


def milliseconds(step, n=20):
    for _ in range(3):
        step()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        step()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / n


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--vocab", type=int, default=131072)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--inter", type=int, default=1024)
    p.add_argument("--topk", type=int, default=8)
    a = p.parse_args()
    dev, cols = "cuda:0", 5
    torch.manual_seed(0)
    randn = lambda *s: torch.randn(s, device=dev)

    def experts(matrix, rows, k):
        t = torch.empty(a.experts * rows * (k // 32) * moeq8.Q8_0_BLOCK_BYTES, dtype=torch.uint8, device=dev)
        return moeq8.synth_q8_0_fill(t, a.experts, rows * k // 32, a.experts, 1, 0, 0, matrix)

    weights = vs.VerifyWeights(
        norm=1 + 0.1 * randn(a.hidden), router=vs.quantize_dense(randn(a.experts, a.hidden) / a.hidden ** 0.5),
        router_bias=None,
        experts=ml.RoutedExperts(experts(0, a.inter, a.hidden), experts(1, a.inter, a.hidden),
                                 experts(2, a.hidden, a.inter), a.experts, a.hidden, a.inter),
        final_norm=1 + 0.1 * randn(a.hidden), head=vs.quantize_dense(randn(a.vocab, a.hidden) / a.hidden ** 0.5))
    ws = vs.VerifyWorkspace(cols, weights, a.topk, dev)

    history = torch.randint(0, a.vocab, (2000 + cols,), device=dev).int()
    column = torch.arange(cols, device=dev)
    allowed = torch.randint(-2**31, 2**31, (cols, (a.vocab + 31) // 32), device=dev).int()
    rules = dict(tokens=history, begin=0 * column, end=2000 + column, prompt_end=0 * column + 1500,
                 repetition=torch.full((cols,), 1.1, device=dev), frequency=torch.full((cols,), 0.2, device=dev),
                 mask=allowed)
    x, residual = randn(cols, a.hidden), randn(cols, a.hidden)
    step = lambda: vs.forward(x, residual, weights, ws, rules=rules)

    print("tokens", step().argmax(1).tolist())
    eager = milliseconds(step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    print(f"a step: {eager * 1e3:.0f} us eager, {milliseconds(graph.replay) * 1e3:.0f} us in a graph", flush=True)
    print("tokens", ws.logits.argmax(1).tolist())


if __name__ == "__main__":
    main()
