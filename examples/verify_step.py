"""A verify step on random weights: five columns of one request through attention
over its cached history, the routed experts and the head, under a grammar, with
penalties over the history, and a token drawn for each column.

    python examples/verify_step.py [--vocab 131072] [--experts 64] [--history 2000]

Prints the drawn tokens and the time of a step, eager and as a HIP graph."""

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
    p.add_argument("--heads", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--head-dim", type=int, default=128)
    p.add_argument("--history", type=int, default=2000)
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

    heads, kv, d, page, length = a.heads, a.kv_heads, a.head_dim, 64, a.history + cols
    attention = vs.AttentionWeights(
        norm=1 + 0.1 * randn(a.hidden), qkv=vs.quantize_dense(randn((heads + 2 * kv) * d, a.hidden) / a.hidden ** 0.5),
        out=vs.quantize_dense(randn(a.hidden, heads * d) / (heads * d) ** 0.5), heads=heads, kv_heads=kv, d=d)
    aws = vs.AttentionWorkspace(1, cols, attention, length, dev)
    cache = moeq8.kv_cache_i8(-(-length // page), kv, page, d, dev)
    moeq8.kv_cache_write_i8(randn(length, kv, d), randn(length, kv, d), cache, torch.arange(length, device=dev))
    pages = torch.arange(-(-length // page), device=dev).int()[None]
    column = torch.arange(cols, device=dev)
    visible, slots = (a.history + 1 + column).int()[None], a.history + column

    history = torch.randint(0, a.vocab, (length,), device=dev).int()
    allowed = torch.randint(-2**31, 2**31, (cols, (a.vocab + 31) // 32), device=dev).int()
    rules = dict(tokens=history, begin=0 * column, end=a.history + column, prompt_end=0 * column + a.history * 3 // 4,
                 repetition=torch.full((cols,), 1.1, device=dev), frequency=torch.full((cols,), 0.2, device=dev),
                 mask=allowed)
    sampling = dict(u=torch.rand(cols, device=dev), temperature=torch.full((cols,), 0.8, device=dev),
                    top_p=torch.full((cols,), 0.95, device=dev), min_p=torch.full((cols,), 0.02, device=dev))
    x, residual = randn(cols, a.hidden), randn(cols, a.hidden)

    def step():
        y, r = vs.attend(x, residual, attention, aws, cache, pages, visible, slots)
        vs.forward(y, r, weights, ws, rules=rules, sampling=sampling)
        return ws.token

    print("tokens", step().tolist())
    eager = milliseconds(step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    print(f"a step: {eager * 1e3:.0f} us eager, {milliseconds(graph.replay) * 1e3:.0f} us in a graph", flush=True)
    print("tokens", ws.token.tolist())


if __name__ == "__main__":
    main()
