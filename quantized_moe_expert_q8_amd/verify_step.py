"""A verify / decode step around the routed experts as fixed sequences of libmoeq8
calls.

attend(): the attention block in front of them, over a paged int8 cache.

    q, s, r     = rms_norm_q8(x, w, residual)        int8 rows and the residual stream
    qkv         = gemm_i8(q, s, Wqkv)                queries, keys and values of the columns
    kv_cache_write_i8(k, v, cache, slots)            the columns' own rows
    a           = paged_attention_i8(q, cache, pages, visible)
    y           = gemm_i8(i8_quantize_rows(a), Wo)   into the next norm, with r

forward(): the norm in front of a routed MoE block, the block, the final norm, the
vocabulary head, the sampling rules on its logits, and the draw of the tokens.

    q, s, xq, r = rms_norm_q8(x, w, residual)        one pass: residual, int8 rows and q8_1 rows
    router      = gemm_i8(q, s, Wr)                  expert scores
    y           = routed experts on xq               grouped products, as in moe_layer
    q, s, r     = rms_norm_q8(y, w_out, residual=r)
    z           = gemm_i8(q, s, Wv)                  vocabulary logits
    z           = logits_process(z, ...)             penalties, biases, grammar mask, in place
    t, logprob  = logits_sample(z, u, ...)           where asked for

Weights are int8 with a scale per output channel (quantize_dense, once at load
time); buffers live in a workspace, so a step allocates nothing and can be
captured in a HIP graph.  No arithmetic happens here.
"""

from __future__ import annotations

from dataclasses import dataclass

import torch

from . import ops
from .moe_layer import RoutedExperts

QK = ops.QK


@dataclass
class DenseI8:
    """int8 weights [channels, k] with an fp32 scale per channel."""
    codes: torch.Tensor
    scale: torch.Tensor


def quantize_dense(w: torch.Tensor) -> DenseI8:
    """Weights [channels, k] (fp32, fp16 or bf16) as int8 with a scale a channel."""
    return DenseI8(*ops.i8_quantize_rows(w))


@dataclass
class VerifyWeights:
    norm: torch.Tensor               # [hidden], the activations' dtype
    router: DenseI8                  # [n_expert, hidden]
    router_bias: torch.Tensor | None  # fp32 [n_expert]
    experts: RoutedExperts           # plain Q8_0
    final_norm: torch.Tensor         # [hidden], fp32
    head: DenseI8                    # [vocab, hidden]


@dataclass
class AttentionWeights:
    norm: torch.Tensor               # [hidden], the activations' dtype
    qkv: DenseI8                     # [(heads + 2 kv_heads) * d, hidden]: queries, keys, values
    out: DenseI8                     # [hidden, heads * d]
    heads: int
    kv_heads: int
    d: int


class AttentionWorkspace:
    """Buffers of attend() for seqs sequences of cols columns; no sequence sees
    more than max_visible positions."""

    def __init__(self, seqs: int, cols: int, weights: AttentionWeights, max_visible: int, device):
        dev = torch.device(device)
        w, n, hidden = weights, seqs * cols, weights.qkv.codes.shape[1]
        new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device=dev)
        self.seqs, self.cols, self.max_visible = seqs, cols, max_visible
        self.q, self.scale = new(n, hidden, dtype=torch.int8), new(n)
        self.qkv = new(n, (w.heads + 2 * w.kv_heads) * w.d)
        self.attended = new(seqs, cols, w.heads, w.d)
        self.rows, self.row_scale = new(n, w.heads * w.d, dtype=torch.int8), new(n)
        self.out, self.residual = new(n, hidden), new(n, hidden)
        self.workspace = new(ops.paged_attention_workspace_bytes(seqs, cols, w.heads, w.kv_heads, w.d, max_visible),
                             dtype=torch.uint8)


def attend(x: torch.Tensor, residual: torch.Tensor, weights: AttentionWeights, ws: AttentionWorkspace,
           cache: ops.KVCacheI8, pages: torch.Tensor, visible: torch.Tensor, slots: torch.Tensor, *, eps: float = 1e-6,
           scale: float | None = None, rotate=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Enqueue the attention block of seqs * cols tokens on the current stream: x
    and residual [tokens, hidden] fp32, a sequence's columns in a row.

    slots (int64 [tokens]) are where the tokens' own keys and values go, pages and
    visible as for ops.paged_attention_i8.  rotate(q, k), if given, puts positions
    into the views q [tokens, heads, d] and k [tokens, kv_heads, d] in place before
    they are used.  Returns the block's output and the residual stream in front of
    it, both [tokens, hidden], which forward takes."""
    w, n = weights, ws.seqs * ws.cols
    ops.rms_norm_q8(x, w.norm, eps=eps, residual=residual, residual_out=ws.residual, q=ws.q, scale=ws.scale)
    ops.gemm_i8(ws.q, ws.scale, w.qkv.codes, w.qkv.scale, out=ws.qkv)
    q, k, v = (t.view(n, -1, w.d) for t in ws.qkv.split([w.heads * w.d, w.kv_heads * w.d, w.kv_heads * w.d], dim=1))
    if rotate is not None:
        rotate(q, k)
    ops.kv_cache_write_i8(k, v, cache, slots)
    ops.paged_attention_i8(q.view(ws.seqs, ws.cols, w.heads, w.d), cache, pages, visible, scale=scale,
                           max_visible=ws.max_visible, out=ws.attended, workspace=ws.workspace)
    ops.i8_quantize_rows(ws.attended.view(n, -1), q=ws.rows, scale=ws.row_scale)
    ops.gemm_i8(ws.rows, ws.row_scale, w.out.codes, w.out.scale, out=ws.out)
    return ws.out, ws.residual


class VerifyWorkspace:
    def __init__(self, ncols: int, weights: VerifyWeights, topk: int, device):
        dev = torch.device(device)
        hidden, inter = weights.experts.hidden, weights.experts.inter
        n_expert, vocab = weights.router.codes.shape[0], weights.head.codes.shape[0]
        new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device=dev)
        self.ncols, self.topk = ncols, topk
        self.q, self.scale = new(ncols, hidden, dtype=torch.int8), new(ncols)
        self.xq = new(ncols, hidden // QK * ops.Q8_1_BLOCK_BYTES, dtype=torch.uint8)
        self.router = new(ncols, n_expert)
        self.ids, self.route_weights = new(ncols, topk, dtype=torch.int32), new(ncols, topk)
        self.grouping = new(ops.moe_grouping_bytes(ncols, topk), dtype=torch.uint8)
        self.h, self.y = new(ncols, topk, inter), new(ncols, topk, hidden)
        self.out = new(ncols, hidden)
        self.residual = new(ncols, hidden)
        self.logits = new(ncols, vocab)
        self.token, self.logprob = new(ncols, dtype=torch.int32), new(ncols)
        self.sample = new(ops.logits_sample_workspace_bytes(ncols, vocab), dtype=torch.uint8)


def forward(x: torch.Tensor, residual: torch.Tensor, weights: VerifyWeights, ws: VerifyWorkspace, *,
            eps: float = 1e-6, rules: dict | None = None, sampling: dict | None = None) -> torch.Tensor:
    """Enqueue one step's end on the current stream: x and residual [ncols,
    hidden] fp32 (the columns of a verify step, at most 8), rules the keyword
    arguments of ops.logits_process, sampling those of ops.logits_sample (u among
    them).  Returns ws.logits [ncols, vocab]; the residual stream after the block is
    in ws.residual, drawn tokens and their log probabilities in ws.token and
    ws.logprob."""
    w, c, topk = weights, ws.ncols, ws.topk
    e = w.experts
    if e.packed or e.fmt != "q8_0":
        raise ValueError("the step reads plain Q8_0 experts")
    ops.rms_norm_q8(x, w.norm, eps=eps, residual=residual, residual_out=ws.residual, fmt="both", q=ws.q,
                    scale=ws.scale, xq=ws.xq)
    ops.gemm_i8(ws.q, ws.scale, w.router.codes, w.router.scale, out=ws.router)
    ops.moe_route_topk(ws.router, topk, bias=w.router_bias, ids=ws.ids, weights=ws.route_weights,
                       grouping=ws.grouping)
    ops.moe_grouped_mmvq(ops.GATE_UP_SWIGLU, e.gate, e.up, ws.xq, ws.grouping, n=e.inter, k=e.hidden,
                         n_local_expert=e.n_local, ncols=c, topk=topk, out=ws.h)
    ops.moe_grouped_mmvq_ex(ops.DOWN_F32_ACT, e.down, None, ws.h.view(c * topk, e.inter), ws.grouping,
                            n=e.hidden, k=e.inter, n_local_expert=e.n_local, ncols=c, topk=topk, out=ws.y)
    ops.moe_combine(ws.y, ws.ids, ws.route_weights, out=ws.out)
    ops.rms_norm_q8(ws.out, w.final_norm, eps=eps, residual=ws.residual, residual_out=ws.residual, q=ws.q,
                    scale=ws.scale)
    ops.gemm_i8(ws.q, ws.scale, w.head.codes, w.head.scale, out=ws.logits)
    if rules:
        ops.logits_process(ws.logits, out=ws.logits, **rules)
    if sampling:
        ops.logits_sample(ws.logits, token=ws.token, logprob=ws.logprob, workspace=ws.sample, **sampling)
    return ws.logits
