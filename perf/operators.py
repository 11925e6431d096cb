"""Timed cases of the operators around the expert layer: RMS norm with the
residual's addition and 8-bit outputs (rms_norm_q8), int8 rows with a scale each
(i8_quantize_rows), the int8 matrix product with token and channel scales
(gemm_i8), and penalties, biases and grammar masks on logits (logits_process).

run() computes each in its plain form, elementary torch operations in 32 bits,
or with ``own`` true by the library's calls.  Sums of squares and quotients
that decide an 8-bit code are taken in 64 bits and rounded once, as the
operators are defined, so codes are compared as the signed integers they are,
each beside its scale."""

import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token entering a block in 16 bits: latency alone
        dict(name="norm decode 1x4096", op="norm", rows=1, k=4096, dtype="bf16", residual=True, fmt="i8"),
        # the verify step's 5 columns, fp32, into the expert products' q8_1 rows
        dict(name="norm verify 5x4096", op="norm", rows=5, k=4096, dtype="f32", residual=True, fmt="q8_1"),
        # a prefill chunk in 16 bits, for dense products
        dict(name="norm prefill 8192x8192", op="norm", rows=8192, k=8192, dtype="bf16", residual=True, fmt="i8"),
        # an attention output before its projection, at one verify step's 8 columns
        dict(name="quant verify 8x4096", op="quant", rows=8, k=4096, dtype="f16"),
        # expert activations of a wide batch (1024 columns, 8 routes each), odd length
        dict(name="quant wide 8192x2047", op="quant", rows=8192, k=2047, dtype="f32"),
        # one token through a square projection
        dict(name="gemm decode 1x4096x4096", op="gemm", m=1, n=4096, k=4096, out="bf16", bias=False),
        # the verify step's 5 columns through the vocabulary head
        dict(name="gemm head 5x131072x4096", op="gemm", m=5, n=131072, k=4096, out="f32", bias=False),
        # a small ragged prefill with an odd channel count and a bias
        dict(name="gemm ragged 333x2047x4096", op="gemm", m=333, n=2047, k=4096, out="f16", bias=True),
        # a long prefill chunk
        dict(name="gemm prefill 8192x8192x4096", op="gemm", m=8192, n=8192, k=4096, out="bf16", bias=False),
        # one token, a small vocabulary, a chat's history
        dict(name="logits decode 1x32000", op="logits", rows=1, per=1, vocab=32000, history=600, biases=0,
             mask=False, dtype="f32"),
        # a verify step: 5 columns of one request under one grammar, a long history, biased tokens
        dict(name="logits verify 5x131072", op="logits", rows=5, per=5, vocab=131072, history=8192, biases=300,
             mask=True, dtype="f32"),
        # a serving batch in 16 bits
        dict(name="logits batch 256x131072", op="logits", rows=256, per=1, vocab=131072, history=2048, biases=64,
             mask=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _draw(rng)
    while 3072 in case.values():                            # a size that no workload here has
        case = _draw(rng)
    return case


def _draw(rng):
    op = rng.choice(["norm", "norm", "quant", "gemm", "gemm", "gemm", "logits", "logits"])
    if op == "norm":
        fmt = rng.choice(["i8", "q8_1", "both"])
        k = _log(rng, 200, 16384)
        if fmt != "i8":
            k = max(32, k // 32 * 32)
        rows = min(_log(rng, 1, 16384), 8192 * 8192 // (3 * k))
        return dict(op=op, rows=rows, k=k, dtype=rng.choice(list(DTYPES)), residual=rng.random() < 0.7, fmt=fmt)
    if op == "quant":
        k = _log(rng, 64, 16384)
        if rng.random() < 0.5:
            k = max(64, k // 64 * 64)
        return dict(op=op, rows=min(_log(rng, 1, 16384), (8192 * 2048) // k), k=k, dtype=rng.choice(list(DTYPES)))
    if op == "gemm":
        m, k = _log(rng, 1, 8192), _log(rng, 128, 8192)
        if rng.random() < 0.75:
            k = max(128, k // 64 * 64)
        top = min(131072 if m <= 16 else 16384, 131072 * 4096 // k, 8192 * 8192 * 2048 // (m * k))
        return dict(op=op, m=m, n=min(_log(rng, 64, 131072 if m <= 16 else 16384), top), k=k,
                    out=rng.choice(list(DTYPES)), bias=rng.random() < 0.3)
    vocab = _log(rng, 8000, 160000)
    per = rng.choice([1, 1, 5, 8])
    rows = per * max(1, min(_log(rng, 1, 192), 256 * 131072 // (2 * per * vocab)))
    return dict(op=op, rows=rows, per=per, vocab=vocab, history=_log(rng, 16, 16384 if rows <= 32 else 2048),
                biases=rng.choice([0, 10, 300]), mask=rng.random() < 0.6, dtype=rng.choice(list(DTYPES)))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _codes(shape, gen):
    """int8 codes of normal rows whose largest value has the code 127."""
    q = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
    return q.mul_(30.0).round_().clamp_(-127, 127).to(torch.int8)


def _blocks(xq):
    """Scales, scaled code sums and codes of q8_1 rows, as views of their bytes."""
    b = xq.view(xq.shape[0], -1, 36)
    return b[:, :, 0:2].view(torch.float16), b[:, :, 2:4].view(torch.float16), b[:, :, 4:].view(torch.int8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=gen, device="cuda")
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")
    empty = lambda s, t: torch.empty(s, dtype=t, device="cuda")
    op = case["op"]
    s = {"op": op, "case": case}
    if op in ("norm", "quant"):
        rows, k, t = case["rows"], case["k"], DTYPES[case["dtype"]]
        loud = 1 + 15 * (rand(k) < 0.01)                    # the few loud channels of a residual stream
        s["x"] = (randn(rows, k) * loud).to(t)
        s["q"], s["scale"] = empty((rows, k), torch.int8), empty((rows,), torch.float32)
        if op == "norm":
            s["w"] = (1 + 0.1 * randn(k)).to(t)
            s["residual"] = (4 * randn(rows, k) * loud).to(t) if case["residual"] else None
            s["residual_out"] = empty((rows, k), t) if case["residual"] else None
            s["xq"] = None
            if case["fmt"] != "i8":
                s["xq"] = empty((rows, k // 32 * 36), torch.uint8)
                s["blocks"] = _blocks(s["xq"])
    elif op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["b"] = _codes((m, k), gen), _codes((n, k), gen)
        s["sa"], s["sb"] = 0.01 + 0.03 * rand(m), 4e-4 + 4e-4 * rand(n)
        s["bias"] = randn(n) if case["bias"] else None
        s["out"] = empty((m, n), DTYPES[case["out"]])
    else:
        rows, per, vocab, hist = case["rows"], case["per"], case["vocab"], case["history"]
        requests = rows // per
        s["logits"] = (3 * randn(rows, vocab)).to(DTYPES[case["dtype"]])
        # histories of about `history` tokens, more of the frequent ones; a
        # request's columns share its list, column j seeing j drafts more
        length = (hist * (0.5 + rand(requests))).long() + per
        ends = torch.cumsum(length, 0)
        starts = ends - length
        total = int(ends[-1])
        s["tokens"] = (vocab * rand(total) ** 3).to(torch.int32).clamp_(max=vocab - 1)
        column = torch.arange(rows, device="cuda") % per
        request = torch.arange(rows, device="cuda") // per
        s["begin"] = starts[request].contiguous()
        s["end"] = (ends[request] - (per - 1) + column).contiguous()
        s["prompt_end"] = (starts + length // 2)[request].contiguous()
        s["seen"] = int((s["end"] - s["begin"]).sum())      # the sum of the lengths, known to who schedules
        s["repetition"], s["frequency"], s["presence"] = 1 + 0.2 * rand(rows), 0.5 * rand(rows), 0.5 * rand(rows)
        nb = case["biases"]
        if nb:
            step = vocab // nb                              # distinct ids, in no order of size
            ids = torch.randint(0, step, (rows, nb), generator=gen, device="cuda")
            ids = ids + step * torch.randperm(nb, generator=gen, device="cuda")
            s["bias_ids"] = ids.to(torch.int32).reshape(-1).contiguous()
            s["bias_values"] = 5 * randn(rows * nb)
            s["bias_offsets"] = nb * torch.arange(rows + 1, device="cuda")
        if case["mask"]:
            words = (vocab + 31) // 32
            r = lambda: torch.randint(-2**31, 2**31, (rows, words), generator=gen, device="cuda")
            few = r() & r() & r() & r()                     # a grammar that allows 1 token in 16
            many = r() | r() | r()
            tight = (torch.arange(rows, device="cuda") % 2 == 0)[:, None]
            s["mask"] = torch.where(tight, few, many).to(torch.int32)
        s["out"] = empty((rows, vocab), DTYPES[case["dtype"]])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _quantize(y):
    """(codes, fp32 scale) of the rows y: the fp32 quotients' roundings, halves away from zero."""
    d = (y.abs().amax(-1, keepdim=True).double() / 127).float()
    t = torch.where(d > 0, y.double() / d.double(), 0.0).float().double()
    return torch.trunc(t + torch.copysign(torch.full_like(t, 0.5), t)).to(torch.int8), d


def _plain_norm(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    square = x.double().square().mean(-1, keepdim=True)
    y = x * (1 / (square + EPS).sqrt()).float() * s["w"].float()
    out = {}
    if s["residual"] is not None:
        out["residual"] = x.to(s["x"].dtype)
    fmt = s["case"]["fmt"]
    if fmt != "q8_1":
        out["q"], d = _quantize(y)
        out["scale"] = d[:, 0]
    if fmt != "i8":
        q, d = _quantize(y.view(y.shape[0], -1, 32))
        out["block_d"], out["block_q"] = d.half(), q
        out["block_s"] = (d * q.float().sum(-1, keepdim=True)).half()
    return out


def _plain_logits(s):
    rows, vocab = s["logits"].shape
    z = s["logits"].float()
    dev = z.device
    length = s["end"] - s["begin"]
    row = torch.repeat_interleave(torch.arange(rows, device=dev), length, output_size=s["seen"])
    place = torch.arange(s["seen"], device=dev) - (torch.cumsum(length, 0) - length)[row] + s["begin"][row]
    token = s["tokens"][place].long()
    written = (place >= s["prompt_end"][row]).float()
    count = torch.zeros((rows, vocab), device=dev).index_put_((row, token), written, accumulate=True)
    seen = torch.zeros((rows, vocab), dtype=torch.bool, device=dev)
    seen[row, token] = True
    rep = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = torch.where(count > 0, z - (count * s["frequency"][:, None] + s["presence"][:, None]), z)
    if "bias_ids" in s:
        n = s["bias_ids"].numel() // rows
        ids = s["bias_ids"].view(rows, n).long()
        z = z.scatter_add(1, ids, s["bias_values"].view(rows, n))
    if "mask" in s:
        bit = (s["mask"][:, :, None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
        z = torch.where(bit.view(rows, -1)[:, :vocab] != 0, z, -math.inf)
    return z.to(s["logits"].dtype)


def _plain(s):
    if s["op"] == "norm":
        return _plain_norm(s)
    if s["op"] == "quant":
        q, d = _quantize(s["x"].float())
        return {"q": q, "scale": d[:, 0]}
    if s["op"] == "gemm":
        out = (s["a"].float() @ s["b"].float().t()) * (s["sa"][:, None] * s["sb"])
        if s["bias"] is not None:
            out = out + s["bias"]
        return {"out": out.to(s["out"].dtype)}
    return {"out": _plain_logits(s)}


def _own(s):
    from quantized_moe_expert_q8_amd import ops
    if s["op"] == "norm":
        ops.rms_norm_q8(s["x"], s["w"], eps=EPS, residual=s["residual"], residual_out=s["residual_out"],
                        fmt=s["case"]["fmt"], q=s["q"], scale=s["scale"], xq=s["xq"])
        out = {} if s["residual"] is None else {"residual": s["residual_out"]}
        if s["case"]["fmt"] != "q8_1":
            out["q"], out["scale"] = s["q"], s["scale"]
        if s["case"]["fmt"] != "i8":
            out["block_d"], out["block_s"], out["block_q"] = s["blocks"]
        return out
    if s["op"] == "quant":
        ops.i8_quantize_rows(s["x"], q=s["q"], scale=s["scale"])
        return {"q": s["q"], "scale": s["scale"]}
    if s["op"] == "gemm":
        return {"out": ops.gemm_i8(s["a"], s["sa"], s["b"], s["sb"], bias=s["bias"], out=s["out"])}
    return {"out": ops.logits_process(
        s["logits"], tokens=s["tokens"], begin=s["begin"], end=s["end"], prompt_end=s["prompt_end"],
        repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
        bias_ids=s.get("bias_ids"), bias_values=s.get("bias_values"), bias_offsets=s.get("bias_offsets"),
        mask=s.get("mask"), out=s["out"])}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "quant"):
        rows, k, e = case["rows"], case["k"], BYTES[case["dtype"]]
        fmt = case.get("fmt", "i8")
        n = rows * k * (e * (3 if case.get("residual") else 1))
        n += (rows * (k + 4) if fmt != "q8_1" else 0) + (rows * k // 32 * 36 if fmt != "i8" else 0)
        return {"bytes": n + (e * k if op == "norm" else 0), "flops": (9 if op == "norm" else 4) * rows * k}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + m * n * BYTES[case["out"]] + 4 * (m + n * (2 if case["bias"] else 1)),
                "flops": 2 * m * n * k}
    rows, vocab = case["rows"], case["vocab"]
    n = 2 * rows * vocab * BYTES[case["dtype"]] + rows * (36 + 8 * case["biases"])
    n += 4 * rows // case["per"] * case["history"] + (rows * ((vocab + 31) // 32 * 4) if case["mask"] else 0)
    return {"bytes": n, "flops": 4 * rows * vocab}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        sums = torch.matmul(s["a"].to(torch.float64), s["b"].to(torch.float64).T)
        value = sums * s["sa"].to(torch.float64).unsqueeze(1) * s["sb"].to(torch.float64).unsqueeze(0)
        return {"out": value if s["bias"] is None else value + s["bias"].to(torch.float64)}
    if op == "logits":
        value = s["logits"].to(torch.float64)
        vocab = case["vocab"]
        for r in range(case["rows"]):
            b, p, e = (int(s[n][r]) for n in ("begin", "prompt_end", "end"))
            before = torch.bincount(s["tokens"][b:p], minlength=vocab)
            after = torch.bincount(s["tokens"][p:e], minlength=vocab)
            rep, freq, pres = (float(s[n][r]) for n in ("repetition", "frequency", "presence"))
            v = value[r]
            hit = (before + after) > 0
            v[hit] = torch.maximum(v[hit], v[hit] * 0) / rep + torch.minimum(v[hit], v[hit] * 0) * rep
            v -= freq * after + pres * (after > 0)
            if case["biases"]:
                lo, hi = int(s["bias_offsets"][r]), int(s["bias_offsets"][r + 1])
                v[s["bias_ids"][lo:hi].long()] += s["bias_values"][lo:hi].to(torch.float64)
            if case["mask"]:
                at = torch.arange(vocab, device=v.device)
                v[torch.bitwise_and(s["mask"][r][at // 32].long() >> (at % 32), 1) == 0] = -math.inf
        return {"out": value}
    h = s["x"].to(torch.float64)
    out = {}
    if op == "norm":
        if s["residual"] is not None:
            h = h + s["residual"].to(torch.float64)
            out["residual"] = h
        h = h / torch.sqrt(torch.sum(h * h, 1, keepdim=True) / case["k"] + EPS) * s["w"].to(torch.float64)
    fmt = case.get("fmt", "i8")
    if fmt != "q8_1":                                       # the codes have no value in 64 bits
        out["q"], out["scale"] = None, torch.max(torch.abs(h), 1).values / 127
    if fmt != "i8":
        b = h.reshape(h.shape[0], case["k"] // 32, 32)
        d = torch.max(torch.abs(b), 2, keepdim=True).values / 127
        code = torch.round(b / torch.clamp(d, min=1e-300))
        out["block_d"], out["block_q"], out["block_s"] = d, None, d * torch.sum(code, 2, keepdim=True)
    return out
