"""Timed cases of the operators that take a verify or decode step from its
hidden states to its tokens: writing keys and values into a paged int8 cache
(kv_cache_write_i8), reading rows back (kv_cache_read_i8), attention of a step's
columns over the cache (paged_attention_i8), and the draw of a token with
temperature, top-k, top-p and min-p from given random numbers (logits_sample).

run() computes each in its plain form, elementary torch operations in 32 bits,
or with ``own`` true by the library's calls.  Quotients that decide an 8-bit
code and the sums that decide a token are taken in 64 bits.  Codes are returned
as the signed integers they are, each beside its scale."""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the verify step's 5 columns entering the cache, fp32 as its activations are
        dict(name="write verify 5x8x128", op="write", tokens=5, kv=8, d=128, page=16, dtype="f32"),
        # a prefill chunk in 16 bits
        dict(name="write prefill 8192x8x128", op="write", tokens=8192, kv=8, d=128, page=64, dtype="bf16"),
        # a short prefix read back, few heads of an odd length
        dict(name="read short 300x4x80", op="read", tokens=300, kv=4, d=80, page=16, dtype="f16"),
        # a long prefix shared by requests, read back for a prefill in 16 bits
        dict(name="read prefix 65536x8x128", op="read", tokens=65536, kv=8, d=128, page=64, dtype="bf16"),
        # one token of a short chat: latency alone
        dict(name="attend decode 1x1x777", op="attend", seqs=1, cols=1, heads=32, kv=8, d=128, page=16, length=777,
             dtype="bf16"),
        # the verify step's 5 columns of one request in a long context
        dict(name="attend verify 1x5x32768", op="attend", seqs=1, cols=5, heads=32, kv=8, d=128, page=64,
             length=32768, dtype="bf16"),
        # a serving batch of one token each, lengths from a quarter of the longest on
        dict(name="attend batch 64x1x8192", op="attend", seqs=64, cols=1, heads=32, kv=8, d=128, page=64,
             length=8192, dtype="bf16"),
        # a ragged batch with drafts, an odd head size, a padded request
        dict(name="attend ragged 37x5x1500", op="attend", seqs=37, cols=5, heads=20, kv=4, d=80, page=16,
             length=1500, dtype="f16"),
        # wide heads, 8 columns and many query heads a key head, fp32 throughout
        dict(name="attend wide 16x8x4096", op="attend", seqs=16, cols=8, heads=16, kv=2, d=256, page=32,
             length=4096, dtype="f32"),
        # one token of a chat, a small vocabulary, top-k
        dict(name="sample decode 1x32000", op="sample", rows=1, vocab=32000, top_k=50, top_p=False, min_p=False,
             mixed=False, dtype="f32"),
        # the verify step's 5 columns with top-p and min-p over the whole vocabulary
        dict(name="sample verify 5x131072", op="sample", rows=5, vocab=131072, top_k=0, top_p=True, min_p=True,
             mixed=False, dtype="f32"),
        # a serving batch in 16 bits, each request with rules of its own, some greedy
        dict(name="sample batch 256x131072", op="sample", rows=256, vocab=131072, top_k=200, top_p=True, min_p=True,
             mixed=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "sample", "sample"])
    dtype = rng.choice(list(DTYPES))
    page = rng.choice([16, 16, 32, 64, 128, 256])
    if op in ("write", "read"):
        kv, d = rng.choice([1, 2, 3, 4, 8, 16]), 16 * rng.randint(1, 16)
        most = min(8192 * 8 * 128 if op == "write" else 65536 * 8 * 64, (1 << 30)) // (kv * d)
        return dict(op=op, tokens=min(_log(rng, 1, 65536), most), kv=kv, d=d, page=page, dtype=dtype)
    if op == "attend":
        kv, d = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128, 128, 16 * rng.randint(1, 16)])
        cols = rng.choice([1, 1, 2, 3, 5, 8])
        group = min(_log(rng, 1, 16), 64 // cols)
        length, seqs = _log(rng, 1, 65536), _log(rng, 1, 128)
        while seqs > 1 and seqs * length * kv * d > 64 * 4096 * 8 * 128:
            seqs //= 2
        while length > 1 and seqs * length * kv * d > 64 * 4096 * 8 * 128:
            length //= 2
        return dict(op=op, seqs=seqs, cols=cols, heads=kv * group, kv=kv, d=d, page=page, length=length, dtype=dtype)
    vocab = _log(rng, 1000, 160000)
    return dict(op=op, rows=max(1, min(_log(rng, 1, 256), 200 * 131072 // vocab)), vocab=vocab,
                top_k=rng.choice([0, 0, 20, 50, 200, 1000]), top_p=rng.random() < 0.5, min_p=rng.random() < 0.4,
                mixed=rng.random() < 0.3, dtype=dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """Tokens in the cache of each sequence, the new columns among them: from a
    quarter of the longest on, the longest itself, and of 8 or more one padded
    entry without any."""
    out = [max(1, int(case["length"] * (0.25 + 0.75 * (i * 0.6180339887 % 1.0)))) for i in range(case["seqs"])]
    out[-1] = case["length"]
    if case["seqs"] >= 8:
        out[0] = 0
    return out


def _padded(case):
    """Entries of a write's or a read's list of slots: padded to whole eights, as a captured step's would be."""
    return (case["tokens"] + 7) // 8 * 8


def _rows(shape, gen, dtype):
    """Keys or values: normal, with the few loud channels that heads have."""
    loud = 1 + 7 * (torch.rand(shape[-1], generator=gen, device="cuda") < 0.04)
    return (torch.randn(shape, generator=gen, device="cuda") * loud).to(dtype)


def _filled(pages, case, gen):
    """A cache in use: codes of normal rows, the scales that such rows have."""
    kv, page, d = case["kv"], case["page"], case["d"]
    out = []
    for _ in range(2):
        codes = torch.randn((pages, kv, page, d), generator=gen, device="cuda", dtype=torch.float16)
        out.append(codes.mul_(40.0).round_().clamp_(-127, 127).to(torch.int8))
        out.append(0.015 + 0.02 * torch.rand((pages, kv, page), generator=gen, device="cuda"))
    return out                                              # k, k_scale, v, v_scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=gen, device="cuda")
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")
    perm = lambda n: torch.randperm(n, generator=gen, device="cuda")
    op = case["op"]
    s = {"op": op, "case": case}
    if op == "sample":
        rows, vocab = case["rows"], case["vocab"]
        # a broad base, and the few tokens that a model finds likely
        z = 2 * randn(rows, vocab) + (rand(rows, vocab) < 60 / vocab) * 9 * rand(rows, vocab)
        s["logits"], s["u"] = z.to(DTYPES[case["dtype"]]), rand(rows)
        on = lambda: (rand(rows) < 0.5) if case["mixed"] else torch.ones(rows, dtype=torch.bool, device="cuda")
        s["temperature"] = 0.5 + 0.8 * rand(rows)
        if case["mixed"]:
            s["temperature"] *= rand(rows) > 0.06           # some greedy
        k = torch.randint(1, case["top_k"] + 1, (rows,), generator=gen, device="cuda") if case["top_k"] else None
        s["top_k"] = torch.where(on(), k, 0).to(torch.int32) if case["top_k"] else None
        s["top_p"] = torch.where(on(), 0.7 + 0.29 * rand(rows), 1.0) if case["top_p"] else None
        s["min_p"] = torch.where(on(), 0.01 + 0.1 * rand(rows), 0.0) if case["min_p"] else None
        s["token"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        s["logprob"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    else:
        kv, d, page, t = case["kv"], case["d"], case["page"], DTYPES[case["dtype"]]
        if op == "attend":
            lengths = _lengths(case)
            count = [-(-n // page) for n in lengths]
            used = sum(count)
            pages = used + 3
            s["k"], s["k_scale"], s["v"], s["v_scale"] = _filled(pages, case, gen)
            table = torch.full((case["seqs"], max(count) + 1), -1, dtype=torch.int32)
            free = perm(pages).to(torch.int32).cpu()
            at = 0
            for i, n in enumerate(count):
                table[i, :n] = free[at:at + n]
                at += n
            cols = case["cols"]
            seen = torch.tensor(lengths)[:, None] - (cols - 1 - torch.arange(cols))[None, :]
            s["pages"], s["visible"] = table.cuda(), seen.clamp(min=0).to(torch.int32).cuda()
            s["q"] = (1.5 * randn(case["seqs"], cols, case["heads"], d)).to(t)
            s["out"] = torch.empty_like(s["q"])
        else:
            n, total = case["tokens"], _padded(case)
            count = -(-n // page)
            pages = 2 * count + 1
            s["k"], s["k_scale"], s["v"], s["v_scale"] = _filled(pages, case, gen)
            place = torch.arange(total, device="cuda")
            slots = perm(pages)[(place // page).clamp(max=pages - 1)] * page + place % page
            s["slots"] = torch.where(place < n, slots, -1)
            if op == "write":
                s["new_k"], s["new_v"] = _rows((total, kv, d), gen, t), _rows((total, kv, d), gen, t)
            else:
                s["k_out"] = torch.empty((total, kv, d), dtype=t, device="cuda")
                s["v_out"] = torch.empty((total, kv, d), dtype=t, device="cuda")
    if own:
        from quantized_moe_expert_q8_amd import ops
        if op == "sample":
            s["workspace"] = torch.empty(ops.logits_sample_workspace_bytes(rows, vocab), dtype=torch.uint8, device="cuda")
        else:
            s["cache"] = ops.KVCacheI8(s["k"], s["k_scale"], s["v"], s["v_scale"])
            if op == "attend":
                n = ops.paged_attention_workspace_bytes(case["seqs"], case["cols"], case["heads"], kv, d, case["length"])
                s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _quantize(y):
    """(codes, fp32 scale) of the rows y: the fp32 quotients' roundings, halves away from zero."""
    d = (y.abs().amax(-1, keepdim=True).double() / 127).float()
    t = torch.where(d > 0, y.double() / d.double(), 0.0).float().double()
    return torch.trunc(t + torch.copysign(torch.full_like(t, 0.5), t)).to(torch.int8), d[..., 0]


def _plain_write(s):
    n, page = s["case"]["tokens"], s["case"]["page"]
    at, off = s["slots"][:n] // page, s["slots"][:n] % page
    for name in ("k", "v"):
        q, d = _quantize(s["new_" + name][:n].float())
        s[name][at, :, off] = q
        s[name + "_scale"][at, :, off] = d
    return {name: s[name] for name in ("k", "k_scale", "v", "v_scale")}


def _plain_read(s):
    page = s["case"]["page"]
    real = (s["slots"] >= 0)[:, None, None]
    slot = s["slots"].clamp(min=0)
    out = {}
    for name in ("k", "v"):
        rows = s[name][slot // page, :, slot % page].float() * s[name + "_scale"][slot // page, :, slot % page][..., None]
        out[name] = torch.where(real, rows, 0.0).to(s["k_out"].dtype)
    return out


def _plain_attend(s):
    c = s["case"]
    seqs, cols, heads, kv, d = c["seqs"], c["cols"], c["heads"], c["kv"], c["d"]
    table = s["pages"].long().clamp(min=0)

    def rows(name):                                         # [seqs, kv, positions, d]
        x = s[name][table].float() * s[name + "_scale"][table][..., None]
        return x.transpose(1, 2).reshape(seqs, kv, -1, d)
    k = rows("k")
    q = s["q"].float().view(seqs, cols, kv, heads // kv, d).permute(0, 2, 1, 3, 4).reshape(seqs, kv, -1, d)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * d ** -0.5
    del k
    seen = torch.arange(score.shape[-1], device="cuda") < s["visible"][:, :, None]       # [seqs, cols, positions]
    seen = seen[:, None, :, None, :].expand(seqs, kv, cols, heads // kv, -1).reshape(score.shape)
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - torch.where(top == -math.inf, 0.0, top)), 0.0)
    out = torch.matmul(p, rows("v")) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    out = out.view(seqs, kv, cols, heads // kv, d).permute(0, 2, 1, 3, 4).reshape(seqs, cols, heads, d)
    return {"out": out.to(s["q"].dtype)}


def _plain_sample(s):
    z = s["logits"].double()
    rows, vocab = z.shape
    z, order = torch.sort(z, dim=-1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    w = torch.exp((z - z[:, :1]) / torch.where(t > 0, t, 1.0))
    rank = torch.arange(vocab, device="cuda")[None, :]
    w = torch.where((t > 0) | (rank == 0), w, 0.0)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        w = torch.where((k <= 0) | (rank < k), w, 0.0)
    keep = torch.ones_like(w, dtype=torch.bool)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        before = torch.cumsum(w, -1) - w
        keep = (p >= 1) | (before < p * w.sum(-1, keepdim=True)) | (rank == 0)
    if s["min_p"] is not None:
        keep &= (w >= s["min_p"].double()[:, None]) | (rank == 0)
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    mass = torch.cumsum(kept, -1)
    total = mass[:, -1:]
    last = torch.where(kept > 0, rank, 0).amax(-1)
    token = torch.minimum((mass <= s["u"].double()[:, None] * total).sum(-1), last)
    logprob = torch.log(kept.gather(1, token[:, None]) / total)[:, 0]
    return {"token": token.to(torch.int32), "logprob": logprob.float()}


def _own(s):
    from quantized_moe_expert_q8_amd import ops
    op = s["op"]
    if op == "write":
        ops.kv_cache_write_i8(s["new_k"], s["new_v"], s["cache"], s["slots"])
        return {name: s[name] for name in ("k", "k_scale", "v", "v_scale")}
    if op == "read":
        k, v = ops.kv_cache_read_i8(s["cache"], s["slots"], k_out=s["k_out"], v_out=s["v_out"])
        return {"k": k, "v": v}
    if op == "attend":
        return {"out": ops.paged_attention_i8(s["q"], s["cache"], s["pages"], s["visible"],
                                              max_visible=s["case"]["length"], out=s["out"], workspace=s["workspace"])}
    token, logprob = ops.logits_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                       top_p=s["top_p"], min_p=s["min_p"], token=s["token"], logprob=s["logprob"],
                                       workspace=s["workspace"])
    return {"token": token, "logprob": logprob}


def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend, "sample": _plain_sample}[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * e + 24 * case["rows"], "flops": 4 * n}
    kv, d = case["kv"], case["d"]
    if op == "attend":
        total = sum(_lengths(case))
        q = case["seqs"] * case["cols"] * case["heads"] * d
        return {"bytes": total * kv * 2 * (d + 4) + 2 * q * e + total // case["page"] * 4 + case["seqs"] * case["cols"] * 4,
                "flops": 4 * total * case["cols"] * case["heads"] * d}
    n = case["tokens"] * kv * 2
    return {"bytes": n * (d * e + d + 4) + 8 * _padded(case), "flops": (4 if op == "write" else 1) * n * d}


def _exact_sample(s):
    z = s["logits"].to(torch.float64).cpu().numpy()
    host = lambda name, off: [off] * len(z) if s[name] is None else s[name].cpu().tolist()
    temperature, top_k, top_p, min_p = host("temperature", 1.0), host("top_k", 0), host("top_p", 1.0), host("min_p", 0.0)
    u = s["u"].cpu().tolist()
    tokens, logs = [], []
    for r, row in enumerate(z):
        best = int(np.argmax(row))
        if temperature[r] == 0:
            tokens.append(best)
            logs.append(0.0)
            continue
        weight = np.exp((row - row[best]) / temperature[r])
        ranked = np.argsort(-row, kind="stable")
        if top_k[r] > 0:
            ranked = ranked[:top_k[r]]
        if top_p[r] < 1:
            sums = np.cumsum(weight[ranked])
            ranked = ranked[:1 + int(np.searchsorted(sums, top_p[r] * sums[-1], side="left"))]
        ranked = np.sort(ranked[weight[ranked] >= min(min_p[r], 1.0)])
        sums = np.cumsum(weight[ranked])
        i = min(int(np.searchsorted(sums, u[r] * sums[-1], side="right")), len(ranked) - 1)
        tokens.append(int(ranked[i]))
        logs.append(float(np.log(weight[ranked[i]] / sums[-1])))
    return {"token": torch.tensor(tokens, dtype=torch.int32), "logprob": torch.tensor(logs, dtype=torch.float64)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sample":
        return _exact_sample(s)
    page = case["page"]
    if op == "write":                                       # the codes have no value in 64 bits
        out = {"k": None, "v": None}
        for name in ("k", "v"):
            scale = s[name + "_scale"].to(torch.float64).transpose(1, 2).reshape(-1, case["kv"])
            scale[s["slots"][:case["tokens"]]] = torch.max(torch.abs(s["new_" + name][:case["tokens"]].double()), 2).values / 127
            out[name + "_scale"] = scale.view(-1, page, case["kv"]).transpose(1, 2)
        return out
    if op == "read":
        out = {}
        for name in ("k", "v"):
            codes = s[name].permute(0, 2, 1, 3).reshape(-1, case["kv"], case["d"])
            scale = s[name + "_scale"].permute(0, 2, 1).reshape(-1, case["kv"], 1)
            value = codes[s["slots"]].to(torch.float64) * scale[s["slots"]].to(torch.float64)
            value[case["tokens"]:] = 0
            out[name] = value
        return out
    value = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv"]
    for i, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        at = torch.arange(n, device="cuda")
        where, off = s["pages"][i].long()[at // page], at % page
        seen = at[None, :] < s["visible"][i].long()[:, None]                             # [cols, n]
        for h in range(case["kv"]):
            k, v = (s[x][where, h, off].to(torch.float64) * s[x + "_scale"][where, h, off].to(torch.float64)[:, None]
                    for x in ("k", "v"))
            for a in range(h * group, (h + 1) * group):
                score = s["q"][i, :, a].to(torch.float64) @ k.T / math.sqrt(case["d"])
                p = torch.softmax(score.masked_fill(~seen, -1e300), -1) * seen
                value[i, :, a] = p @ v
    return {"out": value}
