"""Plain numpy forms of the operators around the expert layer, independent of
the HIP code: RMS norm with 8-bit outputs, int8 rows, the int8 product and the
logits rules.

Each has two forms.  ``*_def`` is the definition in 64 bits.  ``*_steps`` takes
the same inputs through the fp32 roundings the operators document (sums of
squares in 64 bits, every other operation rounded to fp32), so codes and fp32
results can be compared exactly.  Inputs are fp32 arrays that hold values of
the element type under test; rounding to that type is the caller's.
"""

from __future__ import annotations

import numpy as np

F32 = np.float32


def _round_half_away(t):
    return np.trunc(t + np.copysign(0.5, t))


def _codes_steps(y, amax):
    """(codes int64, scale fp32) of fp32 values y whose group maxima are amax."""
    with np.errstate(all="ignore"):
        d = (amax / F32(127)).astype(F32)
        ok = (d > 0) & np.isfinite(d)
        t = np.divide(y, d, out=np.zeros(np.broadcast(y, d).shape, F32), where=np.broadcast_to(ok, y.shape))
    q = np.clip(_round_half_away(t.astype(np.float64)), -127, 127).astype(np.int64)
    return q, d


def quantize_rows_steps(x):
    """int8 rows: (codes [rows, k], scale fp32 [rows])."""
    x = np.asarray(x, F32)
    amax = np.max(np.abs(x), axis=1, keepdims=True)           # NaN if any is
    q, d = _codes_steps(x, amax)
    return q, d[:, 0]


def quantize_rows_def(x):
    """(quotients y / scale, scale) in 64 bits; quotients 0 for zero rows."""
    x = np.asarray(x, np.float64)
    d = np.max(np.abs(x), axis=1, keepdims=True) / 127.0
    return np.divide(x, d, out=np.zeros_like(x), where=d > 0), d[:, 0]


def q8_1_steps(y):
    """q8_1 fields of fp32 rows: (d fp16, s fp16, codes) per 32 values."""
    b = np.asarray(y, F32).reshape(y.shape[0], -1, 32)
    q, d = _codes_steps(b, np.max(np.abs(b), axis=2, keepdims=True))
    with np.errstate(all="ignore"):
        s = (d[:, :, 0] * q.sum(2).astype(F32)).astype(F32)
        return d[:, :, 0].astype(np.float16), s.astype(np.float16), q


def rms_norm_steps(x, w, eps, residual=None):
    """(s fp32, y fp32) of the norm."""
    with np.errstate(all="ignore"):
        s = np.asarray(x, F32) if residual is None else (np.asarray(x, F32) + np.asarray(residual, F32)).astype(F32)
        mean = np.sum(s.astype(np.float64) ** 2, axis=1, keepdims=True) / s.shape[1]
        inv = np.minimum((1.0 / np.sqrt(mean + eps)).astype(F32), np.finfo(F32).max)
        inv = np.where(np.isfinite(mean), inv, F32(np.nan))
        return s, ((s * inv).astype(F32) * np.asarray(w, F32)).astype(F32)


def rms_norm_def(x, w, eps, residual=None):
    """(s, y) in 64 bits; y 0 for zero rows."""
    s = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    root = np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    return s, np.divide(s, root, out=np.zeros_like(s), where=root != 0) * np.asarray(w, np.float64)


def gemm_i8_sums(a, b):
    """Exact integer sums [m, n] (a sum of k <= 131071 products is exact in 64-bit floats)."""
    return (np.asarray(a, np.float64) @ np.asarray(b, np.float64).T).astype(np.int64)


def gemm_i8_steps(a, sa, b, sb, bias=None):
    v = gemm_i8_sums(a, b).astype(F32)
    v = (v * np.asarray(sa, F32)[:, None]).astype(F32)
    v = (v * np.asarray(sb, F32)).astype(F32)
    return v if bias is None else (v + np.asarray(bias, F32)).astype(F32)


def gemm_i8_def(a, sa, b, sb, bias=None):
    v = gemm_i8_sums(a, b).astype(np.float64) * np.asarray(sa, np.float64)[:, None] * np.asarray(sb, np.float64)
    return v if bias is None else v + np.asarray(bias, np.float64)


def logits_rules(z, dtype, tokens=None, begin=None, end=None, prompt_end=None, repetition=None, frequency=None,
                 presence=None, bias=None, mask=None):
    """The rules token by token, every operation rounded to ``dtype`` (np.float32:
    the documented steps; np.float64: the definition).  bias: per row a list of
    (id, value); mask: per row the words."""
    f = dtype
    z = np.asarray(z).astype(f).copy()
    rows, vocab = z.shape
    with np.errstate(all="ignore"):
        for r in range(rows):
            if tokens is not None:
                b = min(max(int(begin[r]), 0), len(tokens))
                e = min(max(int(end[r]), b), len(tokens))
                p = b if prompt_end is None else min(max(int(prompt_end[r]), b), e)
                seen, count = set(), {}
                for i in range(b, e):
                    t = int(tokens[i])
                    if 0 <= t < vocab:
                        seen.add(t)
                        if i >= p:
                            count[t] = count.get(t, 0) + 1
                rep = f(1 if repetition is None else repetition[r])
                fr = f(0 if frequency is None else frequency[r])
                pr = f(0 if presence is None else presence[r])
                for t in seen:
                    z[r, t] = f(z[r, t] / rep) if z[r, t] > 0 else f(z[r, t] * rep)
                for t, c in count.items():
                    z[r, t] = f(z[r, t] - f(f(f(c) * fr) + pr))
            if bias is not None:
                for t, v in bias[r]:
                    if 0 <= t < vocab:
                        z[r, t] = f(z[r, t] + f(v))
            if mask is not None:
                bits = (np.asarray(mask[r]).astype(np.int64)[np.arange(vocab) // 32] >> (np.arange(vocab) % 32)) & 1
                z[r, bits == 0] = -np.inf
    return z
