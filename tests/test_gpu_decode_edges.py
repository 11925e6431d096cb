"""Edges of the cache, attention and sampling operators on the GPU: value scales
that say nothing of what a position counts, roundings finer than the outputs',
logits masked by finite values, and the forms of the kernels that only larger
calls take.

Against the numpy forms, tokens and cache exactly, attention within bounds that
count its roundings."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_q8_amd as moeq8  # noqa: E402
from oracle import decode_ref as ref  # noqa: E402
from _gpu import DEV, say  # noqa: E402
from test_gpu_decode_operators import TYPES, attention_bound, make_cache, typed  # noqa: E402

pytestmark = pytest.mark.gpu


def half_step(x, dtype):
    """Half of the distance of neighbouring values of dtype at x."""
    return np.ldexp(torch.finfo(dtype).eps / 2, np.frexp(np.maximum(np.abs(x), 1e-30))[1] - 1)


# ---- attention: what is rounded ----------------------------------------------------

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 40])
def test_attention_bf16_outputs_are_rounded_once(n, d):
    """Within half a step of bf16 of the definition, and what fp32 sums lose.

    The scores are near 0 and all values positive, so that little else is lost: the
    rest of the bound is that of fp32 outputs, some 2^-16 of the value.  A weight
    of 11 bits would be off by up to 2^-11."""
    rng = np.random.default_rng(n + d)
    seqs, heads = 4, 24
    cache, arrays, _ = make_cache(seqs * 3, 1, 16, d, seed=n)
    arrays[2][:] = np.maximum(np.abs(arrays[2]), 1)
    cache.v.copy_(torch.from_numpy(arrays[2]))
    q, qv = typed(1e-3 * rng.standard_normal((seqs, 1, heads, d)), torch.bfloat16)
    table = rng.permutation(seqs * 3).astype(np.int32).reshape(seqs, 3)
    visible = np.full((seqs, 1), n, np.int32)
    got = moeq8.paged_attention_i8(q.to(DEV), cache, torch.from_numpy(table).to(DEV), torch.from_numpy(visible).to(DEV))
    want, sizes = ref.attention(qv, *arrays, table, visible, d ** -0.5)
    rest = attention_bound(want, sizes, torch.float32, d)
    bound = half_step(np.abs(want) + rest, torch.bfloat16) + rest
    err = np.abs(got.float().cpu().numpy() - want)
    say(f"attention of {n}, d {d}: {(err / bound).max():.3f} of the bound, {(err > bound).sum()} of {err.size} past it")
    assert (err <= bound).all()
