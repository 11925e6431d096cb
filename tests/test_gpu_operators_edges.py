"""Edges of the operators around the expert layer on the GPU: rows that are zero
or not finite, biases that repeat in long lists, rows of two tensors in one
buffer, and the forms of the kernels that only larger or odder calls take.

Against the numpy forms, exactly where they take the same fp32 roundings."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_q8_amd as moeq8  # noqa: E402
from oracle import operators_ref as ref  # noqa: E402
from _gpu import DEV, say  # noqa: E402
from test_gpu_operators import (TYPES, check_gemm, check_logits, check_norm, framed, frame_kept,  # noqa: E402
                                logits_inputs, norm_inputs, put, q81_fields, typed)

pytestmark = pytest.mark.gpu


# ---- norm ------------------------------------------------------------------------

@pytest.mark.parametrize("k", [32, 96, 2080, 4096, 9216, 33024])
@pytest.mark.parametrize("eps", [0.0, 1e-80, 1e-6])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_norm_zero_rows(k, eps, dtype):
    """A row of zeros has the scale 0 and zero codes whatever eps is: zeros of
    x alone, and a residual that x cancels."""
    say(f"norm zero rows {k} eps={eps} {dtype}")
    x, w, res = norm_inputs(4, k, k, residual=True)
    x[1] = 0
    res[1] = 0
    res[2] = -x[2]
    (xt, xv), (wt, wv), (rt, rv) = (typed(a, TYPES[dtype]) for a in (x, w, res))
    got = moeq8.rms_norm_q8(xt.to(DEV), wt.to(DEV), eps=eps, residual=rt.to(DEV), fmt="both")
    for r in (1, 2):
        assert float(got.scale[r]) == 0 and not got.q[r].any() and not got.xq[r].any() and not got.residual[r].any()
    _, y = ref.rms_norm_steps(xv, wv, eps, rv)
    q, d = ref.quantize_rows_steps(y)
    assert np.array_equal(got.scale.cpu().numpy(), d) and np.array_equal(got.q.cpu().numpy(), q)
    assert got.scale[0] > 0 and got.scale[3] > 0


def test_norm_rows_below_the_normal_range_without_eps():
    """The reciprocal of their root is past fp32: it stops at the largest value."""
    say("norm tiny rows")
    for k in (33, 100, 4100):
        x, w, _ = norm_inputs(3, k, k, residual=False)
        x[1] = 0
        x[1, ::3] = 1e-44
        x[2] *= 1e-39
        (xt, xv), (wt, wv) = (typed(a, torch.float32) for a in (x, w))
        got = moeq8.rms_norm_q8(xt.to(DEV), wt.to(DEV), eps=0.0)
        _, y = ref.rms_norm_steps(xv, wv, 0.0)
        q, d = ref.quantize_rows_steps(y)
        assert bool(torch.isfinite(got.scale).all())
        assert np.array_equal(got.scale.cpu().numpy(), d) and np.array_equal(got.q.cpu().numpy(), q)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,k", [(7, 64), (7, 1504), (7, 4128), (600, 4128), (7, 33024)])
def test_norm_not_finite_in_every_block(rows, k, dtype):
    """An infinity or a NaN anywhere in a row shows in all its scales and
    blocks, and in no other row's."""
    say(f"norm not finite {rows}x{k} {dtype}")
    t = TYPES[dtype]
    x, w, res = norm_inputs(rows, k, k, residual=True)
    xt, wt, rt = (typed(a, t)[0].to(DEV) for a in (x, w, res))
    want = moeq8.rms_norm_q8(xt, wt, residual=rt, fmt="both")
    bad = {1: np.inf, 2: -np.inf, 4: np.nan}
    for r, v in bad.items():
        xt[r, (r * 37) % k] = v
    rt[5, k - 1] = np.inf
    got = moeq8.rms_norm_q8(xt, wt, residual=rt, fmt="both")
    d, s, q = q81_fields(got.xq, rows)
    wd, ws, wq = q81_fields(want.xq, rows)
    scale = got.scale.cpu().numpy()
    for r in range(rows):
        if r in (1, 2, 4, 5):
            assert np.isnan(scale[r]) and not got.q[r].any()
            assert np.isnan(d[r]).all() and np.isnan(s[r]).all() and not q[r].any()
        else:
            assert scale[r] == float(want.scale[r]) and torch.equal(got.q[r], want.q[r])
            assert np.array_equal(d[r], wd[r]) and np.array_equal(s[r], ws[r]) and np.array_equal(q[r], wq[r])
