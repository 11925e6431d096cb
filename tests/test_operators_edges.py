"""Edges of the operators around the expert layer, CPU side."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_q8_amd as moeq8  # noqa: E402
from oracle import operators_ref as ref  # noqa: E402

# fake, never-dereferenced addresses: skipped where a GPU could take a launch
P, Q, R = 0x10000, 0x10000000, 0x20000000
cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host-validation calls use fake pointers")


def test_norm_zero_rows():
    x = np.array([[0, 0, 0], [3, 4, 0]], np.float32)
    for eps in (0.0, 1e-80, 1e-6):
        _, y = ref.rms_norm_steps(x, np.ones(3), eps)
        assert not y[0].any() and np.isfinite(y).all() and y[1, 0] > 0
        _, y64 = ref.rms_norm_def(x, np.ones(3), eps)
        assert not y64[0].any() and np.isfinite(y64).all()
    _, y = ref.rms_norm_steps(np.array([[1e-44, 0]], np.float32), np.ones(2), 0.0)
    assert 0 < y[0, 0] < 1 and y[0, 1] == 0             # the reciprocal stops at the largest value


def test_norm_not_finite_in_every_value():
    x = np.ones((4, 64), np.float32)
    x[1, 40], x[2, 3], x[3, 60] = np.inf, -np.inf, np.nan
    _, y = ref.rms_norm_steps(x, np.ones(64), 1e-6)
    d, _, q = ref.q8_1_steps(y)
    assert np.isfinite(d[0]).all() and np.isnan(d[1:]).all() and not q[1:].any()


@cpu_only
def test_rows_that_take_turns_in_a_buffer_are_no_overlap():
    """Accepted by the host (the launch then fails without a GPU), beside rows
    that do overlap."""
    norm, logits = moeq8.lib().rms_norm_q8, moeq8.lib().logits_process

    def residual(res, rs, out, os, rows=3):
        return norm(P, 200, res, rs, out, os, Q, 0, rows, 64, 1e-6, R, 64, R, None, None)

    def rules(out, stride, rows=3):
        return logits(P, 200, 0, rows, 64, None, 0, None, None, None, None, None, None, None, None, 0, None, None, 0,
                      out, stride, None)

    for off in (64, 100, 136, -64, -136, 264, -264):                # elements, rows 200 apart
        assert residual(Q, 64, P + 4 * off, 200) == rules(P + 4 * off, 200) == -4
        assert residual(P + 4 * off, 200, P + 4 * off, 200) == -4
    for off in (1, 63, 137, 199, 200, -1, -63, -200, 263):
        assert residual(Q, 64, P + 4 * off, 200) == rules(P + 4 * off, 200) == -1
    assert residual(Q, 64, P + 400, 100) == rules(P + 400, 100) == -1               # at another stride
    assert residual(P, 300, P, 500, rows=1) == rules(P, 500, rows=1) == -4          # one row is the same row


@cpu_only
def test_grids_past_32_bits_are_refused():
    """Before a launch (which without a GPU fails with -4)."""
    rows, norm, gemm, logits = (getattr(moeq8.lib(), n) for n in
                                ("i8_quantize_rows", "rms_norm_q8", "gemm_i8", "logits_process"))
    big = 1 << 40
    for n, k, fits in ((1 << 26, 8, False), ((1 << 26) - 4, 8, True), (1 << 24, 4096, False), ((1 << 23) - 1, 8192, True),
                       (1 << 22, 40000, False), ((1 << 22) - 1, 40000, True)):
        assert rows(P, 0, n, k, k, Q + big, k, R + 2 * big, None) == (-4 if fits else -3), (n, k)
    assert norm(P, 8, None, 0, None, 0, Q, 0, 1 << 26, 8, 0.0, Q + big, 8, R + 2 * big, None, None) == -3

    def rules(n, vocab):
        return logits(P, vocab, 2, n, vocab, None, 0, None, None, None, None, None, None, None, None, 0, None, None, 0,
                      Q + big, vocab, None)

    assert rules(1 << 23, 8) == rules(1 << 21, 32000) == -3 and rules((1 << 23) - 1, 8) == -4

    def product(m, n, k):
        return gemm(P, k, Q + big, R + 2 * big, k, Q + big, None, m, n, k, 2, P + 3 * big, n, None)

    # blocks of 512 threads on 256 x 256, of 256 threads on 64 x 64
    assert product(1 << 20, 1 << 20, 64) == product(1 << 18, 1 << 18, 8) == -3
    assert product((1 << 18) - 64, 1 << 18, 8) == -4
