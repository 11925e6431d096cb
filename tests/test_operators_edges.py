"""Edges of the operators around the expert layer, CPU side."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import operators_ref as ref  # noqa: E402


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
