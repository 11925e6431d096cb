"""The operators around the expert layer, CPU side: the numpy forms are pinned
by worked numbers and by each other, and the host rejects bad calls before
anything is enqueued."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_q8_amd as moeq8  # noqa: E402
from quantized_moe_expert_q8_amd import ops  # noqa: E402
from oracle import operators_ref as ref  # noqa: E402
import oracle  # noqa: E402

# fake, never-dereferenced addresses: skipped where a GPU could take a launch
P, Q, R = 0x10000, 0x10000000, 0x20000000
cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host-validation calls use fake pointers")


# ---- pins of the numpy forms ------------------------------------------------

def test_rows_worked_numbers():
    q, d = ref.quantize_rows_steps(np.array([[127.0, 0.5, -0.5, 1.5, -2.5, 0.49, -127.0]], np.float32))
    assert d[0] == 1.0 and q[0].tolist() == [127, 1, -1, 2, -3, 0, -127]          # halves away from zero
    q, d = ref.quantize_rows_steps(np.zeros((2, 3), np.float32))
    assert not q.any() and not d.any()
    q, d = ref.quantize_rows_steps(np.array([[1.0, np.nan], [1.0, np.inf]], np.float32))
    assert not q.any() and np.isnan(d[0]) and np.isinf(d[1])


def test_rows_steps_follow_the_definition():
    x = np.random.default_rng(3).standard_normal((6, 500)).astype(np.float32)
    q, d = ref.quantize_rows_steps(x)
    t, d64 = ref.quantize_rows_def(x)
    assert np.all(np.abs(d - d64) <= 2.0**-24 * d64)
    # the fp32 scale and quotient move a quotient by two half steps of at most 127
    assert np.all(np.abs(q - t) <= 0.5 + 127 * 2 * 2.0**-24 * 1.01)


def test_q8_1_steps_equal_the_block_oracle():
    x = (np.random.default_rng(4).standard_normal((3, 128)) * 3).astype(np.float32)
    x[1, 32:64] = 0
    d, s, q = ref.q8_1_steps(x)
    blocks = oracle.quantize_q8_1(x)
    assert np.array_equal(blocks["d"].reshape(d.shape).view(np.uint16), d.view(np.uint16))
    assert np.array_equal(blocks["s"].reshape(s.shape).view(np.uint16), s.view(np.uint16))
    assert np.array_equal(blocks["qs"].reshape(q.shape), q)


def test_norm_worked_numbers():
    s, y = ref.rms_norm_steps(np.array([[3.0, 4.0]], np.float32), np.array([1.0, 2.0], np.float32), 0.0,
                              residual=np.array([[0.0, 0.0]], np.float32))
    inv = np.float32(1 / np.sqrt(12.5))
    assert y[0, 0] == np.float32(3) * inv and y[0, 1] == np.float32(np.float32(4) * inv) * np.float32(2)
    _, y64 = ref.rms_norm_def(s, [1.0, 2.0], 0.0)
    assert np.allclose(y, y64, rtol=4 * 2.0**-24)


def test_gemm_worked_numbers():
    a, b = np.array([[1, -2, 3]], np.int8), np.array([[4, 5, 6], [-128, 127, -128]], np.int8)
    assert ref.gemm_i8_sums(a, b).tolist() == [[12, -128 - 254 - 384]]
    out = ref.gemm_i8_def(a, [0.5], b, [2.0, 0.25], [1.0, -1.0])
    assert out.tolist() == [[13.0, -766 * 0.125 - 1.0]]
    assert np.array_equal(ref.gemm_i8_steps(a, [0.5], b, [2.0, 0.25], [1.0, -1.0]), out.astype(np.float32))


def test_logits_worked_numbers():
    z = np.array([[2.0, -2.0, 1.0, 0.0, 5.0]])
    out = ref.logits_rules(z, np.float64, tokens=[0, 1, 2, 2, 9, -1], begin=[0], end=[6], prompt_end=[2],
                           repetition=[2.0], frequency=[0.25], presence=[1.0], bias=[[(3, 4.0), (3, -1.0)]],
                           mask=[[0b01111]])
    # seen 0, 1, 2; written 2 twice; ids 9 and -1 are no tokens; token 4 masked
    assert out.tolist() == [[1.0, -4.0, 0.5 - (0.5 + 1.0), 3.0, -np.inf]]


# ---- refusals ----------------------------------------------------------------

@cpu_only
def test_norm_validation():
    f = moeq8.lib().rms_norm_q8

    def call(x=P, xs=64, res=None, rs=0, ro=None, ros=0, w=Q, dt=0, rows=2, k=64, eps=1e-6, q=R, qs=64, scale=R,
             xq=None):
        return f(x, xs, res, rs, ro, ros, w, dt, rows, k, eps, q, qs, scale, xq, None)

    assert call(x=None) == call(w=None) == -1
    assert call(dt=3) == call(dt=-1) == -1
    assert call(rows=-1) == call(k=0) == call(eps=-1.0) == call(eps=float("nan")) == -1
    assert call(xs=63) == call(qs=63) == -1
    assert call(q=None) == call(scale=None) == call(q=None, scale=None) == -1     # no output, half an output
    assert call(res=Q, rs=64) == call(ro=Q, ros=64) == -1                         # one without the other
    assert call(res=Q, rs=63, ro=R, ros=64) == call(res=Q, rs=64, ro=R, ros=63) == -1
    assert call(res=Q, rs=64, ro=P + 4, ros=64) == -1                             # over x, but not x's rows
    assert call(res=Q, rs=64, ro=Q, ros=65) == -1                                 # over residual at another stride
    assert call(k=48, xs=48, qs=48, xq=R) == -1                                   # q8_1 blocks of 32
    assert call(x=P + 2) == call(scale=R + 2) == call(xq=R + 2) == call(w=Q + 1, dt=2) == -2
    assert call(rows=0) == 0


@cpu_only
def test_rows_validation():
    f = moeq8.lib().i8_quantize_rows
    assert f(None, 0, 2, 64, 64, R, 64, R, None) == -1
    assert f(P, 0, 2, 64, 64, None, 64, R, None) == -1
    assert f(P, 0, 2, 64, 64, R, 64, None, None) == -1
    assert f(P, 3, 2, 64, 64, R, 64, R, None) == -1
    assert f(P, 0, 2, 64, 63, R, 64, R, None) == -1
    assert f(P, 0, 2, 64, 64, R, 63, R, None) == -1
    assert f(P, 0, -1, 64, 64, R, 64, R, None) == -1
    assert f(P + 1, 1, 2, 64, 64, R, 64, R, None) == -2
    assert f(P, 0, 2, 64, 64, R, 64, R + 1, None) == -2
    assert f(P, 0, 0, 64, 64, R, 64, R, None) == 0


@cpu_only
def test_gemm_validation():
    f = moeq8.lib().gemm_i8

    def call(a=P, as_=64, sa=Q, b=P, bs=64, sb=Q, bias=None, m=2, n=3, k=64, dt=0, out=R, os_=3):
        return f(a, as_, sa, b, bs, sb, bias, m, n, k, dt, out, os_, None)

    assert call(a=None) == call(sa=None) == call(b=None) == call(sb=None) == call(out=None) == -1
    assert call(m=-1) == call(n=-1) == call(k=0) == call(dt=3) == -1
    assert call(as_=63) == call(bs=63) == call(os_=2) == -1
    assert call(k=131072, as_=131072, bs=131072) == -3                            # sums past int32
    assert call(sa=Q + 2) == call(sb=Q + 2) == call(bias=Q + 2) == call(out=R + 2) == call(out=R + 1, dt=2) == -2
    assert call(m=0) == call(n=0) == 0


@cpu_only
def test_logits_validation():
    f = moeq8.lib().logits_process

    def call(z=P, zs=64, dt=0, rows=2, vocab=64, tok=Q, nt=8, b=Q, e=Q, p=Q, rep=Q, fr=Q, pr=Q, ids=Q, val=Q, nb=4,
             off=Q, mask=Q, ms=2, out=R, os_=64):
        return f(z, zs, dt, rows, vocab, tok, nt, b, e, p, rep, fr, pr, ids, val, nb, off, mask, ms, out, os_, None)

    assert call(z=None) == call(out=None) == call(dt=3) == call(rows=-1) == call(vocab=-1) == -1
    assert call(zs=63) == call(os_=63) == call(ms=1) == call(nt=-1) == call(nb=-1) == -1
    assert call(b=None) == call(e=None) == call(tok=None) == -1                   # lists without bounds, bounds without lists
    assert call(val=None) == call(off=None) == call(ids=None) == -1
    assert call(out=P + 64) == call(out=P, os_=65) == -1                          # over logits, but not its rows
    assert call(nt=1 << 30) == -3
    assert call(vocab=1 << 31, zs=1 << 31, os_=1 << 31, ms=1 << 26) == -3
    assert call(z=P + 2) == call(out=R + 1, dt=1) == call(tok=Q + 1) == call(mask=Q + 2) == call(val=Q + 2) == -2
    assert call(b=Q + 4) == call(off=Q + 4) == -2
    assert call(rows=0) == call(vocab=0) == 0


def test_ops_refuse_host_tensors():
    x, w = torch.zeros(2, 64), torch.zeros(64)
    c = torch.zeros(2, 64, dtype=torch.int8)
    for f in (lambda: ops.rms_norm_q8(x, w), lambda: ops.i8_quantize_rows(x),
              lambda: ops.gemm_i8(c, w[:2], c, w[:2]), lambda: ops.logits_process(x)):
        with pytest.raises(ValueError):
            f()


def test_matrix_and_vector_checks():
    t = torch.zeros(4, 6)
    assert ops._matrix(t, "t", torch.float32, -1, 4, 6) == 6
    assert ops._matrix(t[:, :5], "t", torch.float32, -1, 4, 5) == 6
    assert ops._matrix(t[:1], "t", torch.float32, -1, 1, 6) == 6
    for bad in (t.t(), t[:, ::2], t[0], t[:3]):
        with pytest.raises(ValueError):
            ops._matrix(bad, "t", torch.float32, -1, 4, 6)
    with pytest.raises(ValueError):
        ops._matrix(t.t(), "t", torch.float32, -1, 6, 4)                          # columns apart
    with pytest.raises(TypeError):
        ops._matrix(t, "t", torch.float16, -1, 4, 6)
    with pytest.raises(ValueError):
        ops._matrix(t, "t", torch.float32, 0, 4, 6)                               # another device
    with pytest.raises(ValueError):
        ops._vector(t[:, 0], "t", torch.float32, -1, 4)
    with pytest.raises(ValueError):
        ops._vector(t[0], "t", torch.float32, -1, 5)
    with pytest.raises(TypeError):
        ops._vector(t[0], "t", torch.int32, -1, 6)


def test_compiled_checks_name_the_argument():
    t, f = torch.zeros(4, 6), torch.float32
    for err, words, call in [
            (ValueError, "t must be a device tensor", lambda: ops._matrix(None, "t", f, -1, 4, 6)),
            (ValueError, "t must be a device tensor", lambda: ops._vector([1.0], "t", f, -1, 1)),
            (TypeError, "t must be torch.float16, got torch.float32", lambda: ops._matrix(t, "t", torch.float16, -1, 4, 6)),
            (ValueError, r"t must be \[4, 7\], got \[4, 6\]", lambda: ops._matrix(t, "t", f, -1, 4, 7)),
            (ValueError, "t must have unit inner stride", lambda: ops._vector(t[:, 0], "t", f, -1, 4)),
            (ValueError, "logits must be a device tensor", lambda: ops.logits_process(None)),
            (ValueError, "a must be a device tensor", lambda: ops.gemm_i8(t.to(torch.int8), t[0], None, t[0])),
            (TypeError, "not a torch dtype", lambda: ops._vector(t[0], "t", 3, -1, 6))]:
        with pytest.raises(err, match=words):
            call()
