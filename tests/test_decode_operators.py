"""The cache, attention and sampling operators, CPU side: the numpy forms are
pinned by worked numbers, and the host rejects bad calls before anything is
enqueued."""

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_q8_amd as moeq8  # noqa: E402
from quantized_moe_expert_q8_amd import _lib, ops  # noqa: E402
from oracle import decode_ref as ref  # noqa: E402

# fake, never-dereferenced addresses: skipped where a GPU could take a launch
P, Q, R, S = 0x10000, 0x10000000, 0x20000000, 0x30000000
cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host-validation calls use fake pointers")


# ---- pins of the numpy forms ------------------------------------------------

def test_cache_worked_numbers():
    k = np.zeros((2, 1, 16, 16), np.int8)
    s = np.zeros((2, 1, 16), np.float32)
    x = np.zeros((3, 1, 16), np.float32)
    x[0, 0, :3] = [12.7, -12.7, 0.05]
    x[1, 0, :2] = [254.0, 3.0]
    ref.cache_write(k, s, x, [17, -1, 5])
    assert s[1, 0, 1] == np.float32(12.7) / np.float32(127) and k[1, 0, 1, :4].tolist() == [127, -127, 1, 0]
    assert not s[0].any() and not k[0].any() and k[1].any(axis=-1).sum() == 1
    out = ref.cache_read(k, s, [17, 32, -1, 17])
    assert np.array_equal(out[0], out[3]) and not out[1:3].any()
    assert out[0, 0, 1] == np.float32(-127) * s[1, 0, 1]


def test_attention_worked_numbers():
    k = np.zeros((2, 1, 16, 16), np.int8)
    v = np.zeros_like(k)
    one = np.ones((2, 1, 16), np.float32)
    k[1, 0, 0, 0], k[1, 0, 1, 0] = 1, 2
    v[1, 0, 0, 0], v[1, 0, 1, 0], v[1, 0, 2, 0] = 10, 20, 99
    q = np.zeros((1, 3, 1, 16))
    q[..., 0] = np.log(3.0)
    out, (absolute, _, largest, count) = ref.attention(q, k, one, v, one, [[1, -1]], [[0, 1, 2]], 1.0)
    # weights 1/4 and 3/4 of the two positions
    assert np.allclose(out[0, :, 0, 0], [0.0, 10.0, 0.25 * 10 + 0.75 * 20])
    assert count[0, :, 0].tolist() == [0, 1, 2] and np.isclose(largest[0, 2, 0], 2 * np.log(3.0))
    assert np.allclose(absolute, np.abs(out))
    # a page outside the cache is not seen
    out2, _ = ref.attention(q, k, one, v, one, [[1, 7]], [[0, 1, 20]], 1.0)
    w = np.array([3.0, 9.0] + [1.0] * 14)
    assert np.isclose(out2[0, 2, 0, 0], (w[:3] @ [10, 20, 99]) / w.sum())


def test_sample_worked_numbers():
    z = np.log([4.0, 1.0, 3.0, 2.0])
    draw = lambda u, **k: ref.sample_row(z, u, **k)[0]
    assert [draw(u) for u in (0.0, 0.39, 0.41, 0.49, 0.51, 0.79, 0.81, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [draw(u, top_k=2) for u in (0.0, 0.56, 0.58, 0.99)] == [0, 0, 2, 2]
    assert [draw(u, top_p=0.71) for u in (0.0, 0.43, 0.45, 0.77, 0.79)] == [0, 0, 2, 2, 3]
    assert [draw(u, top_p=0.5) for u in (0.56, 0.58)] == [0, 2]
    assert draw(0.99, top_p=0.0) == draw(0.99, min_p=0.8) == draw(0.99, temperature=0.0) == 0
    assert [draw(u, min_p=0.6) for u in (0.56, 0.58)] == [0, 2]
    assert ref.sample_row(z, 0.9)[1] == pytest.approx(np.log(0.2))
    assert ref.sample_row(z, 0.0, top_k=2)[1] == pytest.approx(np.log(4 / 7))
    assert ref.sample_row([1.0, 1.0, 1.0], 0.99, top_k=2) == (1, pytest.approx(np.log(0.5)))      # equals by index
    assert ref.sample_row([np.nan, -np.inf], 0.5) == (-1, -np.inf)
    assert ref.sample_row([0.0, np.inf, np.inf], 0.7) == (2, pytest.approx(np.log(0.5)))


# ---- refusals ----------------------------------------------------------------

def cache(**change):
    c = dict(k=P, k_scale=P + 0x100000, v=P + 0x200000, v_scale=P + 0x300000, n_pages=4, n_heads=2, page_size=16, d=32,
             page_stride=1024, head_stride=512, token_stride=32, scale_page_stride=32, scale_head_stride=16)
    c.update(change)
    return ctypes.byref(_lib.KvCache(**c))


BAD_CACHES = [(dict(k=None), -1), (dict(v_scale=None), -1), (dict(n_pages=0), -1), (dict(n_heads=0), -1),
              (dict(d=0), -1), (dict(page_size=0), -1), (dict(page_size=8), -3), (dict(page_size=24), -3),
              (dict(d=40), -3), (dict(d=272, token_stride=272, head_stride=4352, page_stride=8704), -3),
              (dict(token_stride=16), -1), (dict(head_stride=16), -1), (dict(page_stride=16), -1),
              (dict(scale_head_stride=8), -1), (dict(scale_page_stride=8), -1),
              (dict(k=P + 8), -2), (dict(k_scale=P + 4), -2), (dict(token_stride=40), -2), (dict(page_stride=1032), -2),
              (dict(scale_head_stride=18), -2), (dict(n_pages=1 << 31), -3)]


@cpu_only
@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_cache_validation(change, status):
    L, c = moeq8.lib(), cache(**change)
    assert L.kv_cache_write_i8(Q, 64, 32, R, 64, 32, 0, 3, S, c, None) == status
    assert L.kv_cache_read_i8(c, S, 3, 0, Q, 64, 32, R, 64, 32, None) == status
    assert L.paged_attention_i8(Q, 128, 128, 32, 0, 1, 1, 4, c, S, 4, 4, S, 64, 1.0, R, 128, 128, 32, None, 0, None) == status


@cpu_only
def test_cache_rows_validation():
    L = moeq8.lib()

    def write(k=Q, kt=64, kh=32, v=R, vt=64, vh=32, dt=0, n=3, slots=S, c=None):
        a = L.kv_cache_write_i8(k, kt, kh, v, vt, vh, dt, n, slots, c or cache(), None)
        b = L.kv_cache_read_i8(c or cache(), slots, n, dt, k, kt, kh, v, vt, vh, None)
        assert a == b
        return a

    assert write(k=None) == write(v=None) == write(slots=None) == write(dt=3) == write(dt=-1) == write(n=-1) == -1
    assert write(kt=31) == write(kh=31) == write(vt=31) == write(vh=0) == -1
    assert write(k=Q + 2) == write(v=R + 1, dt=2) == write(slots=S + 4) == -2
    assert write(k=P + 16) == write(v=P + 0x300000 - 64) == -1                   # over the cache
    assert write(n=1 << 30) == -3
    assert L.kv_cache_write_i8(Q, 64, 32, R, 64, 32, 0, 3, S, cache(v=P), None) == -1             # values over keys
    assert L.kv_cache_write_i8(Q, 64, 32, R, 64, 32, 0, 3, S, cache(v_scale=P + 0x100000), None) == -1
    assert L.kv_cache_read_i8(cache(), S, 3, 0, Q, 64, 32, Q, 64, 32, None) == -1
    assert write(n=0) == write(n=0, k=None, v=None, slots=None) == 0
    assert L.kv_cache_write_i8(Q, 64, 32, R, 64, 32, 0, 3, S, None, None) == -1


@cpu_only
def test_attention_validation():
    L = moeq8.lib()

    def call(q=Q, qs=128, qc=128, qh=32, dt=0, seqs=2, cols=1, heads=4, c=None, pages=S, row=4, table=4, vis=S, most=64,
             scale=1.0, out=R, os_=128, oc=128, oh=32, ws=None, n=0):
        return L.paged_attention_i8(q, qs, qc, qh, dt, seqs, cols, heads, c or cache(), pages, row, table, vis, most,
                                    scale, out, os_, oc, oh, ws, n, None)

    assert call(q=None) == call(out=None) == call(pages=None) == call(vis=None) == -1
    assert call(dt=3) == call(seqs=-1) == call(cols=0) == call(cols=9) == call(heads=3) == call(heads=0) == -1
    assert call(table=-1) == call(row=3) == call(most=-1) == -1
    assert call(scale=float("nan")) == call(scale=float("inf")) == -1
    assert call(qs=31) == call(qh=16) == call(os_=0) == call(oh=31) == call(cols=2, qc=16) == -1
    assert call(out=Q) == call(out=Q + 512) == call(out=P) == -1                  # over q, over the cache
    assert call(q=Q + 2) == call(out=R + 1, dt=1) == call(pages=S + 2) == call(vis=S + 1) == -2
    assert call(most=1 << 30) == -3
    assert call(c=cache(token_stride=1 << 27, head_stride=1 << 31, page_stride=1 << 33)) == -3
    assert call(seqs=0) == 0
    need = L.paged_attention_workspace_bytes(2, 1, 4, 2, 32, 1 << 16)
    assert need > 0 and L.paged_attention_workspace_bytes(2, 1, 4, 2, 32, 64) == 0
    big = dict(most=1 << 16, table=1 << 12, row=1 << 12)
    assert call(**big) == call(ws=0x50000000, n=need - 1, **big) == -1
    assert call(ws=0x50000008, n=need, **big) == -2
    for bad in ((-1, 1, 4, 2, 32, 64), (2, 9, 4, 2, 32, 64), (2, 1, 3, 2, 32, 64), (2, 1, 4, 0, 32, 64), (2, 1, 4, 2, 40, 1 << 16),
                (2, 1, 4, 2, 32, -1), (2, 1, 4, 2, 32, 1 << 30)):
        assert L.paged_attention_workspace_bytes(*bad) == 0


@cpu_only
def test_sample_validation():
    L = moeq8.lib()
    need = L.logits_sample_workspace_bytes(2, 1000)

    def call(z=Q, zs=1000, dt=0, rows=2, vocab=1000, u=P, t=P, k=P, p=P, m=P, token=R, log=R + 64, ws=0x50000000, n=need):
        return L.logits_sample(z, zs, dt, rows, vocab, u, t, k, p, m, token, log, ws, n, None)

    assert call(z=None) == call(u=None) == call(token=None) == call(dt=3) == call(rows=-1) == call(vocab=-1) == -1
    assert call(zs=999) == -1
    assert call(z=Q + 2) == call(z=Q + 1, dt=2) == call(u=P + 2) == call(t=P + 1) == call(k=P + 2) == call(token=R + 2) == -2
    assert call(log=R + 1) == call(p=P + 2) == call(m=P + 3) == -2
    assert call(vocab=1 << 30, zs=1 << 30) == -3
    assert call(rows=0) == 0


@cpu_only
def test_written_arrays_lie_apart():
    L = moeq8.lib()
    W = 0x50000000
    need = L.logits_sample_workspace_bytes(2, 1000)

    def sample(z=Q, rows=2, u=P, k=P + 64, token=R, log=R + 64, ws=W):
        return L.logits_sample(z, 1000, 0, rows, 1000, u, None, k, None, None, token, log, ws, need, None)

    assert sample(token=Q) == sample(token=Q + 7996) == sample(log=Q + 400) == -1             # in the logits
    assert sample(token=P) == sample(log=P + 68) == sample(u=R + 4) == sample(k=W + 16) == -1
    assert sample(log=R) == sample(log=R + 4) == sample(token=W) == sample(log=W + need - 4) == -1
    assert sample(z=W + need - 16) == sample(ws=Q) == sample(ws=Q - need + 16 * (need % 16 == 0)) == -1

    bytes_ = L.paged_attention_workspace_bytes(2, 1, 4, 2, 32, 1 << 16)

    def attend(ws):
        return L.paged_attention_i8(Q, 128, 128, 32, 0, 2, 1, 4, cache(), S, 1 << 12, 1 << 12, S, 1 << 16, 1.0, R, 128,
                                    128, 32, ws, bytes_, None)

    assert attend(Q) == attend(R) == attend(R + 1008) == attend(P) == -1


def test_ops_refuse_host_tensors():
    c = ops.kv_cache_i8(2, 2, 16, 32, "cpu")
    x, s = torch.zeros(3, 2, 32), torch.zeros(3, dtype=torch.int64)
    i = torch.zeros(1, 1, dtype=torch.int32)
    for f in (lambda: ops.kv_cache_write_i8(x, x, c, s), lambda: ops.kv_cache_read_i8(c, s),
              lambda: ops.paged_attention_i8(x[None], c, i, i), lambda: ops.logits_sample(x[0], x[0, :, 0])):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        ops.kv_cache_read_i8(c.k, s)
