"""Edges of the cache, attention and sampling operators, CPU side: arrays that lie
over one another, and sizes past what a call can index."""

import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_q8_amd as moeq8  # noqa: E402
from test_decode_operators import P, Q, R, S, cache, cpu_only  # noqa: E402

W = 0x50000000


@cpu_only
def test_attention_writes_nothing_that_it_reads():
    """Two sequences of 4096 entries, whose work is split: outputs and workspace over
    the page table, its last entry, or what the columns see."""
    L = moeq8.lib()
    T, V, n = 0x60000000, 0x70000000, 1 << 12
    need = L.paged_attention_workspace_bytes(2, 1, 4, 2, 32, 1 << 16)
    table, seen = 4 * (n + 8 + n), 8

    def call(out=R, ws=W, pages=T, visible=V):
        return L.paged_attention_i8(Q, 128, 128, 32, 0, 2, 1, 4, cache(), pages, n + 8, n, visible, 1 << 16, 1.0, out, 128, 128,
                                    32, ws, need, None)

    fine = call()
    assert fine not in (0, -1, -2, -3)                      # nothing but the missing GPU
    assert call(out=T) == call(out=T + table - 4) == call(out=T - 1020) == -1
    assert call(out=V) == call(out=V + seen - 4) == call(visible=R + 1020) == -1
    assert call(ws=T) == call(pages=W + need - 4) == call(ws=V) == call(visible=W + need - 8) == -1
    assert call(out=Q) == call(ws=Q) == call(ws=R) == call(out=P) == -1
    assert call(out=T + table) == call(out=T - 1024) == call(pages=W + (need + 3) // 4 * 4) == call(visible=V + 4) == fine


def read(k, kt, kh, v, vt, vh, n=5, slots=S, c=None, dt=0):
    return moeq8.lib().kv_cache_read_i8(c or cache(), slots, n, dt, k, kt, kh, v, vt, vh, None)


def write(c, slots=S):
    return moeq8.lib().kv_cache_write_i8(Q, 64, 32, R, 64, 32, 0, 5, slots, c, None)


@cpu_only
def test_cache_rows_read_apart():
    """Outputs [5][2][32] fp32 that overlap partly, and that take turns in a buffer."""
    fine = read(Q, 64, 32, R, 64, 32)
    assert fine not in (0, -1, -2, -3)
    for off in (4, 16, 128, 256, 640, 1276):                # a value, a head, a token, some tokens, the last value
        assert read(Q, 64, 32, Q + off, 64, 32) == read(Q + off, 64, 32, Q, 64, 32) == -1, off
    assert read(Q, 64, 32, Q + 1280, 64, 32) == read(Q + 1280, 64, 32, Q, 64, 32) == fine
    assert read(Q, 128, 32, Q + 256, 128, 32) == fine       # [token][k or v][head]
    assert read(Q, 128, 32, Q + 252, 128, 32) == read(Q, 128, 32, Q + 260, 128, 32) == -1
    assert read(Q, 128, 64, Q + 128, 128, 64) == fine       # [token][head][k or v]
    assert read(Q, 128, 64, Q + 124, 128, 64) == -1
    assert read(Q, 32, 320, Q + 640, 32, 320) == fine       # [head][k or v][token]
    assert read(Q, 64, 320, Q + 128, 64, 320) == fine       # [head][token][k or v]
    assert read(Q, 64, 320, Q + 64, 64, 320) == -1
    # a token's 132 values: heads side by side (64), and 36 apart (68)
    assert read(Q, 132, 32, Q + 256, 132, 36) == fine and read(Q, 131, 32, Q + 256, 131, 36) == -1
    # one token, one head: their strides say nothing
    assert read(Q, 1, 32, Q + 256, 1, 32, n=1) == fine and read(Q, 1, 32, Q + 252, 1, 32, n=1) == -1
    # slots among the outputs
    assert read(Q, 64, 32, R, 64, 32, slots=Q) == read(Q, 64, 32, R, 64, 32, slots=R + 1272) == -1
    assert read(Q, 64, 32, R, 64, 32, slots=Q - 32) == -1 and read(Q, 64, 32, R, 64, 32, slots=Q - 40) == fine


@cpu_only
def test_cache_arrays_written_lie_apart():
    """A cache of 4 pages, 2 heads, 16 places of 32 codes: 4096 bytes of codes, 512 of scales."""
    fine = write(cache())
    assert fine not in (0, -1, -2, -3)
    for change in (dict(v=P + 4080), dict(v=P + 32), dict(v=P - 1024), dict(v_scale=P + 0x100000 + 448), dict(v_scale=P + 0x100000 - 64),
                   dict(k_scale=P + 2048), dict(v_scale=P + 4080), dict(k_scale=P + 0x200000)):
        assert write(cache(**change)) == -1, change
    assert write(cache(v=P + 4096, k_scale=P + 8192, v_scale=P + 8704)) == fine
    # [page][k or v][head][place], [page][head][k or v][place], [page][head][place][k or v]
    assert write(cache(v=P + 1024, page_stride=2048)) == write(cache(v=P + 512, page_stride=2048, head_stride=1024)) == fine
    assert write(cache(v=P + 32, page_stride=2048, head_stride=1024, token_stride=64)) == fine
    assert write(cache(v=P + 16, page_stride=2048, head_stride=1024, token_stride=64)) == -1
    # [page][codes of k, of v, scales of k, of v]
    whole = dict(v=P + 1024, k_scale=P + 2048, v_scale=P + 2176, page_stride=2304, scale_page_stride=576)
    assert write(cache(**whole)) == fine
    assert write(cache(**{**whole, "k_scale": P + 2032})) == write(cache(**{**whole, "page_stride": 2288})) == -1
    # slots in the cache
    assert write(cache(), slots=P + 8) == write(cache(), slots=P + 0x300000 + 504) == write(cache(), slots=P - 32) == -1
    assert write(cache(), slots=P + 4096) == write(cache(), slots=P - 40) == fine


@cpu_only
def test_attention_tables_past_what_positions_count():
    """Entries times the page's size would pass 64 bits: refused before anything is made of them."""
    L = moeq8.lib()
    for n in (1 << 31, 1 << 40, (1 << 59) + 1, 1 << 62):
        assert L.paged_attention_i8(Q, 128, 128, 32, 0, 1, 1, 4, cache(), S, n, n, 0x70000000, 64, 1.0, R, 128, 128, 32, None, 0,
                                    None) == -3
    big = cache(page_size=1 << 20, head_stride=32 << 20, page_stride=64 << 20, scale_head_stride=1 << 20, scale_page_stride=2 << 20)
    assert L.paged_attention_i8(Q, 128, 128, 32, 0, 1, 1, 4, big, 0x60000000, 1 << 44, 1 << 44, 0x70000000, 64, 1.0, R, 128, 128, 32,
                                None, 0, None) == -3
