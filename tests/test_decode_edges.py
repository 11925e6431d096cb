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
