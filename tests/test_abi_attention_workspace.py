"""Refusals of the attention workspace with batches that need one, for both
kernels: one byte too little, none, and misaligned (CPU-only: every argument is
checked before anything is enqueued)."""
import ctypes

import pytest

from helpers import ensure_lib

ENOSPACE, EALIGN = 7, 2


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n_tokens,max_q", [(4, 1), (600, 600)])
def test_workspace_refusals(dim, n_tokens, max_q):
    import moe_expert_gb300 as mx
    L = ensure_lib()
    buf = ctypes.create_string_buffer(4096 + 64)
    base = (ctypes.addressof(buf) + 15) // 16 * 16
    kv = mx.PagedKV(type=1, page_size=16, n_kv_heads=2, head_dim=dim, n_pages=8192, page_stride=32 * dim,
                    head_stride=16 * dim, row_stride=dim, k=base, v=base)
    b = mx.Batch(n_seqs=1, n_tokens=n_tokens, max_q=max_q, table_width=8192, table_stride=8192, cu_q=base, ctx_len=base,
                 page_table=base)
    need = L.moex_paged_attention_workspace_bytes(ctypes.byref(kv), ctypes.byref(b), 4)
    assert need > 0 and need % 4 == 0

    def f(ws, n):
        return L.moex_paged_attention(ctypes.c_void_p(base), 4 * dim, ctypes.byref(kv), ctypes.byref(b), 4, 0.125, 0,
                                      ctypes.c_void_p(base), 1, 4 * dim, None, ctypes.c_void_p(ws), n, None)

    assert f(base, need - 1) == ENOSPACE and f(base, 0) == ENOSPACE
    assert f(0, need) == ENOSPACE
    for off in (1, 4, 8):
        assert f(base + off, need) == EALIGN, off
