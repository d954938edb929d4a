"""Refusals of the operators around a layer's products: bad arguments are
rejected on the host before anything is enqueued (CPU-only)."""
import ctypes

import pytest

from helpers import ensure_lib

NULL = ctypes.c_void_p(0)
EINVAL, EALIGN, EUNSUPPORTED, ENOSPACE = 1, 2, 3, 7


def _p():
    buf = ctypes.create_string_buffer(4096 + 64)
    base = (ctypes.addressof(buf) + 15) // 16 * 16
    return buf, base, ctypes.c_void_p(base), ctypes.c_void_p(base + 4)


def test_norm_refusals():
    L = ensure_lib()
    buf, base, p, odd = _p()

    def f(x=p, xt=0, ldx=64, r=p, ldr=64, g=p, eps=1e-6, T=1, H=64, s=p, lds=64, y=p, yt=1, ldy=64, q=p, ds=p):
        return L.moex_add_rms_norm(x, xt, ldx, r, ldr, g, eps, T, H, s, lds, y, yt, ldy, q, ds, NULL)

    assert f(x=NULL) == EINVAL and f(g=NULL) == EINVAL
    assert f(s=NULL, y=NULL, q=NULL, ds=NULL) == EINVAL          # nothing asked for
    assert f(q=NULL) == EINVAL and f(ds=NULL) == EINVAL          # q and ds together
    assert f(xt=7) == EUNSUPPORTED and f(yt=7) == EUNSUPPORTED
    assert f(T=0) == EINVAL and f(H=48) == EINVAL and f(H=0) == EINVAL
    assert f(H=32800, ldx=32800, ldr=32800, lds=32800, ldy=32800) == EUNSUPPORTED
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert f(eps=eps) == EINVAL
    assert f(ldx=60) == EINVAL and f(ldr=60) == EINVAL and f(lds=60) == EINVAL and f(ldy=60) == EINVAL
    assert f(ldx=66) == EALIGN and f(ldy=66) == EALIGN
    for name in ("x", "r", "g", "s", "y", "q", "ds"):
        assert f(**{name: odd}) == EALIGN, name


def test_dequantize_refusals():
    L = ensure_lib()
    buf, base, p, odd = _p()
    f = lambda q=p, ds=p, T=1, K=64, y=p, t=0: L.moex_dequantize_q8_1(q, ds, T, K, y, t, NULL)  # noqa: E731
    assert f(q=NULL) == EINVAL and f(y=NULL) == EINVAL and f(T=0) == EINVAL and f(K=40) == EINVAL
    assert f(t=3) == EUNSUPPORTED
    assert f(q=odd) == EALIGN and f(ds=odd) == EALIGN and f(y=odd) == EALIGN


def test_route_refusals():
    L = ensure_lib()
    buf, base, p, odd = _p()

    def f(x=p, t=0, ld=64, T=2, E=64, k=4, score=0, groups=1, top=1, gt=1, scale=1.0, ids=p, w=p):
        return L.moex_route_experts(x, t, ld, NULL, T, E, k, score, groups, top, gt, 1, scale, ids, w, NULL)

    assert f(x=NULL) == EINVAL and f(ids=NULL) == EINVAL and f(w=NULL) == EINVAL
    assert f(t=5) == EUNSUPPORTED and f(score=2) == EUNSUPPORTED
    assert f(T=0) == EINVAL and f(E=1025, ld=1025) == EINVAL and f(ld=63) == EINVAL
    assert f(k=0) == EINVAL and f(k=17) == EINVAL and f(E=3, k=4) == EINVAL
    assert f(groups=5) == EINVAL and f(groups=0) == EINVAL and f(groups=64, E=64) == EINVAL
    assert f(groups=8, top=9) == EINVAL and f(groups=8, top=0) == EINVAL
    assert f(groups=8, top=1, k=9) == EINVAL                      # more than the groups hold
    assert f(groups=8, top=2, gt=3) == EINVAL and f(groups=32, E=32, top=8, gt=2) == EINVAL
    assert f(scale=float("nan")) == EINVAL


def _kv(mx, base, **kw):
    d = dict(type=1, page_size=16, n_kv_heads=2, head_dim=64, n_pages=4, page_stride=2048, head_stride=1024,
             row_stride=64, k=base, v=base)
    d.update(kw)
    return mx.PagedKV(**d)


def _batch(mx, base, **kw):
    d = dict(n_seqs=1, n_tokens=4, max_q=4, table_width=4, table_stride=4, cu_q=base, ctx_len=base, page_table=base)
    d.update(kw)
    return mx.Batch(**d)


BAD_KV = [(dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(type=0), EUNSUPPORTED), (dict(n_kv_heads=0), EINVAL),
          (dict(n_pages=0), EINVAL), (dict(page_size=12), EUNSUPPORTED), (dict(page_size=4), EUNSUPPORTED),
          (dict(page_size=2048), EUNSUPPORTED), (dict(row_stride=60), EALIGN), (dict(page_stride=-8), EINVAL)]
BAD_BATCH = [(dict(cu_q=None), EINVAL), (dict(ctx_len=None), EINVAL), (dict(page_table=None), EINVAL),
             (dict(n_seqs=0), EINVAL), (dict(n_tokens=0), EINVAL), (dict(max_q=0), EINVAL), (dict(max_q=5), EINVAL),
             (dict(table_width=0), EINVAL), (dict(table_stride=-1), EINVAL), (dict(table_width=1 << 28), EUNSUPPORTED)]


def test_write_refusals():
    import moe_expert_gb300 as mx
    L = ensure_lib()
    buf, base, p, odd = _p()

    def f(kv=None, b=None, x=p, t=0, ld=512, h=4, cs=p, n_pos=64, rot=64, q=p, ldq=256):
        kv, b = kv or _kv(mx, base), b or _batch(mx, base)
        return L.moex_rope_kv_write(x, t, ld, ctypes.byref(kv), ctypes.byref(b), h, cs, n_pos, rot, 0, q, ldq, NULL)

    for kw, want in BAD_KV:
        assert f(kv=_kv(mx, base, **kw)) == want, kw
    for kw, want in BAD_BATCH:
        assert f(b=_batch(mx, base, **kw)) == want, kw
    assert f(x=NULL) == EINVAL and f(q=NULL) == EINVAL and f(h=0) == EINVAL and f(t=9) == EUNSUPPORTED
    assert f(rot=24) == EUNSUPPORTED and f(rot=80) == EINVAL and f(rot=0) == EINVAL and f(cs=NULL) == EINVAL
    assert f(kv=_kv(mx, base, head_dim=72)) == EUNSUPPORTED and f(n_pos=0) == EINVAL
    assert f(ld=511) == EINVAL and f(ldq=255) == EINVAL and f(ld=516) == EALIGN
    assert f(x=odd) == EALIGN and f(q=odd) == EALIGN and f(cs=odd) == EALIGN


def test_attention_refusals():
    import moe_expert_gb300 as mx
    L = ensure_lib()
    buf, base, p, odd = _p()
    big = 1 << 40

    def f(kv=None, b=None, q=p, ldq=256, h=4, scale=0.125, window=0, out=p, ot=1, ldo=256, ws=p, n=big):
        kv, b = kv or _kv(mx, base), b or _batch(mx, base)
        return L.moex_paged_attention(q, ldq, ctypes.byref(kv), ctypes.byref(b), h, scale, window, out, ot, ldo, NULL,
                                      ws, n, NULL)

    for kw, want in BAD_KV:
        assert f(kv=_kv(mx, base, **kw)) == want, kw
    for kw, want in BAD_BATCH:
        assert f(b=_batch(mx, base, **kw)) == want, kw
    assert f(q=NULL) == EINVAL and f(out=NULL) == EINVAL and f(h=3) == EINVAL and f(h=0) == EINVAL
    assert f(h=2 * 129, ldq=1 << 20, ldo=1 << 20) == EINVAL
    assert f(kv=_kv(mx, base, head_dim=80)) == EUNSUPPORTED and f(ot=2) == EUNSUPPORTED
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert f(scale=s) == EINVAL
    assert f(window=-1) == EINVAL and f(ldq=248) == EINVAL and f(ldo=255) == EINVAL
    assert f(ldq=260) == EALIGN and f(ldo=260) == EALIGN and f(q=odd) == EALIGN and f(out=odd) == EALIGN
    need = L.moex_paged_attention_workspace_bytes(ctypes.byref(_kv(mx, base)), ctypes.byref(_batch(mx, base)), 4)
    if need:
        assert f(n=need - 1) == ENOSPACE and f(ws=NULL) == ENOSPACE and f(ws=odd) == EALIGN


def test_attention_refuses_rows_past_32_bits():
    import moe_expert_gb300 as mx
    L = ensure_lib()
    buf, base, p, odd = _p()
    kv = _kv(mx, base, n_kv_heads=1)
    # 128 heads: 2^31 - 128 rows fit 32 bits, the end of the last tile does not
    for n in (1 << 24, (1 << 24) - 1, (1 << 24) - 4):
        b = _batch(mx, base, n_tokens=n, max_q=1)
        assert L.moex_paged_attention(p, 1 << 13, ctypes.byref(kv), ctypes.byref(b), 128, 0.125, 0, p, 1, 1 << 13, NULL,
                                      p, 1 << 40, NULL) == EUNSUPPORTED, n


def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    import moe_expert_gb300 as mx
    ensure_lib()
    x = torch.zeros(2, 64)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    cu, ctx, table = (torch.zeros(*s, dtype=torch.int32) for s in ((2,), (1,), (1, 4)))
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: mx.add_rms_norm(x, torch.zeros(64)), lambda: mx.route_experts(x, 2),
                 lambda: mx.dequantize_q8_1(torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2, 2, 2)),
                 lambda: mx.rope_kv_write(torch.zeros(3, 512), k, k, cu, ctx, table, n_heads=4),
                 lambda: mx.paged_attention(q, k, k, cu, ctx, table)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        mx.add_rms_norm(None, x)
    with pytest.raises(ValueError):
        mx.route_experts(x, 2, score="tanh")
