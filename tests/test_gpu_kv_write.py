"""Rotary embedding and the cache write on the GPU against the 64-bit formula.

A turned feature is two FP32 products and an addition of FP32 inputs (3
roundings of terms below |a| + |b|), then one rounding to the cache type;
values are one rounding of the input, bit for bit."""
import numpy as np
import pytest

from layer_cases import HALF_ULP, TINY, U32, Paged, dtype, f64, mx, status
from oracle import layer as ol

pytestmark = pytest.mark.gpu


def _table(n_pos, rot):
    import torch
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * inv[None]
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def _qkv(T, width, kind):
    import torch
    g = torch.Generator().manual_seed(T * 7 + width)
    return (torch.randn(T, width, generator=g) * 2).to(dtype(kind)).cuda()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,total,Hq,Hkv,D,page,rot,inter,cache,layout", [
    ([1], [1], 4, 1, 64, 16, 64, False, "bf16", "hpd"),
    ([1, 0, 3, 17], [900, 5, 3, 40], 8, 2, 128, 16, 128, False, "bf16", "phd"),
    ([33, 2], [33, 130], 5, 5, 128, 64, 64, True, "f16", "pool"),
    ([5], [77], 3, 1, 96, 8, 32, False, "f16", "hpd"),
    ([9, 9], [9, 30], 2, 2, 80, 32, 0, False, "bf16", "hpd"),
    ([2, 1], [300, 1], 2, 1, 512, 128, 512, True, "bf16", "hpd"),
])
def test_matches_formula(kind, n, total, Hq, Hkv, D, page, rot, inter, cache, layout):
    import torch
    m = mx()
    p = Paged(len(n) + D, n, total, Hkv, D, page, cache, layout, junk=0.5)
    qkv = _qkv(p.T, (Hq + 2 * Hkv) * D, kind)
    cs = _table(max(total), rot) if rot else None
    k0, v0 = f64(p.k), f64(p.v)
    q = m.rope_kv_write(qkv, p.k, p.v, *p.batch(), n_heads=Hq, cos_sin=cs, interleaved=inter)
    rq, rk, rv = ol.rope_kv_write(f64(qkv), k0, v0, p.cu_np, p.ctx_np, p.table_np, Hq,
                                  None if cs is None else cs.cpu().numpy(), inter)
    big = 2 * np.abs(f64(qkv)).max()
    for got, ref in ((q, rq), (p.k, rk)):
        tol = HALF_ULP[cache] * 1.01 * np.abs(ref) + 3 * U32 * big + TINY[cache]
        assert np.all(np.abs(f64(got) - ref) <= tol)
    want = torch.from_numpy(rv).to(dtype(cache)) if kind != "f32" else torch.from_numpy(rv.astype(np.float32)).to(dtype(cache))
    assert torch.equal(p.v.cpu(), want)
    # slots of no new token keep their bits
    touched = np.zeros((p.n_pages, page), bool)
    for b, pos in ol.places(p.cu_np, p.ctx_np):
        touched[p.table_np[b, pos // page], pos % page] = True
    keep = ~np.broadcast_to(touched[:, None, :], (p.n_pages, Hkv, page))
    assert np.array_equal(f64(p.k)[keep], k0[keep])
    assert status() == 0


def test_strided_rows_and_given_output():
    import torch
    m = mx()
    p = Paged(3, [4, 2], [50, 2], 2, 64, 16, junk=0.0)
    wide = _qkv(6, 1024, "f32")
    qkv = wide[:, 64:64 + 8 * 64]
    out = torch.full((6, 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    q = m.rope_kv_write(qkv, p.k, p.v, *p.batch(), n_heads=4, cos_sin=_table(50, 64), q=out[:, 1:5])
    k1 = p.k.clone()
    want = m.rope_kv_write(qkv.contiguous(), p.k, p.v, *p.batch(), n_heads=4, cos_sin=_table(50, 64))
    assert torch.equal(q, want) and torch.equal(k1, p.k) and (out[:, 0] == 7).all() and (out[:, 5] == 7).all()


def test_positions_outside_are_left_out():
    """A length shorter than the new tokens gives negative positions (zeros,
    nothing written); positions past the angle table, page ids past the cache
    and lengths past the page table are flagged and left out."""
    import torch
    m = mx()

    def case(change):
        p = Paged(5, [3, 4], [20, 30], 1, 64, 16, junk=0.0)
        change(p)
        qkv = _qkv(7, 3 * 64, "f32")
        k0 = p.k.clone()
        cs = p.cs if hasattr(p, "cs") else _table(64, 64)
        q = m.rope_kv_write(qkv, p.k, p.v, *p.batch(), n_heads=1, cos_sin=cs)
        return p, q, (p.k != k0).flatten(1).any(1).sum().item(), status()

    def short(p):
        p.ctx[0] = 2
    p, q, _, st = case(short)
    assert st == 0 and (q[0] == 0).all() and (q[1] != 0).any()

    def past(p):
        p.cs = _table(28, 64)
    p, q, _, st = case(past)
    assert st == 16 and (q[5:] == 0).all() and (q[:5] != 0).flatten(1).any(1).all()

    def page(p):
        p.table[1, 1] = p.n_pages
    p, q, pages, st = case(page)
    assert st == 16 and pages == 1 and (q != 0).flatten(1).any(1).all()

    def long(p):
        p.ctx[1] = 1 << 28
    p, q, pages, st = case(long)
    assert st == 16 and (q[3:] == 0).all()
    m.device_status()
