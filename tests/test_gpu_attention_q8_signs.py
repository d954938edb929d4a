"""Scales of a Q8_0 cache with the sign bit set: a block's value is scale * int8,
so (-d) * (-q) is d * q and the formula's result stays what it was.  The library's
writer stores none, a cache from elsewhere may."""
import numpy as np
import pytest

from layer_cases import dtype, f64, mx
from q8_cases import PagedQ8, attention_q8_bound, status

pytestmark = pytest.mark.gpu

SHAPES = [  # new tokens, lengths, query heads, key heads, head size, page: clusters, ranges, tiles of 8 and 16 rows
    ([1], [200], 4, 1, 128, 16),
    ([1, 1, 1], [1000, 33, 8], 8, 2, 64, 16),
    ([1] * 9, [3000, 20, 1, 700, 700, 64, 5000, 90, 1200], 8, 8, 128, 16),
    ([3, 5, 1], [400, 4500, 70], 10, 2, 64, 32),
    ([12, 2], [900, 130], 6, 2, 128, 64),
]


def _flip(codes, scales, where):
    """(-q, -d) in the blocks of `where`."""
    import torch
    return torch.where(where.repeat_interleave(32, -1), -codes, codes), torch.where(where, -scales, scales)


def _compare(p, q, kind, cache, window=0):
    import torch
    m = mx()
    ref, rl, tol, tol32, ltol = attention_q8_bound(p, f64(q), kind, p.D ** -0.5, window)
    lse = torch.empty(p.T, q.shape[1], device="cuda")
    out = m.paged_attention_q8(q, *cache, *p.batch(), max_q=p.max_q, window=window, lse=lse)
    o32 = m.paged_attention_q8(q, *cache, *p.batch(), max_q=p.max_q, window=window, out_dtype=torch.float32)
    for got, t in ((out, tol), (o32, tol32)):
        err = np.abs(f64(got) - ref)
        assert (err <= t).all(), (float((err / t).max()), float(np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)))
    assert np.all(np.abs(f64(lse) - rl) <= ltol) and status() == 0


@pytest.mark.parametrize("which", ["all", "one key", "half", "keys", "both"])
@pytest.mark.parametrize("n,total,Hq,Hkv,D,page", SHAPES)
def test_negative_scales(n, total, Hq, Hkv, D, page, which):
    import torch
    p = PagedQ8(50 + D + len(n), n, total, Hkv, D, page)
    g = torch.Generator(device="cuda").manual_seed(1)
    one = torch.zeros(p.ks.shape, dtype=torch.bool, device="cuda")
    for b, t in enumerate(total):
        one[p.table_np[b, t // 3 // page], :, t // 3 % page] = True
    half = torch.rand(p.ks.shape, device="cuda", generator=g) < 0.5
    every = torch.ones_like(one)
    of_v = {"all": every, "one key": one, "half": half, "both": half}.get(which)
    of_k = {"keys": half, "both": every}.get(which)
    k, ks = (p.k, p.ks) if of_k is None else _flip(p.k, p.ks, of_k)
    v, vs = (p.v, p.vs) if of_v is None else _flip(p.v, p.vs, of_v)
    kind = "bf16" if D == 64 else "f16"
    q = torch.from_numpy(p.g.standard_normal((p.T, Hq, D)).astype(np.float32) * 1.5).to(dtype(kind)).cuda()
    _compare(p, q, kind, (k, v, ks, vs))
    _compare(p, q, kind, (k, v, ks, vs), window=77)


@pytest.mark.parametrize("n,total,Hq,Hkv,D,page", SHAPES)
def test_scales_of_minus_zero(n, total, Hq, Hkv, D, page):
    """Blocks of zeros, whose scale a quantiser may leave as -0: some blocks of some keys, and the last key whole."""
    import torch
    p = PagedQ8(60 + D + len(n), n, total, Hkv, D, page)
    zero = p.g.random(p.vd.shape) < 0.1
    for b, t in enumerate(total):
        zero[p.table_np[b, (t - 1) // page], :, (t - 1) % page] = True
    live = zero & np.isfinite(p.vd)
    p.vd[live], p.kd[live] = 0, 0
    at = torch.from_numpy(live).cuda()
    ks, vs = (torch.where(at, torch.full_like(s, -0.0), s) for s in (p.ks, p.vs))
    assert (vs[at].view(torch.int16) == -32768).all()
    kind = "bf16" if D == 64 else "f16"
    q = torch.from_numpy(p.g.standard_normal((p.T, Hq, D)).astype(np.float32) * 1.5).to(dtype(kind)).cuda()
    _compare(p, q, kind, (p.k, p.v, ks, vs))


def test_read_back_of_negative_scales():
    import torch
    m = mx()
    p = PagedQ8(70, [1, 1], [100, 37], 2, 64, 16)
    k, ks = _flip(p.k, p.ks, torch.ones_like(p.ks, dtype=torch.bool))
    v, vs = _flip(p.v, p.vs, torch.ones_like(p.vs, dtype=torch.bool))
    to = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    outs = [tuple(torch.zeros(8, 2, 32, 64, dtype=torch.float16, device="cuda") for _ in range(2)) for _ in range(2)]
    m.kv_read_q8(*p.cache, p.ctx, p.table, *outs[0], to)
    m.kv_read_q8(k, v, ks, vs, p.ctx, p.table, *outs[1], to)
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and status() == 0
