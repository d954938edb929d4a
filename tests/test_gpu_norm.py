"""Residual addition + RMS norm on the GPU against the 64-bit formula.

Bounds: s is one FP32 addition; the sum of squares is a sum of at most 8 chunks
of 4 and a tree of 10 levels (under 24 roundings), halved by the square root,
then the division, the root and two products: under 20 units of 2^-24 in all,
plus the output's own rounding.  q8_1 of the FP32 y is bit-exact (the oracle
quantises the GPU's own y)."""
import numpy as np
import pytest

from layer_cases import HALF_ULP, TINY, U32, dtype, f64, mx, status
from oracle import layer as ol
from oracle import q8_1 as oq

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _inputs(T, H, kind, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed + 31 * T + H)
    x = (torch.randn(T, H, generator=g) * 2).to(dtype(kind)).cuda()
    r = (torch.randn(T, H, generator=g) * 5).cuda()
    gamma = (1 + 0.3 * torch.randn(H, generator=g)).cuda()
    return x, r, gamma


def _check_y(got, ref, kind):
    h = HALF_ULP[kind]
    tol = (20 * U32 + (h if kind != "f32" else 0)) * 1.01 * np.abs(ref) + TINY[kind]
    bad = np.abs(f64(got) - ref) > tol
    assert not bad.any(), (int(bad.sum()), float((np.abs(f64(got) - ref) / np.maximum(tol, 1e-30)).max()))


@pytest.mark.parametrize("T,H", [(1, 32), (1, 2560), (3, 64), (7, 4096), (5, 4128), (64, 2560), (2, 8192), (2, 8224),
                                 (2, 20000), (1, 32768), (1111, 544)])
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
def test_norm_matches_formula(T, H, xt):
    import torch
    m = mx()
    x, r, gamma = _inputs(T, H, xt)
    for res in (r, None):
        s, y, q, ds = m.add_rms_norm(x, gamma, EPS, residual=res, y_dtype=torch.float32, quantize=True,
                                     sum_out=None if res is not None else torch.empty(T, H, device="cuda"))
        rs, ry = ol.add_rms_norm(f64(x), f64(gamma), EPS, None if res is None else f64(res))
        assert np.all(np.abs(f64(s) - rs) <= U32 * np.abs(rs))
        _check_y(y, ry, "f32")
        rq, rd, rsum = oq.quantize_q8_1(y.cpu().numpy())
        assert np.array_equal(q.cpu().numpy(), rq)
        assert np.array_equal(ds.cpu().numpy(), np.stack([rd, rsum], axis=2))
        for yt in ("bf16", "f16"):
            s2, y2, q2, ds2 = m.add_rms_norm(x, gamma, EPS, residual=res, y_dtype=dtype(yt), quantize=True)
            _check_y(y2, ry, yt)
            assert torch.equal(q2, q) and torch.equal(ds2, ds)
    assert status() == 0


def test_outputs_one_at_a_time_and_in_place():
    import torch
    m = mx()
    x, r, gamma = _inputs(9, 2560, "f32")
    s, y, q, ds = m.add_rms_norm(x, gamma, EPS, residual=r, y_dtype=torch.bfloat16, quantize=True)
    r2 = r.clone()
    s2, y2, q2, ds2 = m.add_rms_norm(x, gamma, EPS, residual=r2, sum_out=r2)
    assert s2 is r2 and torch.equal(r2, s) and y2 is None and q2 is None and ds2 is None
    x2 = x.clone()
    m.add_rms_norm(x2, gamma, EPS, residual=r, sum_out=x2, y=y)
    assert torch.equal(x2, s)
    assert m.add_rms_norm(x, gamma, EPS, y_dtype=torch.bfloat16)[0] is None


def test_strided_rows():
    import torch
    m = mx()
    big = torch.randn(6, 3 * 640 + 16, device="cuda")
    x, res = big[:, 16:16 + 640], torch.randn(6, 1000, device="cuda")[:, 200:840]
    gamma = torch.rand(640, device="cuda")
    wide = torch.full((6, 700), 9.0, dtype=torch.bfloat16, device="cuda")
    s, y, _, _ = m.add_rms_norm(x, gamma, EPS, residual=res, y=wide[:, 8:648])
    a, b, _, _ = m.add_rms_norm(x.contiguous(), gamma, EPS, residual=res.contiguous(), y_dtype=torch.bfloat16)
    assert torch.equal(s, a) and torch.equal(wide[:, 8:648], b)
    assert (wide[:, :8] == 9).all() and (wide[:, 648:] == 9).all()


def test_zero_rows_and_large_values():
    import torch
    m = mx()
    x = torch.zeros(3, 96, device="cuda")
    x[1] = 3e18
    x[2, 5] = -1e-30
    gamma = torch.ones(96, device="cuda")
    _, y, q, ds = m.add_rms_norm(x, gamma, EPS, y_dtype=torch.float32, quantize=True)
    assert (y[0] == 0).all() and (q[0] == 0).all() and (ds[0] == 0).all()
    assert torch.allclose(y[1], torch.ones(96, device="cuda"), rtol=20 * U32, atol=0)
    assert q[2, 5] == -127 and (q[2, :5] == 0).all()


def test_dequantize_is_the_product():
    import torch
    m = mx()
    q = torch.randint(-127, 128, (5, 160), dtype=torch.int8, device="cuda")
    ds = torch.rand(5, 5, 2, device="cuda")
    ref = (q.view(5, 5, 32).float() * ds[:, :, :1]).view(5, 160)
    for kind in ("f32", "bf16", "f16"):
        assert torch.equal(m.dequantize_q8_1(q, ds, dtype=dtype(kind)), ref.to(dtype(kind)))


def test_other_stream():
    import torch
    m = mx()
    x, r, gamma = _inputs(33, 2560, "f32")
    want = m.add_rms_norm(x, gamma, EPS, residual=r, y_dtype=torch.bfloat16)[1]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(want)
    s = torch.empty_like(x)
    m.add_rms_norm(x, gamma, EPS, residual=r, sum_out=s, y=y, stream=st)
    st.synchronize()
    assert torch.equal(y, want)
