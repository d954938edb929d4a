"""Small probabilities with FP16 caches.  Most of FP16's range lies above 1, so
probabilities are held relative to a power of two below the row's maximum (by 2^7
at least): one that is 2^-26 of the largest still counts in the output, as in the
sum.

Tolerance: with the largest probability at 2^7 a rounding is off by half an ulp
(2^-11 of the value) or half a subnormal spacing (2^-25, so 2^-32 of the largest);
the latter once a key, over the sum of the probabilities relative to the largest.
FP32 sums of these equal terms and exponentials are far below (2^-16)."""
import numpy as np
import pytest

from layer_cases import Paged, f64, mx, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,total", [([1], [500]), ([1], [9000]), ([70], [700]), ([120], [9000])])
@pytest.mark.parametrize("gap", [12.0, 15.0, 18.0])
def test_many_small_probabilities_beside_large_ones(D, n, total, gap):
    """Every eighth key has the largest score and a value of 0; the others are
    e^-gap of it and share one value."""
    import torch
    m = mx()
    p = Paged(41, n, total, 1, D, 16, "f16", junk=0.0)
    p.k.zero_()
    p.k[:, :, ::8, 0] = 1.0
    p.v.fill_(30000.0)
    p.v[:, :, ::8] = 0.0
    q = torch.zeros(p.T, 2, D, dtype=torch.float16, device="cuda")
    q[:, :, 0] = gap
    lse = torch.empty(p.T, 2, device="cuda")
    out = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q, scale=1.0, out_dtype=torch.float32, lse=lse)
    for i in range(p.T):
        keys = total[0] - n[0] + i + 1
        large = -(-keys // 8)
        small = keys - large
        den = large + small * np.exp(-gap)
        ref = small * np.exp(-gap) * 30000.0 / den
        tol = (2.0 ** -11 + 2.0 ** -16) * ref + 2.0 ** -32 * small * 30000.0 / den
        assert np.all(np.abs(f64(out[i]) - ref) <= tol), (i, ref, f64(out[i]).min(), tol)
        assert np.all(np.abs(f64(lse[i]) - (gap + np.log(den))) <= 1e-5)
    assert status() == 0


@pytest.mark.parametrize("n,total", [([1, 3], [5000, 40]), ([100, 40], [5000, 40])])
def test_largest_values_and_long_sums_stay_finite(n, total):
    """The largest FP16 values under equal probabilities: sums far above FP16's range on the way."""
    import torch
    m = mx()
    p = Paged(42, n, total, 2, 64, 16, "f16")
    p.v.masked_fill_(p.v == p.v, 65504.0)
    q = torch.zeros(p.T, 4, 64, dtype=torch.float16, device="cuda")
    out = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q)
    assert (out == 65504.0).all()
    out = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q, out_dtype=torch.float32)
    assert ((out - 65504.0).abs() <= 65504.0 * 2.0 ** -16).all() and status() == 0
