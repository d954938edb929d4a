"""The norm of rows whose squares leave FP32's range, up to the largest values, and
q8_1 blocks of the smallest.
The bounds are those of the ordinary rows (test_gpu_norm.py): the scaling by a
power of two is exact.  Beside a value of 2^128 others give results below 2^-126,
where even the nearest FP32 number is off by up to 2^-150 (BF16: 2^-134): there
that much comes in twice in FP32, once times gamma, and once more in BF16."""
import numpy as np
import pytest

from layer_cases import HALF_ULP, U32, f64, mx, status
from oracle import layer as ol
from oracle import q8_1 as oq
from test_gpu_norm import EPS

pytestmark = pytest.mark.gpu
BIG = 3.4028234663852886e38   # FP32's largest value


def _check_y(got, ref, gamma, kind):
    h = HALF_ULP[kind] if kind != "f32" else 0
    tol = (20 * U32 + h) * 1.01 * np.abs(ref) + 2.0 ** -150 * (1 + f64(gamma).max())
    tol = tol + (2.0 ** -134 if kind == "bf16" else 0)
    assert np.all(np.abs(f64(got) - ref) <= tol)


def _check(x, gamma, residual=None, eps=EPS):
    import torch
    m = mx()
    s, y, q, ds = m.add_rms_norm(x, gamma, eps, residual=residual, y_dtype=torch.float32, quantize=True)
    ref = ol.add_rms_norm(f64(x), f64(gamma), eps, None if residual is None else f64(residual))[1]
    _check_y(y, ref, gamma, "f32")
    rq, rd, rsum = oq.quantize_q8_1(y.cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(ds.cpu().numpy(), np.stack([rd, rsum], axis=2))
    _check_y(m.add_rms_norm(x, gamma, eps, residual=residual, y_dtype=torch.bfloat16)[1], ref, gamma, "bf16")
    assert status() == 0


@pytest.mark.parametrize("H", [32, 96, 2560, 32768])
@pytest.mark.parametrize("value", [3e18, 1e19, 7e36, 1e37, 3e38, BIG])
def test_rows_of_one_large_value(H, value):
    import torch
    x = torch.full((3, H), value, device="cuda")
    x[1] *= -1
    x[2, ::2] *= -1
    g = torch.Generator().manual_seed(H)
    _check(x, (1 + 0.3 * torch.randn(H, generator=g)).cuda())
    _check(x, torch.ones(H, device="cuda"), residual=torch.zeros(3, H, device="cuda"))


@pytest.mark.parametrize("H", [64, 2560, 32768])
def test_large_values_among_others(H):
    """One or a few large values beside ordinary ones, and values spread over many powers of two."""
    import torch
    g = torch.Generator().manual_seed(H + 1)
    x = torch.randn(4, H, generator=g)
    x[0, H // 3] = BIG
    x[1, ::32] = -1e38
    x[2] *= torch.exp2(torch.rand(H, generator=g) * 40 + 80)
    x[3] *= 3e37
    gamma = (1 + 0.3 * torch.randn(H, generator=g)).cuda()
    _check(x.cuda(), gamma)
    r = torch.randn(4, H, generator=g) * 1e37
    _check(x.clamp(-3e38, 3e38).cuda(), gamma, residual=r.cuda())


def test_eps_beside_large_values():
    """eps counts wherever it is not small beside the mean square."""
    import torch
    x = torch.zeros(1, 32768, device="cuda")
    x[0, :2] = 1.5e19
    _check(x, torch.ones(32768, device="cuda"), eps=1e34)


def test_smallest_values_do_not_wrap():
    """Below FP32's smallest normal number amax / 127 rounds to few units, and a
    value may be more than 127 of them: it is then held as +-127."""
    import torch
    m = mx()
    unit = 2.0 ** -149
    sign = torch.ones(1, 32, device="cuda")
    sign[0, 1::2] = -1
    for units in (64, 100, 127, 150, 190, 250, 1000, 100000):
        gamma = torch.full((32,), units * unit, device="cuda")
        _, y, q, ds = m.add_rms_norm(sign, gamma, 1e-30, y_dtype=torch.float32, quantize=True)
        assert (y.sign() == sign).all()
        d = ds[0, 0, 0].item()
        want = 0 if d == 0 else min(127, int(y.abs().max().item() / d + 0.5))
        assert (q.abs() == want).all() and (q * sign >= 0).all(), units
