"""Batches whose sequences fill an odd number of thread blocks, three and more:
3, 5 and 7 of 128 (the kernel for few rows), 3 of 384 (the one for many)."""
import numpy as np
import pytest

from layer_cases import Paged, mx, status
from test_gpu_paged_attention import _check, _q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,hint", [(257, 1), (300, 1), (384, 1), (600, 1), (896, 1), (769, 200), (900, 200),
                                    (1152, 200)])
def test_odd_numbers_of_blocks(B, hint):
    import torch
    g = np.random.Generator(np.random.PCG64(B + hint))
    n = g.integers(0, 3, B)
    n[[0, B // 3, B - 1]] = [40, 60, 25]
    total = n + np.exp(g.uniform(0, np.log(200), B)).astype(int)   # over two orders of magnitude
    p = Paged(B, n.tolist(), total.tolist(), 1, 64, 16)
    q = _q(p, 2)
    out = _check(p, 2, max_q=hint, q=q)
    for _ in range(20):
        again = mx().paged_attention(q, p.k, p.v, *p.batch(), max_q=hint)
        assert torch.equal(again, out)
    assert status() == 0
