"""Tokens that no sequence of the batch covers are flagged by attention, as by
the cache write; what the sequences cover is computed all the same."""
import pytest

from layer_cases import Paged, mx, status
from test_gpu_paged_attention import _q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,n", [(3, 2), (3, 60), (40, 1), (500, 1)])
def test_uncovered_tokens_are_flagged(B, n):
    import torch
    m = mx()
    p = Paged(51 + B, [n] * B, [n + 7 * (b % 9) for b in range(B)], 2, 64, 16)
    q = _q(p, 4)
    call = lambda q, cu: m.paged_attention(q, p.k, p.v, cu, p.ctx, p.table, max_q=p.max_q)  # noqa: E731
    good = call(q, p.cu)
    assert status() == 0
    # two rows more than the sequences have: behind them, then in front of them
    longer = torch.cat([q, q[:2]])
    out = call(longer, p.cu)
    assert status() == 16 and torch.equal(out[: p.T], good)
    out = call(torch.cat([q[:2], q]), p.cu + 2)
    assert status() == 16 and torch.equal(out[2:], good)
    assert torch.equal(call(q, p.cu), good) and status() == 0
