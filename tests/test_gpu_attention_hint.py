"""Without max_q the largest count that sequences of one token or more leave is
taken, so that a batch of single tokens gets the kernel for few rows."""
import pytest

from layer_cases import Paged, mx
from test_gpu_paged_attention import _check, _q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [[1] * 64, [3, 70, 1], [5], [0, 1, 0, 0]])
def test_default_hint(n):
    import torch
    m = mx()
    B, T = len(n), sum(n)
    p = Paged(61 + B, n, [x + 100 + 13 * b for b, x in enumerate(n)], 2, 128, 16, extra_width=400)
    q = _q(p, 4)
    most = T - B + 1 if T >= B else T
    need = lambda hint: m.paged_attention_workspace_bytes(p.k, p.v, *p.batch(), n_tokens=T, n_heads=4,  # noqa: E731
                                                          max_q=hint)
    assert need(None) == need(most)
    if n[0] == 1:
        assert need(None) < need(T)      # the larger workspace is that of the large tiles
    a = m.paged_attention(q, p.k, p.v, *p.batch())
    assert torch.equal(a, m.paged_attention(q, p.k, p.v, *p.batch(), max_q=most))
    _check(p, 4, q=q, max_q=most)
