"""Keys in front of a sliding window have no influence, whatever lies there: a
server frees and reuses those pages, so here they hold NaN, and where a page has
no key that any new token of the sequence sees, its entry in the table is -1."""
import pytest

from layer_cases import Paged
from test_gpu_paged_attention import _check

pytestmark = pytest.mark.gpu


def _evict(p, window):
    """NaN below the first key that a new token of each sequence sees, -1 for
    the pages that lie wholly below it; the last such position of each sequence."""
    import torch
    table = p.table_np.copy()
    gone = torch.zeros(p.n_pages, p.page, dtype=torch.bool)
    for b, (n, total) in enumerate(zip(p.n, p.total)):
        # without new tokens nothing is seen
        first = max(0, total - n - window + 1) if n else total
        for j in range(first):
            gone[p.table_np[b, j // p.page], j % p.page] = True
        table[b, : first // p.page] = -1
    gone = gone.cuda()[:, None, :, None]
    p.k.masked_fill_(gone, float("nan"))
    p.v.masked_fill_(gone, float("nan"))
    p.table = torch.from_numpy(table).cuda()
    assert (table == -1).any() or p.page > min(p.total)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 6, 2)])
@pytest.mark.parametrize("page", [8, 16, 64])
@pytest.mark.parametrize("window", [1, 15, 37, 200])
def test_few_rows(kind, D, Hq, Hkv, page, window):
    n, total = [1, 2, 3, 1, 0, 2], [20, 300, 777, 1025, 90, 4000]
    p = Paged(D + page + window, n, total, Hkv, D, page, kind)
    _evict(p, window)
    _check(p, Hq, window=window)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 1), (64, 8, 2)])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 256])
@pytest.mark.parametrize("window", [1, 50, 129, 500])
def test_many_rows(kind, D, Hq, Hkv, page, window):
    n, total = [90, 1, 33, 300], [700, 1000, 95, 1500]
    p = Paged(D + page + window, n, total, Hkv, D, page, kind)
    _evict(p, window)
    _check(p, Hq, window=window)


@pytest.mark.parametrize("n,Hq", [([1], 8), ([40], 8)])
def test_long_context(n, Hq):
    """Tiles that many CTAs share begin inside a block as well."""
    p = Paged(31, n, [20000], 1, 128, 64)
    _evict(p, 12345)
    _check(p, Hq, window=12345)


@pytest.mark.parametrize("layout", ["phd", "pool"])
@pytest.mark.parametrize("n", [[1, 1], [40, 70]])
def test_layouts(layout, n):
    p = Paged(32, n, [300, 500], 2, 128, 32, "bf16", layout)
    _evict(p, 77)
    _check(p, 6, window=77)
