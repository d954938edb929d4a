"""General expert routing on the GPU against the 64-bit formula.

Scores are FP32: an exponential (2 ulp, its argument rounded once: under
1e-6 for the logits here), a sum of at most 32 terms a lane and 5 levels, a
division: under 6e-6 of the score.  A selection is compared where every rank
that decides it is further from the next than 1e-5 of the token's largest score
(twice the error, for either of the two) and the rounding of the bias."""
import numpy as np
import pytest

from layer_cases import dtype, f64, mx, status
from oracle import layer as ol

pytestmark = pytest.mark.gpu


def _run(logits, k, **kw):
    import torch
    m = mx()
    bias = kw.pop("bias", None)
    b = None if bias is None else torch.from_numpy(bias).cuda()
    ids, w = m.route_experts(logits, k, bias=b, **kw)
    return ids.cpu().numpy(), w.cpu().numpy()


def _near(logits, kw):
    x = f64(logits)
    top = x.max(1)
    big = 1 / (1 + np.exp(-top)) if kw.get("score") == "sigmoid" else 1 / np.exp(x - top[:, None]).sum(1)
    return 1.2e-5 * big + (0.0 if kw.get("bias") is None else 2.0 ** -22 * np.abs(kw["bias"]).max())


def _compare(logits, k, rel=6e-6, share=0.5, **kw):
    ids, w = _run(logits, k, **kw)
    rid, rw, margin = ol.route_experts(f64(logits), k, **kw)
    sure = margin > _near(logits, kw)
    assert sure.mean() > share
    assert np.array_equal(ids[sure], rid[sure])
    scale = abs(kw.get("scale", 1.0))
    assert np.all(np.abs(w - rw)[sure] <= 2 * rel * np.abs(rw[sure]) + 1e-9 * scale)
    E = logits.shape[1]
    assert ids.min() >= 0 and ids.max() < E and all(len(set(r)) == k for r in ids.tolist())
    assert status() == 0


@pytest.mark.parametrize("T,E,k,groups,top_groups", [(1, 8, 1, 1, 1), (3, 128, 8, 1, 1), (129, 160, 6, 8, 3),
                                                     (65, 256, 8, 8, 4), (5, 1000, 16, 1, 1), (7, 33, 4, 3, 2),
                                                     (4, 1024, 16, 32, 5), (9, 40, 5, 8, 1), (300, 64, 6, 1, 1),
                                                     (6, 1, 1, 1, 1), (11, 384, 8, 4, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_matches_formula(T, E, k, groups, top_groups, score, biased):
    import torch
    g = torch.Generator().manual_seed(T + E + k)
    logits = torch.randn(T, E, generator=g).cuda() * 1.5
    bias = (0.05 * np.random.default_rng(E).standard_normal(E)).astype(np.float32) if biased else None
    for group_top in ((1, 2) if groups > 1 else (1,)):
        _compare(logits, k, score=score, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top)
    _compare(logits, k, score=score, bias=bias, groups=groups, top_groups=top_groups, renorm=False, scale=2.5)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_sixteen_bit_logits_and_strides(kind):
    import torch
    big = torch.randn(50, 300, device="cuda").to(dtype(kind))
    logits = big[:, 3:3 + 192]
    _compare(logits, 8, score="sigmoid", groups=4, top_groups=2, group_top=2)
    _compare(logits, 8, score="softmax")


def test_ties_go_to_the_lower_index():
    import torch
    logits = torch.zeros(3, 64, device="cuda")
    logits[0, [5, 9, 40]] = 1.0
    logits[2, 63] = -0.0
    ids, w = _run(logits, 4)
    assert ids.tolist() == [[5, 9, 40, 0], [0, 1, 2, 3], [0, 1, 2, 3]]
    ids, _ = _run(logits, 4, groups=8, top_groups=2, group_top=2, score="sigmoid")
    assert ids[0].tolist() == [5, 9, 0, 1]     # groups 0 and 1 tie at 1 + 1/2, group 5 comes after
    assert ids[1].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("E,k,groups", [(1024, 16, 1), (256, 8, 8), (512, 3, 4), (100, 16, 2)])
def test_few_distinct_logits(E, k, groups):
    """Hundreds of equal ranks around the k-th: the lowest indices of them."""
    import torch
    g = torch.Generator().manual_seed(E)
    logits = torch.randint(0, 3, (64, E), generator=g).float().cuda()
    for score in ("softmax", "sigmoid"):
        ids, w = _run(logits, k, score=score, groups=groups, top_groups=max(1, groups // 2))
        rid, rw, _ = ol.route_experts(f64(logits), k, score=score, groups=groups, top_groups=max(1, groups // 2))
        assert np.array_equal(ids, rid)
        assert np.allclose(w, rw, rtol=1.2e-5, atol=0)


def test_bias_moves_the_selection_only():
    import torch
    logits = torch.tensor([[2.0, 1.0, 0.0, -1.0]], device="cuda")
    bias = np.array([-10, 0, 0, 10], np.float32)
    ids, w = _run(logits, 2, score="sigmoid", bias=bias, renorm=False)
    assert ids.tolist() == [[3, 1]]
    assert np.allclose(w, 1 / (1 + np.exp([[1.0, -1.0]])), rtol=1e-6)


def test_masked_and_infinite_logits():
    import torch
    inf, nan = float("inf"), float("nan")
    rows = torch.tensor([[-inf] * 8,
                         [nan] * 8,
                         [-inf, 0.5, nan, -inf, 0.25, -inf, -inf, -inf],
                         [inf, 1.0, inf, 0.0, -inf, nan, 3.0, 2.0],
                         [-200.0] * 8,
                         [88.0, 89.0, 200.0, -88.0, -104.0, 0, 0, 0]], device="cuda")
    bias = np.array([9, -1, 9, 0, -2, 9, 0, 0], np.float32)
    for score in ("softmax", "sigmoid"):
        for kw in (dict(), dict(bias=bias), dict(groups=4, top_groups=2, group_top=2, bias=bias),
                   dict(groups=2, top_groups=1, group_top=1)):
            for renorm in (True, False):
                ids, w = _run(rows, 3, score=score, renorm=renorm, **kw)
                rid, rw, margin = ol.route_experts(f64(rows), 3, score=score, renorm=renorm, **kw)
                sure = margin > 1e-5
                assert np.array_equal(ids[sure], rid[sure]), (score, kw)
                # scores far below one lose their last bits to the smallest FP32 numbers
                fine = sure & (np.arange(6) != 4)
                assert np.allclose(w[fine], rw[fine], rtol=2e-5, atol=1e-9)
                assert np.isfinite(w).all()
                assert (w[:2] == 0).all()


def test_equals_plain_router_where_both_apply():
    import torch
    m = mx()
    logits = torch.randn(777, 128, device="cuda")
    a, wa = m.route_topk(logits, 8)
    b, wb = m.route_experts(logits, 8)
    assert torch.equal(a, b)
    assert torch.allclose(wa, wb, rtol=2e-5, atol=0)
