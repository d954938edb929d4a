"""Pins of the oracle of the operators around a layer's products: closed
forms, exact rationals, invariants, and mistakes planted in the oracle."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import layer as ol
from oracle import moe as om


def test_norm_closed_forms():
    x = np.array([[3.0, -4.0, 0.0, 0.0]])
    s, y = ol.add_rms_norm(x, np.array([1.0, 2.0, 1.0, 1.0]), 0.0)
    assert np.array_equal(s, x)
    assert np.allclose(y, [[3 / 2.5, -8 / 2.5, 0, 0]], rtol=1e-15)         # mean square 25 / 4
    s, y = ol.add_rms_norm(np.zeros((1, 4)), np.ones(4), 1e-6)
    assert (y == 0).all()
    a = np.random.default_rng(0).standard_normal((3, 64))
    r = np.random.default_rng(1).standard_normal((3, 64))
    s, y = ol.add_rms_norm(a, np.ones(64), 1e-12, r)
    assert np.array_equal(s, a + r)
    assert np.allclose(np.mean(y ** 2, 1), 1.0, rtol=1e-9)                 # unit mean square
    assert np.allclose(ol.add_rms_norm(4 * a, np.ones(64), 1e-12, 4 * r)[1], y, rtol=1e-9)


def test_route_reduces_to_the_plain_router():
    x = np.random.default_rng(2).standard_normal((20, 24)).astype(np.float32)
    ids, w, _ = ol.route_experts(x, 5)
    rid, rw = om.route_topk(x, 5)
    assert np.array_equal(ids, rid) and np.allclose(w, rw, rtol=1e-12)
    _, p, _ = ol.route_experts(x, 24, renorm=False)
    assert np.allclose(p.sum(1), 1.0, rtol=1e-12)                          # a softmax over all experts


def test_route_by_hand():
    """Two groups of three; sigmoid scores 1/2, 2/3, 3/4 | 4/5, 1/3, 1/4."""
    p = [Fraction(1, 2), Fraction(2, 3), Fraction(3, 4), Fraction(4, 5), Fraction(1, 3), Fraction(1, 4)]
    x = np.array([[math.log(v / (1 - v)) for v in map(float, p)]])
    ids, w, margin = ol.route_experts(x, 2, score="sigmoid", groups=2, top_groups=1, group_top=2)
    # 3/4 + 2/3 = 17/12 against 4/5 + 1/3 = 17/15
    assert ids.tolist() == [[2, 1]]
    assert np.allclose(w, [[9 / 17, 8 / 17]], rtol=1e-12)
    assert abs(margin[0] - 1 / 12) < 1e-12                                 # 3/4 - 2/3 < 2/3 - 1/2 < 17/12 - 17/15
    ids, w, _ = ol.route_experts(x, 2, score="sigmoid", groups=2, top_groups=1, group_top=1)
    assert ids.tolist() == [[3, 4]]                                        # 4/5 is the best single expert
    ids, w, _ = ol.route_experts(x, 2, score="sigmoid", bias=np.array([0, 0, 0, 0, 0, 1.0]), renorm=False, scale=2.0)
    assert ids.tolist() == [[5, 3]] and np.allclose(w, [[0.5, 1.6]], rtol=1e-12)


def test_route_masks():
    inf = np.inf
    x = np.array([[-inf, 1.0, np.nan, 0.0], [-inf] * 4, [inf, 0.0, inf, 1.0]])
    ids, w, _ = ol.route_experts(x, 3, bias=np.array([9.0, 0, 9, 0]))
    assert ids.tolist() == [[1, 3, 0], [0, 1, 2], [0, 2, 1]]
    e = math.e
    assert np.allclose(w, [[e / (e + 1), 1 / (e + 1), 0], [0, 0, 0], [0.5, 0.5, 0]], rtol=1e-12)


def test_rope_is_a_turn_of_the_plane():
    g = np.random.default_rng(3)
    h, ang = g.standard_normal(12), g.standard_normal(4)
    for inter in (False, True):
        t = ol.rope(h, np.cos(ang), np.sin(ang), inter)
        a, b = (h[:8:2], h[1:8:2]) if inter else (h[:4], h[4:8])
        z = (a + 1j * b) * np.exp(1j * ang)
        ta, tb = (t[:8:2], t[1:8:2]) if inter else (t[:4], t[4:8])
        assert np.allclose(ta + 1j * tb, z, rtol=1e-12)
        assert np.array_equal(t[8:], h[8:])
        back = ol.rope(t, np.cos(ang), -np.sin(ang), inter)
        assert np.allclose(back, h, rtol=1e-12)


def test_scores_after_rope_depend_on_distance():
    """Turning q by position p and k by position j leaves q.k a function of p - j."""
    g = np.random.default_rng(4)
    q, k, f = g.standard_normal(8), g.standard_normal(8), g.random(4)
    at = lambda x, p: ol.rope(x, np.cos(p * f), np.sin(p * f))  # noqa: E731
    assert abs(at(q, 9) @ at(k, 4) - at(q, 105) @ at(k, 100)) < 1e-12


def _case():
    g = np.random.default_rng(5)
    k, v = g.standard_normal((6, 2, 4, 8)), g.standard_normal((6, 2, 4, 8))
    return g.standard_normal((5, 4, 8)), k, v, [0, 2, 5], [7, 3], [[5, 1], [0, 3]]


def test_write_places_tokens():
    _, k, v, cu, ctx, table = _case()
    rows = np.arange(5 * 8 * 8, dtype=np.float64).reshape(5, 64)
    q, k2, v2 = ol.rope_kv_write(rows, k, v, cu, ctx, table, 4)
    r = rows.reshape(5, 8, 8)
    assert np.array_equal(q, r[:, :4])
    # sequence 0: positions 5, 6 of pages (5, 1); sequence 1: positions 0, 1, 2 of page 0
    for t, (pg, s) in enumerate([(1, 1), (1, 2), (0, 0), (0, 1), (0, 2)]):
        assert np.array_equal(k2[pg, :, s], r[t, 4:6]) and np.array_equal(v2[pg, :, s], r[t, 6:8])
    same = np.ones((6, 4), bool)
    same[[1, 1, 0, 0, 0], [1, 2, 0, 1, 2]] = False
    assert np.array_equal(k2.transpose(0, 2, 1, 3)[same], k.transpose(0, 2, 1, 3)[same])


def test_attention_brute_force():
    q, k, v, cu, ctx, table = _case()
    out, lse = ol.paged_attention(q, k, v, cu, ctx, table, 0.3)
    where = [(0, 5), (0, 6), (1, 0), (1, 1), (1, 2)]
    for t, (b, p) in enumerate(where):
        for h in range(4):
            num, den = np.zeros(8), 0.0
            for j in range(p + 1):
                pg, s = table[b][j // 4], j % 4
                e = math.exp(0.3 * sum(q[t, h, d] * k[pg, h // 2, s, d] for d in range(8)))
                num += e * v[pg, h // 2, s]
                den += e
            assert np.allclose(out[t, h], num / den, rtol=1e-12)
            assert abs(lse[t, h] - math.log(den)) < 1e-12


def test_attention_special_cases():
    q, k, v, cu, ctx, table = _case()
    # one key only: its value; no key: zeros
    out, lse = ol.paged_attention(q, k, v, cu, ctx, table, 0.3, window=1)
    assert np.allclose(out[2, 3], v[0, 1, 0], rtol=1e-14) and np.allclose(out[1, 0], v[1, 0, 2], rtol=1e-14)
    out, lse = ol.paged_attention(q, k, v, cu, [1, 3], table, 0.3)
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all() and np.isfinite(lse[1]).all()
    # equal scores: the mean of the values seen
    out, _ = ol.paged_attention(0 * q, k, v, cu, ctx, table, 0.3)
    assert np.allclose(out[4, 0], v[0, 0, :3].mean(0), rtol=1e-12)
    # a window as long as the context changes nothing
    a = ol.paged_attention(q, k, v, cu, ctx, table, 0.3)[0]
    assert np.array_equal(a, ol.paged_attention(q, k, v, cu, ctx, table, 0.3, window=7)[0])


@pytest.mark.parametrize("plant", ["uncausal", "wrong_group", "wrong_page"])
def test_planted_mistakes_are_caught(plant, monkeypatch):
    q, k, v, cu, ctx, table = _case()
    good = ol.paged_attention(q, k, v, cu, ctx, table, 0.3)[0]
    if plant == "uncausal":
        monkeypatch.setattr(ol, "places", lambda cu_q, n: [(0, 6), (0, 6), (1, 2), (1, 2), (1, 2)])
        bad = ol.paged_attention(q, k, v, cu, ctx, table, 0.3)[0]
    elif plant == "wrong_group":
        bad = ol.paged_attention(q[:, [0, 2, 1, 3]], k, v, cu, ctx, table, 0.3)[0][:, [0, 2, 1, 3]]
    else:
        bad = ol.paged_attention(q, k, v, cu, ctx, [[1, 5], [0, 3]], 0.3)[0]
    assert np.abs(bad - good).max() > 1e-3
