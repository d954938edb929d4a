"""Paged attention on the GPU against the 64-bit formula (the bound is derived
in layer_cases.attention_bound), over head layouts, ragged batches, page sizes,
windows, strides, empty rows and bad batches."""
import numpy as np
import pytest

from layer_cases import Paged, attention_bound, dtype, f64, mx, status

pytestmark = pytest.mark.gpu


def _q(p, Hq, gain=1.5):
    import torch
    x = p.g.standard_normal((p.T, Hq, p.D)).astype(np.float32) * gain
    return torch.from_numpy(x).to(dtype(p.kind)).cuda()


def _check(p, Hq, window=0, scale=None, max_q=None, gain=1.5, q=None):
    import torch
    m = mx()
    q = _q(p, Hq, gain) if q is None else q
    lse = torch.full((p.T, Hq), 123.0, device="cuda")
    out = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=max_q or p.max_q, window=window, scale=scale, lse=lse)
    o32 = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=max_q or p.max_q, window=window, scale=scale,
                            out_dtype=torch.float32)
    sc = p.D ** -0.5 if scale is None else scale
    ref, rl, tol, ltol = attention_bound(p, f64(q), sc, window, Hq // p.Hkv)
    for got in (out, o32):
        err = np.abs(f64(got) - ref)
        bad = err > tol
        assert not bad.any(), (int(bad.sum()), bad.size, float((err / tol).max()), np.argwhere(bad)[:4].tolist())
    assert torch.equal(o32.to(out.dtype), out)
    got = f64(lse)
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(got), empty)
    assert np.all(np.abs(got[~empty] - rl[~empty]) <= ltol[~empty])
    assert status() == 0
    return out


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (20, 4), (12, 12), (16, 1)])
@pytest.mark.parametrize("page", [8, 16, 64])
def test_single_tokens(kind, D, Hq, Hkv, page):
    total = [1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1025]
    p = Paged(Hq + D + page, [1] * len(total), total, Hkv, D, page, kind)
    _check(p, Hq)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hq,Hkv,page", [(64, 40, 8, 32), (128, 8, 2, 16), (128, 5, 5, 128), (64, 7, 1, 8)])
def test_drafts(kind, D, Hq, Hkv, page):
    n = [1, 2, 3, 4, 5, 6, 7, 8, 0, 5]
    total = [1, 2, 60, 4, 300, 77, 1000, 8, 40, 129]
    _check(Paged(D + Hq, n, total, Hkv, D, page, kind), Hq)
    _check(Paged(D + Hq + 1, n, total, Hkv, D, page, kind), Hq, window=37)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hq,Hkv,page", [(128, 4, 1, 16), (64, 6, 2, 64), (128, 3, 3, 32), (64, 10, 2, 8),
                                           (128, 16, 1, 256)])
def test_prompts(kind, D, Hq, Hkv, page):
    n = [1, 31, 33, 64, 100, 257]
    _check(Paged(D + page, n, n, Hkv, D, page, kind), Hq)
    _check(Paged(D + page + 1, n, n, Hkv, D, page, kind), Hq, window=50)


@pytest.mark.parametrize("D,Hq,Hkv,page", [(128, 8, 2, 16), (64, 8, 2, 64), (128, 1, 1, 32)])
@pytest.mark.parametrize("n,total", [([130], [700]), ([17, 300], [1600, 333]), ([1, 40, 1, 129], [800, 1000, 3, 129])])
def test_chunks(D, Hq, Hkv, page, n, total):
    _check(Paged(D + sum(n), n, total, Hkv, D, page), Hq)
    _check(Paged(D + sum(n) + 1, n, total, Hkv, D, page), Hq, window=200)


@pytest.mark.parametrize("layout", ["phd", "pool"])
@pytest.mark.parametrize("n", [[1, 1, 1], [40, 3, 90]])
def test_cache_layouts(layout, n):
    p = Paged(11, n, [200, 50, 90], 2, 128, 16, "bf16", layout)
    _check(p, 6)


def test_strided_queries_and_output():
    import torch
    m = mx()
    for n in ([1, 1], [70, 9]):
        p = Paged(12, n, [100, 33], 2, 64, 16)
        wide = torch.randn(p.T, 10, 64, device="cuda").bfloat16()
        q = wide[:, 2:8]
        want = _check(p, 6, q=q)
        out = torch.full((p.T, 8, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q, out=out[:, 1:7])
        assert torch.equal(out[:, 1:7], want) and (out[:, 0] == 5).all() and (out[:, 7] == 5).all()


@pytest.mark.parametrize("n,total", [([1, 1, 1], [0, 5, 0]), ([4, 3, 2], [2, 0, 9]), ([50, 200], [20, 0]),
                                     ([90, 0, 40], [300, 12, 0])])
def test_rows_without_keys_give_zeros(n, total):
    p = Paged(13, n, total, 2, 128, 16)
    out = _check(p, 8)
    assert (out[: max(0, n[0] - total[0])] == 0).all()


@pytest.mark.parametrize("n,total", [([1], [500]), ([120], [500])])
def test_window_of_one_returns_the_value(n, total):
    """A window of one key leaves the token's own value, bit for bit."""
    import torch
    p = Paged(14, n, total, 2, 64, 16)
    m = mx()
    out = m.paged_attention(_q(p, 4), p.k, p.v, *p.batch(), max_q=p.max_q, window=1)
    for i in range(n[0]):
        pos = total[0] - n[0] + i
        v = p.v[p.table_np[0, pos // 16], :, pos % 16]
        assert torch.equal(out[i], v.repeat_interleave(2, 0))


@pytest.mark.parametrize("n,total", [([1, 1], [700, 900]), ([150], [600])])
def test_peaked_scores(n, total):
    """Scores of hundreds: one key takes nearly all the weight, and the running
    maximum moves many times."""
    p = Paged(15, n, total, 2, 128, 16)
    _check(p, 4, gain=60.0)
    p = Paged(16, n, total, 2, 64, 16, "f16")
    _check(p, 4, gain=60.0)


def test_growing_scores():
    """Keys whose scores rise along the sequence, so that every tile brings a new maximum."""
    import torch
    for n in ([1], [140]):
        p = Paged(17, n, [900], 1, 64, 16, junk=0.0)
        ramp = torch.zeros(p.n_pages, p.page, device="cuda")
        for j in range(900):
            ramp[p.table_np[0, j // 16], j % 16] = j / 20.0
        p.k[:, 0, :, 0] = ramp.bfloat16()
        q = torch.zeros(p.T, 2, 64, device="cuda").bfloat16()
        q[:, :, 0] = 8.0
        q[:, 1, 0] = -8.0
        _check(p, 2, q=q)


@pytest.mark.parametrize("B", [33, 150, 700])
@pytest.mark.parametrize("hint", [None, 200])
def test_many_sequences(B, hint):
    """More sequences than a warp, a CTA of either kernel, has lanes."""
    g = np.random.Generator(np.random.PCG64(B))
    n = g.integers(0, 4, B)
    n[B // 2] = 60
    total = n + g.integers(0, 70, B)
    p = Paged(B, n.tolist(), total.tolist(), 2, 64, 16)
    _check(p, 4, max_q=min(hint or 1, p.T))


def test_wrong_hint_costs_time_only():
    import torch
    m = mx()
    p = Paged(18, [3, 70, 1], [400, 90, 33], 2, 128, 16)
    q = _q(p, 8)
    for hint in (1, 4, 70, p.T):
        _check(p, 8, q=q, max_q=hint)


def test_results_repeat_bit_for_bit():
    import torch
    m = mx()
    for n, total in (([1] * 9, [3000, 20, 1, 700, 700, 64, 5000, 90, 1200]), ([300, 50], [2000, 50])):
        p = Paged(19, n, total, 2, 128, 16)
        q = _q(p, 8)
        a = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q)
        for _ in range(3):
            assert torch.equal(a, m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q))


def test_long_context_past_32_bit_offsets():
    """A cache whose element offsets pass 2^32: pages at its far end."""
    import torch
    m = mx()
    pages, page, Hkv, D = 70000, 64, 8, 128          # 4.6e9 elements a plane
    k = torch.empty(pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    for n, total in (([1], [500]), ([100], [500])):
        p = Paged(20, n, total, Hkv, D, page, junk=0.0)
        far = torch.arange(p.n_pages, device="cuda") + (pages - p.n_pages)
        k[far], v[far] = p.k, p.v
        q = _q(p, 8)
        a = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q)
        b = m.paged_attention(q, k, v, p.cu, p.ctx, p.table + (pages - p.n_pages), max_q=p.max_q)
        assert torch.equal(a, b)
    assert status() == 0


def test_bad_batches_are_flagged_and_left_out():
    import torch
    m = mx()
    for n, total in (([1, 1], [40, 40]), ([100, 60], [140, 90])):
        p = Paged(21, n, total, 1, 64, 16, extra_width=1)
        q = _q(p, 2)
        good = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q)
        assert status() == 0
        bad = p.table.clone()
        bad[1, 0] = -3
        out = m.paged_attention(q, p.k, p.v, p.cu, p.ctx, bad, max_q=p.max_q)
        assert status() == 16 and torch.equal(out[: n[0]], good[: n[0]]) and torch.isfinite(out).all()
        cu = p.cu.clone()
        cu[2] += 1000
        m.paged_attention(q, p.k, p.v, cu, p.ctx, p.table, max_q=p.max_q)
        assert status() == 16
        ctx = p.ctx.clone()
        ctx[0] = 1 << 29
        m.paged_attention(q, p.k, p.v, p.cu, ctx, torch.zeros_like(p.table), max_q=p.max_q)
        assert status() == 16
        assert torch.equal(m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q), good) and status() == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,total", [([1, 2, 1], [90, 40, 17]),          # few rows, tiles left whole
                                     ([1, 2, 1], [3000, 40, 900]),       # few rows, tiles cut
                                     ([100, 30], [140, 30]),             # many rows, tiles left whole
                                     ([100, 30], [2900, 700])])          # many rows, tiles cut
def test_nan_in_a_query_stays_in_its_row(n, total, dim):
    import torch
    m = mx()
    p = Paged(24, n, total, 2, dim, 16)
    q = _q(p, 8)
    lse, clean_lse = (torch.empty(p.T, 8, device="cuda") for _ in range(2))
    clean = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q, lse=clean_lse)
    q[1, 3, 5] = float("nan")
    out = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q, lse=lse)
    assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3])
    out[1, 3], lse[1, 3] = clean[1, 3], clean_lse[1, 3]
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse) and status() == 0


@pytest.mark.parametrize("n,total,Hq", [([10, 1], [5, 300], 4), ([300, 30], [295, 700], 2)])
def test_largest_window_is_no_window(n, total, Hq):
    import torch
    m = mx()
    p = Paged(25, n, total, 2, 64, 16)     # the first tokens have negative positions
    q = _q(p, Hq)
    want = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q)
    for window in ((1 << 30) - 1, 1 << 30, (1 << 31) - 1):
        assert torch.equal(m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q, window=window), want)


def test_other_stream_and_given_workspace():
    import torch
    m = mx()
    for n, total in (([1] * 3, [4000, 100, 900]), ([200], [1500])):
        p = Paged(22, n, total, 2, 128, 32)
        q = _q(p, 8)
        want = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q)
        need = m.paged_attention_workspace_bytes(p.k, p.v, *p.batch(), n_tokens=p.T, n_heads=8, max_q=p.max_q)
        ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN bits: nothing stale is read
        out = torch.empty_like(q)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q, out=out, ws=ws, stream=st)
        st.synchronize()
        assert torch.equal(out, want)


def test_binding_refusals():
    import torch
    m = mx()
    p = Paged(23, [3], [40], 2, 64, 16, extra_width=100)   # wide enough to need a workspace
    q = _q(p, 4)
    b = p.batch()
    for bad in (lambda: m.paged_attention(q, p.k, p.v[:, :1], *b), lambda: m.paged_attention(q.half(), p.k, p.v, *b),
                lambda: m.paged_attention(q, p.k, p.v, p.cu.long(), p.ctx, p.table),
                lambda: m.paged_attention(q, p.k, p.v, p.cu[:1], p.ctx, p.table),
                lambda: m.paged_attention(q, p.k, p.v, *b, out=torch.empty(3, 4, 65, device="cuda")),
                lambda: m.paged_attention(q, p.k, p.v, *b, lse=torch.empty(3, 5, device="cuda")),
                lambda: m.rope_kv_write(torch.zeros(3, 100, device="cuda"), p.k, p.v, *b, n_heads=4),
                lambda: m.add_rms_norm(torch.zeros(2, 64, device="cuda"), torch.zeros(32, device="cuda")),
                lambda: m.add_rms_norm(torch.zeros(2, 64, device="cuda"), torch.zeros(64, device="cuda"),
                                       residual=torch.zeros(2, 64, device="cuda").half()),
                lambda: m.route_experts(torch.zeros(2, 64, device="cuda"), 2, bias=torch.zeros(63, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(m.MoexError):
        m.paged_attention(q, p.k, p.v, *b, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(m.MoexError):
        m.paged_attention(q, p.k, p.v, *b, scale=-1.0)


def test_workspace_belongs_to_the_given_stream():
    """Calls on a side stream that allocate their workspace and output, while the
    current stream takes and overwrites every block that comes free."""
    import torch
    m = mx()
    for n, total in (([1] * 3, [4000, 100, 900]), ([200], [1500])):
        p = Paged(24, n, total, 2, 128, 32)
        q = _q(p, 8)
        want = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q)
        need = m.paged_attention_workspace_bytes(p.k, p.v, *p.batch(), n_tokens=p.T, n_heads=8, max_q=p.max_q)
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        outs = []
        for _ in range(20):
            outs.append(m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q, stream=st))
            junk = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
            del junk
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
