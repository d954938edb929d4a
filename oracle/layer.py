"""The operators around a layer's quantized products (oracle; test infrastructure only).

Plain float64 restatements of the formulas in ``include/moex.h``:

    add_rms_norm     s = x + r;  y = s * gamma / sqrt(mean(s^2) + eps)
    route_experts    scores, bias, groups, top-k, weights
    rope_kv_write    (a, b) -> (a cos - b sin, b cos + a sin); tokens to slots
    paged_attention  softmax(scale q.k) v over the keys a position sees

Each is a loop over tokens in the order the formula is written, slow on purpose.
"""
from __future__ import annotations

import math

import numpy as np


def add_rms_norm(x, gamma, eps, residual=None):
    """Returns (s, y), float64 [T, H]."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    y = np.empty_like(s)
    for t in range(s.shape[0]):
        y[t] = s[t] * np.asarray(gamma, np.float64) / math.sqrt(float(np.mean(s[t] ** 2)) + eps)
    return s, y


def route_experts(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    """Returns (ids int64 [T, k], w float64 [T, k], margin [T]): margin is the
    smallest distance between two ranks (of experts or of groups) whose order
    decides the answer, so that a caller can tell a near tie from an error."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    size = E // groups
    ids = np.empty((T, k), np.int64)
    w = np.empty((T, k))
    margin = np.full(T, np.inf)
    for t in range(T):
        masked = np.isnan(x[t]) | (x[t] == -np.inf)
        p = np.zeros(E)
        if score == "softmax":
            if not masked.all():
                top = x[t][~masked].max()
                with np.errstate(invalid="ignore"):
                    z = np.where(x[t] == top, 0.0, x[t] - top)
                p[~masked] = np.exp(z[~masked])
                p /= p.sum()
        else:
            with np.errstate(over="ignore"):
                p[~masked] = 1.0 / (1.0 + np.exp(-x[t][~masked]))
        rank = p + (0.0 if bias is None else np.asarray(bias, np.float64))
        # (class, value): unmasked before masked
        stay = list(range(groups))
        if groups > 1:
            value = []
            for g in range(groups):
                best = sorted((rank[e] for e in range(g * size, (g + 1) * size) if not masked[e]), reverse=True)[:group_top]
                value.append((1, sum(best)) if best else (0, 0.0))
            order = sorted(range(groups), key=lambda g: (-value[g][0], -value[g][1], g))
            stay = order[:top_groups]
            if top_groups < groups:
                a, b = value[order[top_groups - 1]], value[order[top_groups]]
                if a[0] == b[0] == 1 and a[1] != b[1]:
                    margin[t] = min(margin[t], a[1] - b[1])
        cand = [e for g in stay for e in range(g * size, (g + 1) * size)]
        cand.sort(key=lambda e: (1, 0.0, e) if masked[e] else (0, -rank[e], e))
        for a, b in zip(cand[:k], cand[1:k + 1]):
            if not masked[a] and not masked[b] and rank[a] != rank[b]:
                margin[t] = min(margin[t], rank[a] - rank[b])
        ids[t] = cand[:k]
        w[t] = p[ids[t]]
        if renorm:
            tot = w[t].sum()
            w[t] = w[t] / tot if tot > 0 else 0.0
        w[t] *= scale
    return ids, w, margin


def places(cu_q, ctx_len):
    """[(sequence, position)] of every token."""
    out = []
    for b in range(len(ctx_len)):
        n = cu_q[b + 1] - cu_q[b]
        out += [(b, ctx_len[b] - n + i) for i in range(n)]
    return out


def rope(head, cos, sin, interleaved=False):
    """Turns the first 2 * len(cos) features of a head (float64)."""
    h = np.array(head, np.float64)
    half = len(cos)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        x, y = h[a], h[b]
        h[a], h[b] = x * cos[i] - y * sin[i], y * cos[i] + x * sin[i]
    return h


def rope_kv_write(qkv, k_cache, v_cache, cu_q, ctx_len, table, n_heads, cos_sin=None, interleaved=False):
    """Returns (q [T, n_heads, D], k_cache, v_cache), float64; caches [pages, heads, page, D]."""
    k, v = np.array(k_cache, np.float64), np.array(v_cache, np.float64)
    _, Hkv, page, D = k.shape
    rows = np.asarray(qkv, np.float64).reshape(len(qkv), n_heads + 2 * Hkv, D)
    q = np.zeros((len(qkv), n_heads, D))
    for t, (b, p) in enumerate(places(cu_q, ctx_len)):
        if p < 0:
            continue
        def turn(h):
            if cos_sin is None:
                return h
            half = cos_sin.shape[1] // 2
            return rope(h, cos_sin[p, :half].astype(np.float64), cos_sin[p, half:].astype(np.float64), interleaved)
        for h in range(n_heads):
            q[t, h] = turn(rows[t, h])
        for h in range(Hkv):
            k[table[b][p // page], h, p % page] = turn(rows[t, n_heads + h])
            v[table[b][p // page], h, p % page] = rows[t, n_heads + Hkv + h]
    return q, k, v


def paged_attention(q, k_cache, v_cache, cu_q, ctx_len, table, scale, window=0):
    """Returns (out [T, Hq, D], lse [T, Hq]) in float64."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    _, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    out = np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    for t, (b, p) in enumerate(places(cu_q, ctx_len)):
        lo = max(0, p - window + 1) if window else 0
        if p < lo:
            continue
        js = np.arange(lo, p + 1)
        pages = np.asarray(table[b])[js // page]
        k = np.asarray(k_cache[pages, :, js % page], np.float64)   # [L, Hkv, D]
        v = np.asarray(v_cache[pages, :, js % page], np.float64)
        for h in range(Hq):
            x = scale * (k[:, h // G] @ q[t, h])
            m = x.max()
            e = np.exp(x - m)
            out[t, h] = (e @ v[:, h // G]) / e.sum()
            lse[t, h] = m + math.log(e.sum())
    return out, lse
