"""Shared inputs and bounds of the tests of the operators around a layer's products."""
import numpy as np

from helpers import ensure_lib, to_np

U32 = 2.0 ** -24            # FP32 unit roundoff
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # 2^-p for p significant bits
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}   # half the spacing of FP16 subnormals


def dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def mx():
    import moe_expert_gb300
    ensure_lib()
    return moe_expert_gb300


def f64(t):
    return to_np(t.float()).astype(np.float64)


def status():
    return mx().device_status()


class Paged:
    """A random paged cache and a batch over it: new tokens n[b], lengths
    total[b] (the new tokens included).  Slots that no position of the batch
    holds, and pages that belong to nobody, are filled with `junk`."""

    def __init__(self, seed, n, total, Hkv, D, page, kind="bf16", layout="hpd", junk=float("nan"), extra_pages=3,
                 extra_width=0):
        import torch
        g = np.random.Generator(np.random.PCG64(seed))
        self.n, self.total, self.page, self.Hkv, self.D, self.kind = list(n), list(total), page, Hkv, D, kind
        per = [max(0, -(-t // page)) for t in total]
        self.n_pages = sum(per) + extra_pages
        self.width = max(max(per), 1) + extra_width
        ids = g.permutation(self.n_pages)
        table = np.full((len(n), self.width), -7, np.int32)   # never read past a sequence's pages
        live = np.zeros((self.n_pages, page), bool)
        at = 0
        for b, p in enumerate(per):
            table[b, :p] = ids[at:at + p]
            at += p
            for j in range(max(0, total[b])):
                live[table[b, j // page], j % page] = True
        self.table_np = table
        self.cu_np = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.ctx_np = np.array(total, np.int32)
        shape = (self.n_pages, Hkv, page, D)
        dt = dtype(kind)

        def plane():
            x = torch.from_numpy(g.standard_normal(shape).astype(np.float32))
            x[~torch.from_numpy(live)[:, None, :].expand(-1, Hkv, -1)] = junk
            x = x.to(dt)
            if layout == "phd":      # [page][slot][head][dim] memory seen as [page][head][slot][dim]
                x = x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
            elif layout == "pool":   # a layer's slice of a larger pool
                big = torch.full((self.n_pages, 3, Hkv, page, D + 8), junk, dtype=dt, device="cuda")
                big[:, 1, :, :, :D] = x.cuda()
                x = big[:, 1, :, :, :D]
            else:
                x = x.cuda()
            return x

        self.k, self.v = plane(), plane()
        self.cu, self.ctx, self.table = (torch.from_numpy(a).cuda() for a in (self.cu_np, self.ctx_np, table))
        self.T = int(sum(n))
        self.max_q = max(1, max(n))
        self.g = g

    def batch(self):
        return self.cu, self.ctx, self.table


def attention_bound(p, q, scale, window, G):
    """(out, lse, tolerance of out, tolerance of lse) of the formula in 64 bits.

    With A = sum_j p_j |v_j| (p the softmax) an element may be off by the
    rounding of each probability to 16 bits (half an ulp of p_j |v_j|, and half
    a subnormal spacing for FP16, the largest probability being 1 or more before
    the division), the rounding of the result, and by the FP32 score sums:
    D products of FP32 partial sums are off by at most D * 2^-24 * |q|.|k| scale,
    which moves every p_j by that relative amount twice (numerator, sum)."""
    from oracle import layer as ol
    kind = p.kind
    out, lse = ol.paged_attention(q, f64(p.k), f64(p.v), p.cu_np, p.ctx_np, p.table_np, scale, window)
    D = q.shape[2]
    finite = lambda a: np.where(np.isfinite(a), a, 0.0)  # noqa: E731
    va, ka = finite(np.abs(f64(p.v))), finite(np.abs(f64(p.k)))
    A, _ = ol.paged_attention(q, f64(p.k), va, p.cu_np, p.ctx_np, p.table_np, scale, window)
    # |q|.|k| is at most the product of the two lengths
    s = scale * np.sqrt((q ** 2).sum(2).max(initial=0.0) * (ka ** 2).sum(3).max(initial=0.0))
    es = 2 * (D + 4) * U32 * s + 64 * U32
    h = HALF_ULP[kind]
    sub = 0.0
    if kind == "f16":
        sub = TINY[kind] * max(p.total + [1]) * va.max(initial=0.0)
    tol = h * 1.02 * A + h * 1.02 * np.abs(out) + es * A + sub + TINY[kind]
    return out, lse, tol, es + 4 * U32 * np.abs(np.where(np.isfinite(lse), lse, 0.0)) + 64 * U32
