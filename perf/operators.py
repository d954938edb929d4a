"""What the operators around a layer's quantized projections are measured on.

Four operators of a served mixture-of-experts layer, each in its plain form (elementary torch operations in 32 bits,
rounded once at the end) and through the library's entry points:

  norm    residual addition, root-mean-square norm, output as BF16 rows or as q8_1 blocks
  route   router scores (softmax or sigmoid), a balancing bias, expert groups, top-k, renormalised weights
  write   rotary embedding of new queries and keys, new keys and values into a paged cache
  attend  attention of every request's new tokens (one or a chunk) over its paged cache

hidden 2560, 128 experts with top-8 and 8192-token prompts are the repository's own layer; head counts are chosen so that
heads x head size gives 2560 or 4096 features.  `mix` seeds the ragged lengths of a case, so that its work does not depend
on the inputs' seed.
"""
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # the next token of one request between two layers: the residual row, normalised for the quantized products
        dict(name="norm_1x2560_q8", op="norm", T=1, H=2560, x="f32", out="q8"),
        # a full batch of single tokens; BF16 rows from a 16-bit product, both outputs wanted, an odd hidden size
        dict(name="norm_61x5152_both", op="norm", T=61, H=5152, x="bf16", out="both"),
        # a whole prompt of the repository's prefill workload
        dict(name="norm_8192x2560_bf16", op="norm", T=8192, H=2560, x="f32", out="bf16"),
        # the decode layer's window of three tokens, plain softmax routing over 128 experts
        dict(name="route_3x128_softmax", op="route", T=3, E=128, k=8, score="softmax", bias=False, groups=1,
             top_groups=1, renorm=True),
        # a prompt routed by sigmoid scores with a balancing bias inside four of eight groups
        dict(name="route_8192x256_groups", op="route", T=8192, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, renorm=True),
        # single tokens of five requests written into their caches
        dict(name="write_5_tokens", op="write", B=5, n=1, spread=1, ctx=900, mix=1, Hq=20, Hkv=4, D=128, page=16,
             type="bf16"),
        # prompts of different lengths, 8192 tokens at most, written at once
        dict(name="write_prompts", op="write", B=7, n=1170, spread=3, ctx=600, mix=2, Hq=32, Hkv=8, D=128, page=64,
             type="bf16"),
        # the next token of one request: latency
        dict(name="attend_one_token", op="attend", B=1, n=1, spread=1, ctx=1003, mix=3, Hq=32, Hkv=8, D=128, page=16,
             type="bf16", window=0),
        # a served batch: 64 requests, one token each, contexts over two orders of magnitude
        dict(name="attend_batch_64", op="attend", B=64, n=1, spread=1, ctx=16384, mix=4, Hq=32, Hkv=8, D=128, page=16,
             type="bf16", window=0),
        # a window of drafted tokens to verify in nine requests, FP16, 64-wide heads, a sliding window
        dict(name="attend_drafts", op="attend", B=9, n=5, spread=2, ctx=5000, mix=5, Hq=40, Hkv=8, D=64, page=32,
             type="f16", window=4096),
        # packed prompts without history
        dict(name="attend_prompts", op="attend", B=5, n=1637, spread=4, ctx=0, mix=6, Hq=20, Hkv=4, D=128, page=32,
             type="bf16", window=0),
        # a chunk of a long prompt over what is already in the cache
        dict(name="attend_chunk_2048", op="attend", B=1, n=2048, spread=1, ctx=14336, mix=7, Hq=32, Hkv=8, D=128,
             page=64, type="bf16", window=0),
    ]


def _log_int(rng, lo, hi):
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if v != 3072:
            return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["norm", "norm", "route", "route", "write", "attend", "attend", "attend"])
    if op == "norm":
        H = 32 * _log_int(rng, 4, 256)
        if H == 3072:
            H += 32
        return dict(op=op, T=_log_int(rng, 1, max(1, min(8192, 8192 * 2560 // H))), H=H,
                    x=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["q8", "bf16", "both"]))
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log_int(rng, 8 if groups > 1 else 16, 512 // groups)
        top = rng.randint(1, groups)
        return dict(op=op, T=_log_int(rng, 1, min(8192, 8192 * 256 // E)), E=E, k=rng.randint(1, min(12, E // groups * top)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, top_groups=top,
                    renorm=rng.random() < 0.7)
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 3, 4, 5, 8])
    c = dict(op=op, Hq=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
             type=rng.choice(["bf16", "bf16", "f16"]), mix=rng.randrange(1 << 20), spread=rng.randint(1, 4))
    if op == "write":
        c.update(B=_log_int(rng, 1, 48), ctx=rng.choice([0, _log_int(rng, 16, 2000)]))
        c["n"] = _log_int(rng, 1, max(1, 8192 // c["B"]))
        return c
    kind = rng.choice(["tokens", "tokens", "drafts", "prompts", "chunk"])
    c["window"] = rng.choice([0, 0, 0, _log_int(rng, 100, 5000)])
    if kind == "tokens":
        c.update(B=_log_int(rng, 1, 64), n=1, spread=1, ctx=_log_int(rng, 64, 16384))
    elif kind == "drafts":
        c.update(B=_log_int(rng, 1, 32), n=rng.randint(2, 9), ctx=_log_int(rng, 64, 8192))
    elif kind == "prompts":
        c.update(B=_log_int(rng, 1, 12), ctx=0)
        c["n"] = _log_int(rng, 20, 8000 // c["B"])
        c["n"] = min(c["n"], int((1.0e9 / (c["B"] * c["Hq"])) ** 0.5))  # the plain form holds every score
    else:
        c.update(B=1, spread=1, n=_log_int(rng, 100, 2048), ctx=_log_int(rng, 500, 14336))
    return c


def _lengths(c):
    """(new tokens, keys in the cache with them) of every request: ragged ones over a factor of `spread` in new tokens,
    and histories from a hundredth of `ctx` up to it (the first request has the longest)."""
    r = random.Random(c["mix"])
    n, total = [], []
    for b in range(c["B"]):
        nb = c["n"] if b == 0 or c["spread"] == 1 else max(1, int(round(c["n"] * math.exp(-r.random() * math.log(c["spread"])))))
        hist = c["ctx"] if b == 0 or c["ctx"] == 0 else int(c["ctx"] * math.exp(-r.random() * math.log(100)))
        n.append(nb)
        total.append(hist + nb)
    return n, total


# ------------------------------------------------------------------ inputs

_T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        # the residual stream grows along the layers and has a few large channels; gamma is around one
        channel = torch.exp(0.5 * normal(H))
        return dict(case=case, x=(normal(T, H) * 0.7).to(_T[case["x"]]), residual=normal(T, H) * 3.0 * channel,
                    gamma=1.0 + 0.2 * normal(H))
    if case["op"] == "route":
        return dict(case=case, **_router_inputs(case, normal))
    n, total = _lengths(case)
    B, T, page = case["B"], sum(n), case["page"]
    Hq, Hkv, D, dt = case["Hq"], case["Hkv"], case["D"], _T[case["type"]]
    per = [-(-t // page) for t in total]
    width = max(per)
    pages = sum(per) + 3  # a few pages belong to nobody
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)[: sum(per)]
    table = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    filled = torch.arange(width, device=DEV)[None, :] < torch.tensor(per, device=DEV)[:, None]
    table[filled] = order
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
    s = dict(case=case, table=table, cu=cu, ctx=torch.tensor(total, dtype=torch.int32, device=DEV), max_q=max(n),
             k=normal(pages, Hkv, page, D).to(dt), v=normal(pages, Hkv, page, D).to(dt), T=T, longest=max(total))
    if case["op"] == "write":
        # one row of a fused projection a token: queries, keys, values; a table of angles that a server keeps
        s["qkv"] = normal(T, (Hq + 2 * Hkv) * D)
        inv = 10000.0 ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
        ang = torch.arange(max(total), device=DEV, dtype=torch.float64)[:, None] * inv[None, :]
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()
    else:
        s["q"] = (normal(T, Hq, D) * 1.5).to(dt)  # scores spread by about 1.5: some keys matter, none is alone
    return s


def _router_inputs(c, normal):
    """Logits of a router's matrix product and a bias in steps of 1/1024, as a balancing rule moves it.  A token whose
    selection hangs on the last bits of a 32-bit score has no one right answer: it is drawn again."""
    T, E = c["T"], c["E"]
    bias = (normal(E) * 20).round() / 1024 if c["bias"] else None
    logits = normal(T, E)
    for _ in range(6):
        x = logits.double()
        s = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
        sel = s if bias is None else s + bias.double()
        tight = torch.zeros(T, dtype=torch.bool, device=DEV)
        if c["groups"] > 1:
            per = sel.view(T, c["groups"], -1)
            gs = per.topk(min(2, per.shape[2]), dim=2).values.sum(2)
            srt = gs.sort(1, descending=True)
            if c["top_groups"] < c["groups"]:
                tight |= srt.values[:, c["top_groups"] - 1] - srt.values[:, c["top_groups"]] < 2e-6
            keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, srt.indices[:, : c["top_groups"]], True)
            sel = per.masked_fill(~keep[:, :, None], -1e9).reshape(T, E)
        top = sel.topk(min(E, c["k"] + 1), dim=1).values
        tight |= (top[:, :-1] - top[:, 1:] < 2e-6).any(1)
        fresh = normal(T, E)
        logits = torch.where(tight[:, None], fresh, logits)
    return dict(logits=logits, bias=bias)


# ------------------------------------------------------------------ one pass


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _plain_norm(s):
    c = s["case"]
    total = s["x"].float() + s["residual"]
    y = total * torch.rsqrt(total.square().mean(1, keepdim=True) + EPS) * s["gamma"]
    out = {"sum": total}
    if c["out"] != "q8":
        out["y"] = y.bfloat16()
    if c["out"] != "bf16":
        b = y.view(c["T"], -1, 32)
        d = b.abs().amax(2, keepdim=True) / 127.0
        r = b / torch.where(d > 0, d, torch.ones_like(d))
        q = torch.sign(r) * torch.floor(r.abs() + 0.5)
        out["y_q8"] = (q * d).view(c["T"], -1).bfloat16()
    return out


def _plain_route(s):
    c, x = s["case"], s["logits"]
    if c["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    sel = score if s["bias"] is None else score + s["bias"]
    if c["groups"] > 1:
        per = sel.view(c["T"], c["groups"], -1)
        best = per.sort(dim=2, descending=True).values[:, :, :2].sum(2)
        keep = torch.zeros_like(best, dtype=torch.bool)
        keep.scatter_(1, best.sort(dim=1, descending=True, stable=True).indices[:, : c["top_groups"]], True)
        sel = per.masked_fill(~keep[:, :, None], -math.inf).reshape(c["T"], -1)
    ids = sel.sort(dim=1, descending=True, stable=True).indices[:, : c["k"]]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.int(), "w": w * 2.5}


def _places(s):
    """Request, position and cache slot of every new token."""
    tok = torch.arange(s["T"], device=DEV)
    req = torch.bucketize(tok, s["cu"][1:].long(), right=True)
    first = s["cu"][:-1].long()[req]
    count = (s["cu"][1:] - s["cu"][:-1]).long()[req]
    pos = s["ctx"].long()[req] - count + tok - first
    page = s["case"]["page"]
    return req, tok - first, pos, s["table"][req, pos // page].long(), pos % page


def _plain_write(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    _, _, pos, pg, off = _places(s)
    rows = s["qkv"].view(s["T"], Hq + 2 * Hkv, D)
    cos, sin = s["cos_sin"][pos][:, None, : D // 2], s["cos_sin"][pos][:, None, D // 2:]
    a, b = rows[:, : Hq + Hkv, : D // 2], rows[:, : Hq + Hkv, D // 2:]
    turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2).to(s["k"].dtype)
    s["k"][pg, :, off] = turned[:, Hq:]
    s["v"][pg, :, off] = rows[:, Hq + Hkv:].to(s["v"].dtype)
    return {"q": turned[:, :Hq].contiguous(), "k": s["k"], "v": s["v"]}


def _plain_attend(s):
    c = s["case"]
    Hq, Hkv, D, B = c["Hq"], c["Hkv"], c["D"], c["B"]
    L, N = s["longest"], s["max_q"]
    req, nth, pos, _, _ = _places(s)
    at = torch.arange(L, device=DEV)
    pg, off = s["table"].long()[:, at // c["page"]], (at % c["page"])[None, :].expand(B, L)
    k = s["k"][pg, :, off].float().permute(0, 2, 3, 1)  # [B, Hkv, D, L]
    v = s["v"][pg, :, off].float().permute(0, 2, 1, 3)  # [B, Hkv, L, D]
    q = torch.zeros(B, N, Hq, D, device=DEV)
    q[req, nth] = s["q"].float()
    where = torch.full((B, N), -1, dtype=torch.long, device=DEV)
    where[req, nth] = pos
    q = q.view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    p = torch.matmul(q, k).mul_(1.0 / math.sqrt(D)).view(B, Hkv, Hq // Hkv, N, L)
    seen = at[None, None, :] <= where[:, :, None]
    if c["window"]:
        seen &= at[None, None, :] > where[:, :, None] - c["window"]
    p = p.masked_fill_(~seen[:, None, None], -math.inf)
    top = p.amax(4, keepdim=True)
    p = p.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(4, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, L), v).view(B, Hkv, Hq // Hkv, N, D)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)[req, nth].to(s["q"].dtype)}


def _own_norm(s):
    import moe_expert_gb300 as mx
    out = s["case"]["out"]
    total, y, q, ds = mx.add_rms_norm(s["x"], s["gamma"], EPS, residual=s["residual"],
                                      y_dtype=None if out == "q8" else torch.bfloat16, quantize=out != "bf16")
    res = {"sum": total}
    if out != "q8":
        res["y"] = y
    if out != "bf16":
        res["y_q8"] = mx.dequantize_q8_1(q, ds, dtype=torch.bfloat16)
    return res


def _own_route(s):
    import moe_expert_gb300 as mx
    c = s["case"]
    ids, w = mx.route_experts(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                              top_groups=c["top_groups"], group_top=2 if c["groups"] > 1 else 1, renorm=c["renorm"],
                              scale=2.5)
    return {"ids": ids, "w": w}


def _own_write(s):
    import moe_expert_gb300 as mx
    q = mx.rope_kv_write(s["qkv"], s["k"], s["v"], s["cu"], s["ctx"], s["table"], n_heads=s["case"]["Hq"],
                         cos_sin=s["cos_sin"])
    return {"q": q, "k": s["k"], "v": s["v"]}


def _own_attend(s):
    import moe_expert_gb300 as mx
    return {"out": mx.paged_attention(s["q"], s["k"], s["v"], s["cu"], s["ctx"], s["table"], max_q=s["max_q"],
                                      window=s["case"]["window"])}


_plain = {"norm": _plain_norm, "route": _plain_route, "write": _plain_write, "attend": _plain_attend}
_own = {"norm": _own_norm, "route": _own_route, "write": _own_write, "attend": _own_attend}


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        out = (2 if c["out"] != "q8" else 0) + (1 + 8 / 32 + 2 if c["out"] != "bf16" else 0)  # q8_1, then its values
        return {"bytes": n * (4 + (4 if c["x"] == "f32" else 2) + 4 + out) + 4 * c["H"], "flops": 6 * n}
    if c["op"] == "route":
        return {"bytes": c["T"] * (4 * c["E"] + 8 * c["k"]) + (4 * c["E"] if c["bias"] else 0), "flops": 6 * c["T"] * c["E"]}
    n, total = _lengths(c)
    T, Hq, Hkv, D = sum(n), c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "write":
        return {"bytes": T * (4 * (Hq + 2 * Hkv) * D + 2 * (Hq + 2 * Hkv) * D) + 4 * D * min(T, max(total)),
                "flops": 3 * T * (Hq + Hkv) * D}
    w = c["window"] or 1 << 30
    keys = sum(min(t, w + nb - 1) for nb, t in zip(n, total))
    pairs = sum(sum(min(p + 1, w) for p in range(t - nb, t)) for nb, t in zip(n, total))
    return {"bytes": 2 * 2 * T * Hq * D + 2 * 2 * keys * Hkv * D, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "write": _exact_write, "attend": _exact_attend}[case["op"]](case, s)


def _exact_norm(c, s):
    x = s["x"].cpu().numpy().astype(np.float64) if c["x"] != "bf16" else s["x"].float().cpu().numpy().astype(np.float64)
    x = x + s["residual"].cpu().numpy().astype(np.float64)
    y = x / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + EPS) * s["gamma"].cpu().numpy().astype(np.float64)
    out = {"sum": x}
    if c["out"] != "q8":
        out["y"] = y
    if c["out"] != "bf16":
        blocks = y.reshape(c["T"], c["H"] // 32, 32)
        step = np.abs(blocks).max(axis=2, keepdims=True) / 127.0
        ratio = np.divide(blocks, step, out=np.zeros_like(blocks), where=step > 0)
        out["y_q8"] = (np.copysign(np.floor(np.abs(ratio) + 0.5), ratio) * step).reshape(c["T"], c["H"])
    return out


def _exact_route(c, s):
    x = s["logits"].cpu().numpy().astype(np.float64)
    if c["score"] == "softmax":
        p = np.exp(x - x.max(axis=1)[:, None])
        p /= p.sum(axis=1)[:, None]
    else:
        p = 1.0 / (1.0 + np.exp(-x))
    sel = p + (0.0 if s["bias"] is None else s["bias"].cpu().numpy().astype(np.float64)[None, :])
    if c["groups"] > 1:
        size = c["E"] // c["groups"]
        rank = -np.sort(-sel.reshape(c["T"], c["groups"], size), axis=2)[:, :, :2].sum(axis=2)
        chosen = np.argsort(-rank, axis=1, kind="stable")[:, : c["top_groups"]]
        allowed = np.zeros((c["T"], c["groups"]), bool)
        np.put_along_axis(allowed, chosen, True, axis=1)
        sel = np.where(np.repeat(allowed, size, axis=1), sel, -np.inf)
    ids = np.argsort(-sel, axis=1, kind="stable")[:, : c["k"]]
    w = np.take_along_axis(p, ids, axis=1)
    if c["renorm"]:
        w = w / w.sum(axis=1, keepdims=True)
    return {"ids": ids.astype(np.int32), "w": 2.5 * w}


def _exact_write(c, s):
    Hq, Hkv, D, half = c["Hq"], c["Hkv"], c["D"], c["D"] // 2
    n, total = _lengths(c)
    qkv = s["qkv"].cpu().numpy().astype(np.float64).reshape(s["T"], Hq + 2 * Hkv, D)
    k, v = (s[m].float().cpu().numpy().astype(np.float64) for m in ("k", "v"))
    angles, table = s["cos_sin"].cpu().numpy().astype(np.float64), s["table"].cpu().numpy()
    q = np.empty((s["T"], Hq, D))
    t = 0
    for b in range(c["B"]):
        for p in range(total[b] - n[b], total[b]):
            z = qkv[t, : Hq + Hkv, :half] + 1j * qkv[t, : Hq + Hkv, half:]
            z = z * (angles[p, :half] + 1j * angles[p, half:])  # a turn of the plane is a product of complex numbers
            z = np.concatenate([z.real, z.imag], axis=1)
            q[t] = z[:Hq]
            page, off = table[b, p // c["page"]], p % c["page"]
            k[page, :, off] = z[Hq:]
            v[page, :, off] = qkv[t, Hq + Hkv:]
            t += 1
    return {"q": q, "k": k, "v": v}


def _exact_attend(c, s):
    n, total = _lengths(c)
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device=DEV)
    start = 0
    for b in range(c["B"]):
        pages = s["table"][b, : -(-total[b] // page)].long()
        keys, values = (s[m][pages].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, : total[b]].double() for m in ("k", "v"))
        step = max(1, (1 << 26) // (G * total[b]))
        for i in range(0, n[b], step):  # a few query rows at a time, one key head after the other
            rows = s["q"][start + i: start + min(i + step, n[b])].double()
            p = torch.arange(total[b] - n[b] + i, total[b] - n[b] + i + rows.shape[0], device=DEV)[:, None]
            j = torch.arange(total[b], device=DEV)[None, :]
            hidden = (j > p) | (j <= p - c["window"]) if c["window"] else j > p
            for h in range(Hkv):
                scores = torch.einsum("ngd,ld->gnl", rows[:, h * G: (h + 1) * G], keys[h]) * D ** -0.5
                weight = torch.softmax(scores.masked_fill(hidden, -math.inf), dim=2)
                out[start + i: start + i + rows.shape[0], h * G: (h + 1) * G] = torch.einsum("gnl,ld->ngd", weight, values[h])
        start += n[b]
    return {"out": out}
