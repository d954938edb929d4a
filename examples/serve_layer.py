"""One mixture-of-experts transformer layer as a server runs it: a prompt in
chunks over a paged cache, then single tokens, all through the library's calls.

    add_rms_norm -> products for q, k, v -> rope_kv_write -> paged_attention
    -> output product -> add_rms_norm -> router product -> route_experts -> experts

A few tokens take the q8_1 GEMVs and moe_decode, a chunk takes the tensor-core
products and moe_prefill; both leave (residual, delta) for the next layer's norm.
Weights are random, so the output means nothing: the example shows the calls,
prints what they take, and checks that the two ways agree.

    python examples/serve_layer.py [--hidden 2560] [--prompt 600] [--tokens 8]
"""
import argparse
import os
import sys

import numpy as np

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))


class Layer:
    def __init__(self, hidden=2560, inter=1536, experts=128, top_k=8, heads=20, kv_heads=4, head_dim=128,
                 max_pos=4096, seed=0):
        import torch

        import moe_expert_gb300 as mx
        import synth
        g = synth.rng(seed)
        self.heads, self.kv_heads, self.dim, self.top_k = heads, kv_heads, head_dim, top_k

        def weight(fmt, rows, K, n=1):
            # random blocks, their FP16 scales such that inputs of unit variance give outputs of about that
            blocks = np.stack([synth.weight_blocks(fmt, g, rows, K) for _ in range(n)])
            scale = blocks[..., :2].copy().view(np.float16)
            blocks[..., :2] = (scale / np.float16(0.7 * K ** 0.5)).astype(np.float16).view(np.uint8)
            return mx.PackedWeight.from_gguf(fmt, blocks)

        self.w_qkv = weight("q8_0", (heads + 2 * kv_heads) * head_dim, hidden)
        self.w_out = weight("q8_0", hidden, heads * head_dim)
        self.w_router = weight("q8_0", experts, hidden)
        self.gate_up = weight("q8_0", 2 * inter, hidden, experts)
        self.down = weight("iq4_nl", hidden, inter, experts)
        gen = torch.Generator().manual_seed(seed)
        self.gamma1, self.gamma2 = ((1 + 0.1 * torch.randn(hidden, generator=gen)).cuda() for _ in range(2))
        self.balance = (torch.randn(experts, generator=gen) / 256).cuda()  # a balancing rule's bias
        inv = 10000.0 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)
        angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv[None, :]
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()

    def new_cache(self, pages, page=16):
        import torch
        shape = (pages, self.kv_heads, page, self.dim)
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda"), torch.empty(shape, dtype=torch.bfloat16,
                                                                                     device="cuda")

    def route(self, logits):
        import moe_expert_gb300 as mx
        return mx.route_experts(logits, self.top_k, score="sigmoid", bias=self.balance, groups=8, top_groups=4,
                                group_top=2)

    def few(self, residual, delta, cache, batch, max_q):
        """Up to eight tokens: every product reads its quantized weights once."""
        import torch

        import moe_expert_gb300 as mx
        T = residual.shape[0]
        s, _, q, ds = mx.add_rms_norm(delta, self.gamma1, residual=residual, quantize=True)
        qh = mx.rope_kv_write(mx.qgemv(self.w_qkv, q, ds), *cache, *batch, n_heads=self.heads, cos_sin=self.cos_sin)
        o = mx.paged_attention(qh, *cache, *batch, max_q=max_q, out_dtype=torch.float32)
        a = mx.qgemv(self.w_out, *mx.quantize_q8_1(o.view(T, -1)))
        s, y, q, ds = mx.add_rms_norm(a, self.gamma2, residual=s, y_dtype=torch.float32, quantize=True)
        ids, w = self.route(mx.qgemv(self.w_router, q, ds))
        return s, mx.moe_decode(self.gate_up, self.down, y, ids, w)

    def many(self, residual, delta, cache, batch, max_q):
        """A chunk of a prompt: every product on the tensor cores."""
        import torch

        import moe_expert_gb300 as mx
        T = residual.shape[0]
        s, y, _, _ = mx.add_rms_norm(delta, self.gamma1, residual=residual, y_dtype=torch.bfloat16)
        qh = mx.rope_kv_write(mx.dense_prefill(self.w_qkv, y), *cache, *batch, n_heads=self.heads, cos_sin=self.cos_sin)
        o = mx.paged_attention(qh, *cache, *batch, max_q=max_q)
        a = mx.dense_prefill(self.w_out, o.view(T, -1))
        s, y, _, _ = mx.add_rms_norm(a, self.gamma2, residual=s, y_dtype=torch.bfloat16)
        ids, w = self.route(mx.dense_prefill(self.w_router, y))
        return s, mx.moe_prefill(self.gate_up, self.down, y, ids, w)


def batch_of(new, total, tables):
    """cu_q, ctx_len, page_table of sequences with new[b] new tokens of total[b]."""
    import torch
    width = max(len(t) for t in tables)
    table = np.zeros((len(tables), width), np.int32)
    for b, t in enumerate(tables):
        table[b, : len(t)] = t
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return tuple(torch.from_numpy(a).cuda() for a in (cu, np.array(total, np.int32), table))


def serve(layer, prompt, tokens, page=16, chunk=256, seed=1):
    """A prompt of `prompt` tokens in chunks, then `tokens` single ones.  Returns
    the last rows of (residual, delta) computed once as single tokens and once as
    part of a chunk, [tokens, hidden] each."""
    import torch
    g = torch.Generator().manual_seed(seed)
    total = prompt + tokens
    x = torch.randn(total, layer.gamma1.numel(), generator=g).cuda()
    zero = torch.zeros_like(x)
    pages = -(-total // page)
    table = np.random.default_rng(seed).permutation(pages + 3)[:pages]
    cache = layer.new_cache(pages + 3, page)
    for at in range(0, prompt, chunk):
        n = min(chunk, prompt - at)
        layer.many(x[at:at + n], zero[at:at + n], cache, batch_of([n], [at + n], [table]), n)
    one = [layer.few(x[t:t + 1], zero[t:t + 1], cache, batch_of([1], [t + 1], [table]), 1) for t in range(prompt, total)]
    single = torch.cat([r for r, _ in one]), torch.cat([d for _, d in one])
    cache2 = layer.new_cache(pages + 3, page)
    r, d = layer.many(x, zero, cache2, batch_of([total], [total], [table]), total)
    return single, (r[prompt:], d[prompt:])


def main():
    import torch

    import moe_expert_gb300 as mx
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=2560)
    ap.add_argument("--inter", type=int, default=512)
    ap.add_argument("--experts", type=int, default=128, help="a multiple of 128: the router is a dense_prefill product too")
    ap.add_argument("--prompt", type=int, default=600)
    ap.add_argument("--tokens", type=int, default=8)
    a = ap.parse_args()
    layer = Layer(hidden=a.hidden, inter=a.inter, experts=a.experts, heads=a.hidden // 128,
                  kv_heads=4 if a.hidden % 512 == 0 else 1)
    single, chunk = serve(layer, a.prompt, a.tokens)
    for name, u, v in zip(("residual", "delta"), single, chunk):
        print(f"{name}: single tokens against one chunk, relative difference "
              f"{((u - v).norm() / v.norm()).item():.4f}")
    x = torch.randn(1, a.hidden, device="cuda")
    cache = layer.new_cache(256)
    for T, step in ((1, layer.few), (512, layer.many)):
        x = torch.randn(T, a.hidden, device="cuda")
        b = batch_of([T], [2000 + T], [np.arange(256)])
        for _ in range(3):
            step(x, x, cache, b, T)
        t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        t0.record()
        for _ in range(20):
            step(x, x, cache, b, T)
        t1.record()
        torch.cuda.synchronize()
        print(f"{T} new token(s) over 2000: {t0.elapsed_time(t1) / 20 * 1e3:.1f} us a layer")
    if mx.device_status():
        raise SystemExit("device status word set")


if __name__ == "__main__":
    main()
