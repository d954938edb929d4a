"""The layer operators used together, as examples/serve_layer.py uses them."""
import importlib.util
import os

import numpy as np
import pytest

from helpers import ROOT, ensure_lib

pytestmark = pytest.mark.gpu


def _example():
    ensure_lib()
    spec = importlib.util.spec_from_file_location("serve_layer", os.path.join(ROOT, "examples", "serve_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_single_tokens_agree_with_chunks():
    """The same tokens as single ones (q8_1 activations, 8 bits a value: about
    0.4% of a product's norm) and inside a chunk (FP16 activations).  A router
    score within that error of its neighbour may send a token elsewhere, so the
    residual (before the experts) is compared for all, the experts' output for
    most."""
    import torch

    import moe_expert_gb300 as mx
    ex = _example()
    layer = ex.Layer(hidden=512, inter=256, experts=128, heads=8, kv_heads=2, head_dim=64)
    (r1, d1), (r2, d2) = ex.serve(layer, prompt=300, tokens=6, chunk=128)
    assert ((r1 - r2).norm() / r2.norm()).item() < 0.02
    off = (d1 - d2).norm(dim=1) / d2.norm(dim=1)
    assert (off < 0.1).float().mean().item() >= 0.5
    assert torch.isfinite(d1).all() and mx.device_status() == 0


def test_batch_of_tokens_equals_each_alone():
    """Eight sequences' next tokens in one call give each sequence what it gets
    alone: products and experts are bitwise column by column, attention splits the
    keys otherwise (its own tolerance, carried through one q8_1 product)."""
    import torch

    import moe_expert_gb300 as mx
    ex = _example()
    layer = ex.Layer(hidden=512, inter=256, experts=128, heads=8, kv_heads=2, head_dim=64)
    total = [5, 33, 64, 200, 1, 17, 90, 301]
    per = [-(-t // 16) for t in total]
    pages = np.random.default_rng(0).permutation(sum(per))
    tables = np.split(pages, np.cumsum(per)[:-1])
    k, v = layer.new_cache(sum(per))
    g = torch.Generator(device="cuda").manual_seed(3)
    k.normal_(generator=g)
    v.normal_(generator=g)
    x = torch.randn(8, 512, device="cuda", generator=g)
    s, d = layer.few(x, x, (k.clone(), v.clone()), ex.batch_of([1] * 8, total, tables), 1)
    for b in range(8):
        s1, _ = layer.few(x[b:b + 1], x[b:b + 1], (k.clone(), v.clone()), ex.batch_of([1], [total[b]], [tables[b]]), 1)
        assert ((s[b] - s1[0]).norm() / s1.norm()).item() < 0.01
    assert mx.device_status() == 0
