"""What a served layer's attention and experts add, token by token, as single tokens and inside a chunk, over both caches.

The two ways differ by their activations: q8_1 in front of the single tokens' products, FP16 in front of the chunk's.  A
q8_1 block of 32 normal values has a largest of about 2.1 and steps of 2.1 / 127, an error of a step / sqrt(12), 0.5% of
the values; a product's outputs take the same share.  On the way to the attention's contribution there are two such
products (one of them also moves the scores of the queries, whose few hundred weights move as much and average), to the
experts' two more and the weights of the experts: below 1% and 1.5% by root mean square, over 512 numbers, so no token
comes near four times that.  Half a page lost to one token of 300 keys is sqrt(8 / 300), 16%."""
import numpy as np
import pytest

from test_gpu_layer import _example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "q8"])
@pytest.mark.parametrize("prompt,tokens", [(300, 24), (17, 40)])
def test_every_token_as_inside_a_chunk(cache, prompt, tokens):
    import torch

    import moe_expert_gb300 as mx
    ex = _example()
    layer = ex.Layer(hidden=512, inter=256, experts=128, heads=8, kv_heads=2, head_dim=64, cache=cache)
    routed, route = [], layer.route
    layer.route = lambda logits: routed.append(route(logits)) or routed[-1]
    (r1, d1), (r2, d2) = ex.serve(layer, prompt=prompt, tokens=tokens, chunk=128)
    x = torch.randn(prompt + tokens, 512, generator=torch.Generator().manual_seed(1)).cuda()[prompt:]  # as in serve
    a1, a2 = r1 - x, r2 - x
    off = (a1 - a2).norm(dim=1) / a2.norm(dim=1)
    assert (off < 0.04).all(), off.max().item()
    single = torch.cat([ids for ids, _ in routed[-1 - tokens:-1]]).sort(dim=1).values
    chunk = routed[-1][0][prompt:].sort(dim=1).values
    same = (single == chunk).all(dim=1)
    off = (d1 - d2).norm(dim=1) / d2.norm(dim=1)
    assert same.sum() >= tokens // 2 and (off[same] < 0.06).all(), (int(same.sum()), off[same].max().item())
    assert mx.device_status() == 0
