"""Large vocabularies with a random number in the middle of a likely token's interval
and cuts in the middle of a step, so that every row has one answer."""
import pytest

from layer_cases import mx, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("V,R", [(262144, 1), (262143, 1), (262144, 24), (131073, 2), (2041, 2), (50257, 24), (128256, 70),
                                 (16385, 200), (151936, 40)])
@pytest.mark.parametrize("kw", [dict(), dict(top_k=50, top_p=0.9), dict(top_k=150), dict(top_k=1500, top_p=0.8),
                                dict(top_p=0.9), dict(top_p=0.5), dict(min_p=0.02)])
def test_large_vocabularies_every_row(V, R, kw, kind):
    """top_p lies in the middle of a token's share, min_p between two weights, u in the middle of the interval of a
    token of 1e-4 or more: 32-bit roundings (2e-6 of the sum) move a top_p cut by tokens of 4e-6 and the share that it
    lies in, 8e-6 together, every border by twice that, and a likely token's interval keeps its middle."""
    import torch
    m = mx()
    g = torch.Generator(device="cuda").manual_seed(V + R)
    x = torch.randn(R, V, device="cuda", generator=g) * 2
    x[:, :: V // 40] += 6
    x = x.to(torch.bfloat16 if kind == "bf16" else torch.float32)
    xs, order = x.double().sort(dim=1, descending=True, stable=True)
    e = torch.exp((xs - xs[:, :1]) / 0.9)
    args = dict(kw)
    if "top_k" in kw:
        e[:, kw["top_k"]:] = 0
    if "top_p" in kw:
        before = (e.cumsum(1) - e) / e.sum(1, keepdim=True)
        at = (before < kw["top_p"]).sum(1, keepdim=True) - 1
        p = (before + e / e.sum(1, keepdim=True) / 2).gather(1, at).float()
        args["top_p"] = p[:, 0].contiguous()
        e = e * (before < p.double())
    if "min_p" in kw:
        # the middle of the widest step between two weights around min_p
        near = e[:, :-1] / e[:, 1:] * ((e[:, :-1] < 2 * kw["min_p"]) & (e[:, 1:] > kw["min_p"] / 2))
        at = near.argmax(1, keepdim=True)
        low = (e.gather(1, at) * e.gather(1, at + 1)).sqrt().float()
        args["min_p"] = low[:, 0].contiguous()
        e = e * (e >= low.double())
    w = torch.zeros_like(e).scatter_(1, order, e)
    total = w.sum(1, keepdim=True)
    c = w.cumsum(1) / total
    likely = (w / total >= 1e-4).float()
    assert (likely.sum(1) > 0).all()
    for _ in range(4):
        want = torch.multinomial(likely, 1, generator=g)
        pr = w.gather(1, want) / total
        u = (c.gather(1, want) - pr / 2)[:, 0].float()
        ids, prob = m.sample_tokens(x, u, temperature=0.9, **args)
        assert torch.equal(ids.long(), want[:, 0])
        assert ((prob.double() - pr[:, 0]).abs() <= 2e-5 * pr[:, 0]).all() and status() == 0
