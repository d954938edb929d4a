"""Cuts among tokens of tiny probability, and the same rows in batches of other sizes.

Masses are multiples of 2^-43 of the likeliest token's, so one below 2^-20 of it is
rounded; sums of many have to be those of the rounded numbers wherever they are
taken, or a cut may lie where no token is found."""
import numpy as np
import pytest

from layer_cases import mx, status

pytestmark = pytest.mark.gpu
LAST = 1 - 2.0 ** -24     # the largest number below 1
LN2 = float(np.log(2.0))


def _tails(V, many, every, shift, counts):
    """A row: token 0 alone, `many` equal tokens of about 2^-shift of it, and some hundred of 2^-34, which together
    weigh about the 2^-24 that a top_p of LAST takes off, so that the cut lies at the end of the equal ones; rows differ
    in the equal ones' weight and in the number of the smallest."""
    import torch
    x = torch.full((8 * len(counts), V), -float("inf"), device="cuda")
    x[:, 0] = 0
    equal = 1 + every * torch.arange(many, device="cuda")
    small = (2 if every > 1 else 1 + many) + every * torch.arange(max(counts), device="cuda")
    for r in range(len(x)):
        x[r, equal] = -(shift + (r % 8) / 16) * LN2
        x[r, small[: counts[r // 8]]] = -34 * LN2
    return x, int(equal[-1])


@pytest.mark.parametrize("V,many,every,counts", [(140000, 27900, 5, range(1000, 1128, 4)), (16000, 9000, 1, range(1012, 1044)),
                                                 (60000, 9000, 6, range(1012, 1044))])
@pytest.mark.parametrize("shift", [25.25, 30.5])
def test_cut_behind_many_tiny_tokens(V, many, every, counts, shift):
    """u = LAST asks for the last of the tokens that stay: 2^-24 of the weight is 2^(shift - 24) equal tokens, as much
    again is what the cut may take, and the FP32 roundings of the equal tokens' own weight (2^-22 of it) are fewer."""
    import torch
    m = mx()
    x, last = _tails(V, many, every, shift, list(counts))
    R = len(x)
    ids, prob = torch.full((R,), -7, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
    m.sample_tokens(x, torch.full((R,), LAST, device="cuda"), top_p=LAST, ids=ids, prob=prob)
    room = every * (3 * 2 ** max(shift + 0.5 - 24, 0) + 3)
    far = (ids < last - room) | (ids > last + room)
    assert not far.any(), (int(far.sum()), ids[far][:8].tolist(), last)
    e = torch.exp2(-(shift + (torch.arange(R, device="cuda") % 8) / 16).double())
    assert ((prob.double() / (e / (1 + many * e)) - 1).abs() < 1e-3).all() and status() == 0
    m.sample_tokens(x, torch.full((R,), 0.25, device="cuda"), top_p=LAST, ids=ids, prob=prob)
    assert (ids == 0).all() and (prob > 0.9).all()


@pytest.mark.parametrize("V,many,every", [(16000, 9000, 1), (60000, 9000, 6)])
def test_a_row_gets_the_same_in_every_batch(V, many, every):
    """Bit for bit, however many CTAs a row has (the more rows, the fewer)."""
    import torch
    m = mx()
    for shift, p in ((25.25, LAST), (30.5, LAST), (23.0, 0.9995), (21.0, 0.998), (14.0, 0.8), (12.0, 0.8)):
        x, _ = _tails(V, many, every, shift, list(range(1012, 1044)))
        g = torch.Generator(device="cuda").manual_seed(2)
        x[1::2] += 0.5 * torch.randn(len(x) // 2, V, device="cuda", generator=g)
        u = torch.full((len(x),), LAST, device="cuda")
        ids, prob = m.sample_tokens(x, u, top_p=p)
        for size in (1, 9, 40, 100):
            for at in range(0, len(x), max(size, 4)):
                i, q = m.sample_tokens(x[at:at + size], u[at:at + size], top_p=p)
                assert torch.equal(i, ids[at:at + size]) and torch.equal(q, prob[at:at + size]), (shift, p, size, at)
    assert status() == 0


def test_ends_of_fp32():
    """Temperatures below 4.8e-39 count as that, a difference of logits beyond FP32's largest number as infinite."""
    import torch
    m = mx()
    big = float(np.finfo(np.float32).max)
    u = torch.tensor([0.01, LAST], device="cuda")
    x = torch.tensor([[3.0, 3.5, -7.0], [-7.0, 3.5, 3.0]], device="cuda")
    for t in (1e-45, 1e-40, 5e-39):
        ids, prob = m.sample_tokens(x, u, temperature=t, top_p=0.9)
        assert ids.tolist() == [1, 1] and prob.tolist() == [1, 1]
    x = torch.tensor([[-big, big, -big], [-big, 0.0, big]], device="cuda")
    ids, prob = m.sample_tokens(x, u, temperature=1e38)
    e = float(np.exp(-big / 1e38))     # of a difference that FP32 holds
    assert ids.tolist() == [1, 2] and prob[0] == 1 and abs(prob[1].item() * (1 + e) - 1) < 1e-5 and status() == 0
