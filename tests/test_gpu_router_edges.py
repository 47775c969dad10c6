"""The router where 32 bits tell keys apart no more: equal inputs at the last place that is chosen, biases that cancel, scores
below the least fp32 number."""
import pytest
import torch

from combine_get_dispatch_03_gb300 import ep
from test_gpu_experts import DEV, gen
from test_gpu_router import check, handle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [1, 2, 4])
@pytest.mark.parametrize("score,kw", [("sigmoid", {}), ("sigmoid", dict(num_groups=4, kept_groups=2)),
                                      ("softmax", dict(num_groups=4, kept_groups=2)), ("softmax", {})],
                         ids=["sigmoid", "sigmoid-groups", "softmax-groups", "softmax-bias"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_inputs_at_the_last_place(K, score, kw, dtype):
    """Two to four experts with the same logit, one of them at the last place, and up to two others whose logit is larger by less
    than their 32-bit scores show, among higher experts: in 64 bits these come first.

    Sigmoids of 14 to 28 differ from 1 by e^-14 to e^-28 and lie 0.125 e^-28 = 8e-14 apart at least, 700 times the 2^-53 of
    64 bits."""
    g = gen(100 + K)
    E, tokens = 64, 600
    # K - 1 experts that come first and far apart: by the bias, where there is one, and else by a logit that leads by much
    biased = not kw or score == "sigmoid"
    bias = torch.zeros(E, device=DEV) if biased else None
    logits = torch.full((tokens, E), -6.0, device=DEV)
    logits += torch.randn((tokens, E), generator=g, device=DEV) * 0.1
    if score == "sigmoid":
        base = torch.randint(14 * 8, 28 * 8, (tokens, 1), generator=g, device=DEV) / 8.0  # bf16 holds them
        more = base + 0.125
    else:
        base = torch.rand((tokens, 1), generator=g, device=DEV) * 0.1 + 0.25
        base = base.to(dtype).float()
        more = base + (2.0 ** -25 if dtype == torch.float32 else 2.0 ** -9)
    order = torch.rand((tokens, 16), generator=g, device=DEV).argsort(1)  # among the first 16 experts: one group of four
    same = 2 + torch.randint(0, 3, (tokens, 1), generator=g, device=DEV)
    larger = 1 + torch.randint(0, 2, (tokens, 1), generator=g, device=DEV)
    place = torch.arange(16, device=DEV).expand(tokens, 16)
    # the larger ones at the highest experts of those that take part, the equal ones below them
    taken = torch.sort(torch.where(place < same + larger, order, 99), dim=1).values
    for i in range(6):
        at = taken[:, i:i + 1]
        value = torch.where(place[:, i:i + 1] < same, base, more)
        there = (at < 99).squeeze(1)
        logits[there] = logits[there].scatter(1, at[there], value[there])
    for j in range(K - 1):
        e = 16 + j  # the second group
        if biased:
            logits[:, e] = 0.5
            bias[e] = 2.0 + j
        else:
            logits[:, e] = 4.0 + j
    check(handle(E, K), logits.to(dtype), bias=bias, score=score, **kw)


def test_saturated_scores_by_hand():
    """Logits 18, 18 and 18.125, all of whose 32-bit sigmoids are 1: the third expert is the largest in 64 bits."""
    logits = torch.full((1, 32), -5.0, device=DEV)
    logits[0, 3], logits[0, 9], logits[0, 20] = 18.0, 18.0, 18.125
    idx, _ = check(handle(32, 1), logits, bias=torch.zeros(32, device=DEV), score="sigmoid")
    assert idx.tolist() == [[20]]
    idx, _ = check(handle(32, 1), logits, score="sigmoid", num_groups=4, kept_groups=3)
    assert idx.tolist() == [[20]]
    idx, _ = check(handle(32, 2), logits, bias=torch.zeros(32, device=DEV), score="sigmoid")
    assert idx.tolist() == [[20, 3]]


@pytest.mark.parametrize("E,groups,kept", [(64, 8, 4), (256, 8, 4), (160, 8, 3), (96, 32, 9), (32, 16, 8), (512, 4, 1)])
@pytest.mark.parametrize("size", [16.0, 64.0, 1000.0])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_that_cancel_in_a_group(E, groups, kept, size, score):
    """A group's two largest keys with large biases of opposite sign: each is rounded at its own size, and their sum is small.

    Scores of neighbouring groups lie about 1e-5 apart; 64 bits round a key of 1000 by 1e-13."""
    g = gen(E + int(size))
    each = E // groups
    bias = torch.full((groups, each), -4.0 * size, device=DEV)
    first = torch.rand((groups, each), generator=g, device=DEV).argsort(1)
    bias.scatter_(1, first[:, :1], size)
    bias.scatter_(1, first[:, 1:2], -size)
    logits = torch.randn((2000, 1), generator=g, device=DEV) + torch.randn((2000, E), generator=g, device=DEV) * 1e-4
    check(handle(E, 2), logits, bias=bias.view(-1), score=score, num_groups=groups, kept_groups=kept)
    # beside a group of small biases, whose sum 32 bits have right
    bias[0] = torch.randn(each, generator=g, device=DEV) * 0.01
    check(handle(E, 2), logits, bias=bias.view(-1), score=score, num_groups=groups, kept_groups=kept)


def far_logits(g, tokens, E):
    """Logits of -80 to -200, of -600 to -700, of both, and beside an ordinary one."""
    l = -80 - 120 * torch.rand((tokens, E), generator=g, device=DEV)
    l[1::4] = -600 - 100 * torch.rand((l[1::4].shape[0], E), generator=g, device=DEV)
    l[2::4, ::2] = -600 - 100 * torch.rand(l[2::4, ::2].shape, generator=g, device=DEV)
    l[3::4, 0] = torch.randn(l[3::4, 0].shape, generator=g, device=DEV)
    l[0, :3] = torch.tensor([-90.0, -91.0, -89.0])
    return l


def far_weights(l, idx):
    """Normalised sigmoids in 64 bits from their logarithms, so that nothing underflows."""
    c = torch.nn.functional.logsigmoid(l.double().gather(1, idx))
    return torch.softmax(c, 1)


@pytest.mark.parametrize("E,K", [(3, 2), (32, 8), (160, 6), (256, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("groups", [1, 2])
def test_normalised_sigmoids_of_low_logits(E, K, dtype, groups):
    """Scores below the least fp32 number have weights all the same: s / sum, from which the largest score cancels.

    A weight's argument l - max is rounded by 2^-18 at most (it is below 128 wherever the weight is above 1e-37), exp and the
    quotient by 2^-22, the sum of 32 by 31 * 2^-24: 2^-17 together.  A gradient is scale * u * (dw - sum dw u) * (1 - s): two
    such factors, 2^-15.5 of the magnitudes, and one rounding to its type."""
    if E % groups or K > E // groups:
        groups = 1
    g = gen(E + K)
    h = handle(E, K)
    l = far_logits(g, 401, E).to(dtype)
    if groups > 1:
        l[:, E // 2:] = -704.0  # the first half stays
    r = ep.ep_router(h, l, score="sigmoid", scale=2.5, num_groups=groups, kept_groups=max(1, groups // 2))
    h.check()
    idx, w = r["topk_idx"], r["topk_weights"].double()
    want_idx = torch.sort(l.double()[:, :E // groups], dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(idx, want_idx)
    want = 2.5 * far_weights(l, idx)
    assert ((w - want).abs() <= 2.0 ** -17 * want + 1e-37).all()
    assert ((w.sum(1) - 2.5).abs() <= 2.5 * 2.0 ** -17).all()
    dw = torch.randn((401, K), generator=g, device=DEV)
    dl = ep.ep_router_grad(h, l, idx, dw, score="sigmoid", scale=2.5).double()
    u, rest = want / 2.5, torch.sigmoid(-l.double().gather(1, idx))
    d = 2.5 * u * (dw.double() - (dw.double() * u).sum(1, keepdim=True)) * rest
    mag = 2.5 * u * (dw.double().abs() + (dw.double().abs() * u).sum(1, keepdim=True)) * rest
    want = torch.zeros_like(dl).scatter_(1, idx, d)
    mag = torch.zeros_like(dl).scatter_(1, idx, mag)
    assert ((dl - want).abs() <= 2.0 ** -15.5 * mag + torch.finfo(dtype).eps / 2 * want.abs() + 1e-37).all()


def test_sigmoids_that_64_bits_do_not_hold():
    """Below -709.78 a score is 0 in 64 bits too: no weight, and no gradient."""
    h = handle(16, 4)
    l = torch.full((4, 16), -800.0, device=DEV)
    l[1, 5] = -700.0
    l[2] = torch.finfo(torch.float32).min
    l[3, 2], l[3, 7] = 1.0, 2.0
    idx, w = check(h, l[[0, 2, 3]].contiguous(), score="sigmoid")
    assert (w[:2] == 0).all()
    r = ep.ep_router(h, l, score="sigmoid")
    assert r["topk_idx"][1].tolist() == [5, 0, 1, 2] and r["topk_weights"][1].tolist() == [1.0, 0.0, 0.0, 0.0]
    dl = ep.ep_router_grad(h, l, r["topk_idx"], torch.ones((4, 4), device=DEV), score="sigmoid")
    assert (dl[:3] == 0).all()
    h.check()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_normalised_expert_has_no_gradient(score, dtype):
    """With one expert a token and normalised weights the weight is the scale, whatever the logits are: the gradient is 0, not what
    rounding leaves of a difference."""
    g = gen(31)
    h = handle(40, 1)
    logits = (torch.randn((300, 40), generator=g, device=DEV) * 3).to(dtype)
    r = ep.ep_router(h, logits, score=score, scale=2.5)
    assert (r["topk_weights"] == 2.5).all()
    dl = ep.ep_router_grad(h, logits, r["topk_idx"], torch.randn((300, 1), generator=g, device=DEV), score=score, scale=2.5)
    assert (dl == 0).all()
    h.check()


@pytest.mark.parametrize("E,groups,kept", [(16, 4, 1), (64, 8, 3), (256, 8, 4), (160, 8, 3)])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scores_next_to_the_least_number(E, groups, kept, biased, dtype):
    """Sigmoids around 2^-126 (a logit of -87.3), of which 32 bits keep some and flush others to 0: a group of two that are flushed
    can be worth more than one with a single score that is not."""
    g = gen(E)
    logits = (torch.randn((4000, E), generator=g, device=DEV) * 1.5 - 88).to(dtype)
    check(handle(E, 4), logits, bias=torch.zeros(E, device=DEV) if biased else None, score="sigmoid", num_groups=groups, kept_groups=kept)
