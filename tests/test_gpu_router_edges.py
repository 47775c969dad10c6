"""The router where 32 bits tell keys apart no more: equal inputs at the last place that is chosen, biases that cancel."""
import pytest
import torch

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
