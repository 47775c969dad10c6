"""The router against a 64-bit form: scores, groups, ties, masked tokens and experts, its gradient.

Which experts are chosen has to be equal.  Tolerances, fixed before the first run.  A weight is scale * exp(l - m) / sum or
scale / (1 + exp(-l)): the argument's rounding leaves 2^-24 of its size (up to 30 here: 2^-19.1), exp 2^-22, a
sum of up to 2048 terms by 16 + 7 additions 23 * 2^-24 and 2^-22 of its terms, quotient and product 2^-23: together below
2^-17.5 = 5.4e-6.  A gradient is a product of two such factors and a difference of two sums of 32 products: 2^-16 of the sum of magnitudes,
and one rounding to its type."""
import pytest
import torch

from combine_get_dispatch_03_gb300 import ep
from _parity import Guarded
from test_gpu_experts import DEV, gen

pytestmark = pytest.mark.gpu
WEIGHT_EPS, GRAD_EPS = 2.0 ** -17.5, 2.0 ** -16


def handle(E, K, R=1, T=64, max_sms=0):
    return ep.Handle(ep.Config(num_ranks=R, num_max_tokens=T, hidden=128, num_experts=E, num_topk=K, max_sms=max_sms))


def reference(logits, K, bias=None, score="softmax", num_groups=1, kept_groups=1, normalize=True, scale=1.0, mask=None):
    """(topk_idx, topk_weights in 64 bits) by the definition."""
    E = logits.shape[-1]
    l = logits.double().reshape(-1, E)
    l = torch.where(l.isnan(), -torch.inf, l).clamp(max=torch.finfo(torch.float32).max)
    there = l > -torch.inf
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        m = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(m > -torch.inf, m, 0.0))
        s = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    key = s + bias.double() if bias is not None else s
    key = torch.where(there & ~key.isnan(), key, -torch.inf)
    if bias is None and num_groups == kept_groups:
        key = l  # the scores' order without their rounding
    if num_groups != kept_groups:
        parts = key.view(-1, num_groups, E // num_groups)
        top = torch.sort(parts, dim=-1, descending=True).values[..., :2].sum(-1)
        best = torch.sort(top, dim=-1, descending=True, stable=True).indices[:, :kept_groups]
        keep = torch.zeros_like(top, dtype=torch.bool).scatter_(1, best, True)
        key = torch.where(keep[..., None], parts, -torch.inf).view(key.shape)
    value, idx = (t[:, :K] for t in torch.sort(key, dim=1, descending=True, stable=True))
    if K > E:
        value = torch.nn.functional.pad(value, (0, K - E), value=-torch.inf)
        idx = torch.nn.functional.pad(idx, (0, K - E))
    none = value == -torch.inf
    if mask is not None:
        none = none | ~mask.reshape(-1, 1)
    idx = torch.where(none, -1, idx)
    c = torch.where(none, 0.0, s.gather(1, idx.clamp_min(0)))
    if normalize and score == "softmax":
        # the sum cancels: from the largest chosen logit, so that nothing underflows
        lc = torch.where(none, -torch.inf, l.gather(1, idx.clamp_min(0)))
        top = lc.amax(1, keepdim=True)
        c = torch.where(none, 0.0, torch.exp(lc - torch.where(top > -torch.inf, top, 0.0)))
    w = c / c.sum(1, keepdim=True).clamp_min(1e-300) if normalize else c
    return idx.view(*logits.shape[:-1], K), (scale * w).view(*logits.shape[:-1], K)


def check(h, logits, **kw):
    K = h.cfg.num_topk
    mask = kw.pop("token_mask", None)
    shape = tuple(logits.shape[:-1]) + (K,)
    idx, w = Guarded(shape, torch.int64), Guarded(shape, torch.float32)
    ep.ep_router(h, logits, token_mask=mask, topk_idx=idx.t, topk_weights=w.t, **kw)
    h.check()
    idx.check()
    w.check()
    want_idx, want_w = reference(logits, K, mask=mask, **dict(dict(kept_groups=kw.get("num_groups", 1)), **kw))
    assert torch.equal(idx.t, want_idx), f"{int((idx.t != want_idx).sum())} choices differ"
    assert ((w.t.double() - want_w).abs() <= WEIGHT_EPS * want_w.abs() + 1e-37).all()
    return idx.t, w.t


SIZES = [(1, 1), (5, 3), (32, 4), (33, 8), (64, 6), (96, 32), (128, 8), (160, 6), (256, 8), (264, 8), (384, 8), (512, 1),
         (700, 10), (2048, 32)]


@pytest.mark.parametrize("E,K", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("biased", [False, True])
def test_choice_and_weights(E, K, score, dtype, biased):
    g = gen(E * 3 + K)
    h = handle(E, K)
    for tokens in (1, 7, 600):
        logits = (torch.randn((tokens, E), generator=g, device=DEV) * 2).to(dtype)
        bias = torch.randn(E, generator=g, device=DEV) * 0.05 if biased else None
        for normalize in (True, False):
            check(h, logits, bias=bias, score=score, normalize=normalize, scale=2.5)


@pytest.mark.parametrize("E,K,groups,kept", [(256, 8, 8, 4), (64, 4, 32, 3), (96, 6, 3, 2), (160, 6, 8, 3), (48, 5, 16, 7),
                                             (512, 8, 16, 1), (40, 4, 20, 9), (32, 8, 32, 8), (2048, 16, 32, 5), (6, 2, 2, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(E, K, groups, kept, score, dtype, biased):
    g = gen(E + groups)
    logits = (torch.randn((500, E), generator=g, device=DEV) * 1.5).to(dtype)
    bias = torch.randn(E, generator=g, device=DEV) * 0.05 if biased else None
    check(handle(E, K), logits, bias=bias, score=score, num_groups=groups, kept_groups=kept)


@pytest.mark.parametrize("E,K", [(1, 32), (3, 8), (31, 32), (40, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_more_slots_than_experts_and_most_slots(E, K, score, normalize, biased):
    g = gen(E)
    bias = torch.randn(E, generator=g, device=DEV) * 0.05 if biased else None
    logits = torch.randn((37, E), generator=g, device=DEV)
    idx, _ = check(handle(E, K), logits, bias=bias, score=score, normalize=normalize)
    assert (idx[:, E:] == -1).all()
    dw = torch.randn((37, K), generator=g, device=DEV)
    dl = ep.ep_router_grad(handle(E, K), logits, idx, dw, score=score, normalize=normalize)
    want, mag = grad_reference(logits, idx, dw, score, normalize, 1.0)
    assert ((dl.double() - want).abs() <= GRAD_EPS * mag + 2.0 ** -24 * want.abs() + 1e-37).all()


@pytest.mark.parametrize("biased,groups", [(False, 1), (True, 1), (False, 4), (True, 4)])
def test_equal_logits(biased, groups):
    """More keys reach the bound than a warp has lanes."""
    bias = torch.zeros(256, device=DEV) if biased else None
    for score in ("softmax", "sigmoid"):
        same = torch.full((70, 256), 0.25, device=DEV)
        idx, _ = check(handle(256, 8), same, bias=bias, score=score, num_groups=groups, kept_groups=max(1, groups // 2))
        assert torch.equal(idx, torch.arange(8, device=DEV).expand(70, 8))
        same[:, 200] = 0.5
        check(handle(256, 8), same, bias=bias, score=score, num_groups=groups, kept_groups=max(1, groups // 2))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kw", [{}, dict(zero_bias=True), dict(num_groups=8, kept_groups=3), dict(num_groups=8, kept_groups=3, zero_bias=True)],
                         ids=["plain", "bias", "groups", "both"])
def test_ties_go_to_the_lowest(score, kw):
    """Few distinct logits: nearly every comparison ties."""
    kw = dict(kw)
    bias = torch.zeros(64, device=DEV) if kw.pop("zero_bias", False) else None
    g = gen(4)
    logits = torch.randint(-2, 3, (400, 64), generator=g, device=DEV).float()
    check(handle(64, 8), logits, bias=bias, score=score, **kw)
    same = torch.full((3, 64), -0.0, device=DEV)
    same[:, 1::2] = 0.0
    idx, _ = check(handle(64, 8), same, bias=bias, score=score, **kw)
    assert torch.equal(idx, torch.arange(8, device=DEV).expand(3, 8))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_keys_closer_than_32_bits(score, groups):
    """Logits and biases whose keys differ by less than fp32 holds: the choice of 64 bits."""
    g = gen(7)
    E, tokens = 128, 300
    base = torch.randn((tokens, 1), generator=g, device=DEV)
    logits = base + torch.randint(-40, 41, (tokens, E), generator=g, device=DEV) * 2.0 ** -22
    bias = torch.randint(-8, 9, (E,), generator=g, device=DEV) * 2.0 ** -26
    check(handle(E, 8), logits, bias=bias, score=score, num_groups=groups, kept_groups=max(1, groups // 2))
    # keys that saturate: sigmoids of 1 and of nearly 0
    far = torch.randint(0, 2, (tokens, E), generator=g, device=DEV) * 120.0 - 60.0 + logits
    check(handle(E, 8), far, bias=bias, score=score, num_groups=groups, kept_groups=max(1, groups // 2))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("normalize", [False, True])
def test_special_logits(score, biased, groups, normalize):
    g = gen(11)
    E = 32
    logits = torch.randn((12, E), generator=g, device=DEV)
    logits[0, 3] = float("nan")
    logits[1, :] = float("-inf")
    logits[2, 5:] = float("-inf")       # fewer than K are left
    logits[3, 7] = float("inf")
    logits[4, ::2] = float("-inf")
    logits[5, :] = float("nan")
    logits[6, 1:] = torch.finfo(torch.float32).min
    logits[7, :] = torch.finfo(torch.float32).min
    logits[8] *= 1e30
    logits[9, 10] = 3e38
    logits[10, 4:] = -200.0
    bias = torch.randn(E, generator=g, device=DEV) * 0.05 if biased else None
    if biased:
        bias[9], bias[20] = float("-inf"), float("nan")
    check(handle(E, 8), logits, bias=bias, score=score, num_groups=groups, kept_groups=max(1, groups // 2), normalize=normalize)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept", [(32, 1, 1), (32, 4, 2), (64, 8, 3), (48, 16, 5), (160, 8, 3), (256, 8, 4)])
def test_extreme_biases(score, E, groups, kept):
    """Biases that force experts in or to the end: infinite ones, the type's largest and lowest values, and large ones.  Beyond
    2^100 they count as that, so that the sums of two that compare groups stay finite."""
    g = gen(21 + E)
    logits = torch.randn((70, E), generator=g, device=DEV)
    values = torch.tensor([float("inf"), float("-inf"), float("nan"), 3.4e38, -3.4e38, 1e35, -1e35, 2.0 ** 90, -2.0 ** 90, 0.0, 0.1],
                          device=DEV)
    h = handle(E, 8)
    for case in range(6):
        bias = values[torch.randint(0, len(values), (E,), generator=g, device=DEV)]
        if case == 1:
            bias = torch.where(torch.arange(E, device=DEV) % 3 == 0, 0.0, torch.finfo(torch.float32).min)
        if case == 2:
            bias = torch.full((E,), float("inf"), device=DEV)
        if case == 3:
            bias = torch.where(torch.arange(E, device=DEV) % 8 < 2, float("inf"), 0.0)
        counts = torch.where(bias.isinf() & (bias < 0), bias, bias.clamp(-2.0 ** 100, 2.0 ** 100))
        kw = dict(score=score, num_groups=groups, kept_groups=kept)
        out = ep.ep_router(h, logits, bias=bias, **kw)
        want_idx, want_w = reference(logits, 8, bias=counts, **kw)
        assert torch.equal(out["topk_idx"], want_idx), case
        assert ((out["topk_weights"].double() - want_w).abs() <= WEIGHT_EPS * want_w.abs() + 1e-37).all()
    h.check()


def test_token_mask_shapes_streams_and_caps():
    g = gen(5)
    R, T, E, K = 4, 9, 64, 6
    logits = torch.randn((R, T, E), generator=g, device=DEV)
    mask = torch.rand((R, T), generator=g, device=DEV) < 0.5
    mask[1] = False
    h = handle(E, K, R)
    idx, w = check(h, logits, token_mask=mask)
    assert idx.shape == (R, T, K) and (idx[1] == -1).all() and (w[1] == 0).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = ep.ep_router(h, logits, token_mask=mask, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    small = ep.ep_router(handle(E, K, R, max_sms=1), logits, token_mask=mask)
    for o in (out, small):
        assert torch.equal(o["topk_idx"], idx) and torch.equal(o["topk_weights"], w)
    none = ep.ep_router(h, logits[:, :0])
    assert none["topk_idx"].shape == (R, 0, K)
    odd = torch.randn(E * 5 + 1, generator=g, device=DEV)[1:].view(5, E)  # not 16-byte aligned
    check(h, odd, score="sigmoid")
    h.check()


def grad_reference(logits, idx, dw, score, normalize, scale):
    """(d_logits, sum of magnitudes) in 64 bits, by the Jacobians written out."""
    E = logits.shape[-1]
    l, i, g = logits.double().view(-1, E), idx.view(-1, idx.shape[-1]), scale * dw.double().view(-1, idx.shape[-1])
    none = i < 0
    p = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    c = torch.where(none, 0.0, p.gather(1, i.clamp_min(0)))
    g = torch.where(none, 0.0, g)
    dc, mag = g, g.abs()
    if normalize:
        S = c.sum(1, keepdim=True).clamp_min(1e-300)
        dc = g / S - (g * c).sum(1, keepdim=True) / S ** 2
        mag = g.abs() / S + (g.abs() * c).sum(1, keepdim=True) / S ** 2
    ds, dm = (torch.zeros_like(l).scatter_add_(1, i.clamp_min(0), torch.where(none, 0.0, v)) for v in (dc, mag))
    if score == "sigmoid":
        out, m = ds * p * (1 - p), dm * p * (1 - p)
    else:
        out, m = p * (ds - (ds * p).sum(1, keepdim=True)), p * (dm + (dm * p).sum(1, keepdim=True))
    return out.view(logits.shape), m.view(logits.shape)


@pytest.mark.parametrize("E,K", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [False, True])
def test_gradient(E, K, score, dtype, normalize):
    g = gen(E + K)
    h = handle(E, K)
    for tokens in (1, 300):
        logits = (torch.randn((tokens, E), generator=g, device=DEV) * 2).to(dtype)
        idx = ep.ep_router(h, logits, score=score)["topk_idx"]
        idx[torch.rand(idx.shape, generator=g, device=DEV) < 0.1] = -1
        if K > 1 and tokens > 5:
            idx[3] = -1
            idx[4, 1] = idx[4, 0]  # the same expert twice
        dw = torch.randn((tokens, K), generator=g, device=DEV)
        out = Guarded((tokens, E), dtype)
        ep.ep_router_grad(h, logits, idx, dw, score=score, normalize=normalize, scale=1.5, d_logits=out.t)
        h.check()
        out.check()
        want, mag = grad_reference(logits, idx, dw, score, normalize, 1.5)
        tol = GRAD_EPS * mag + torch.finfo(dtype).eps / 2 * want.abs() + 1e-37
        assert ((out.t.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_gradient_against_differences(score, normalize):
    """sum(dw * weights) along a direction of the logits, the choice held."""
    g = gen(3)
    E, K, tokens = 40, 6, 64
    logits = torch.randn((tokens, E), generator=g, device=DEV)
    h = handle(E, K)
    idx = ep.ep_router(h, logits, score=score)["topk_idx"]
    dw, v = torch.randn((tokens, K), generator=g, device=DEV), torch.randn((tokens, E), generator=g, device=DEV).double()
    dl = ep.ep_router_grad(h, logits, idx, dw, score=score, normalize=normalize, scale=2.0).double()

    def f(l):
        p = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
        c = p.gather(1, idx)
        w = 2.0 * (c / c.sum(1, keepdim=True) if normalize else c)
        return (w * dw.double()).sum()

    step = 2.0 ** -13  # the difference is off by step^2 / 6 of third derivatives of order 1: 2.5e-9 a term
    slope = (f(logits.double() + step * v) - f(logits.double() - step * v)) / (2 * step)
    assert abs((dl * v).sum() - slope) <= GRAD_EPS * (dl * v).abs().sum() + 1e-7 * tokens * K


def test_bad_indexes_are_reported():
    h = handle(16, 2)
    logits, dw = torch.zeros((3, 16), device=DEV), torch.ones((3, 2), device=DEV)
    for bad in (16, -2, 1 << 40):
        idx = torch.tensor([[0, 1], [bad, 2], [3, -1]], device=DEV)
        out = Guarded((3, 16), torch.float32)
        ep.ep_router_grad(h, logits, idx, dw, normalize=False, d_logits=out.t)
        assert h.status() == 7
        out.check()
        fine = ep.ep_router_grad(h, logits, idx.clamp(-1, 15) * (idx != bad) - 1 * (idx == bad), dw, normalize=False)
        assert torch.equal(out.t, fine)
        h.check()


def test_refusals():
    h = handle(16, 2)
    l = torch.zeros((3, 16), device=DEV)
    for kw in (dict(score="max"), dict(num_groups=3), dict(num_groups=0), dict(num_groups=4, kept_groups=5), dict(num_groups=4, kept_groups=0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(bias=torch.zeros(15, device=DEV)),
               dict(token_mask=torch.ones(4, dtype=torch.bool, device=DEV)), dict(topk_idx=torch.zeros((3, 3), dtype=torch.int64, device=DEV))):
        with pytest.raises((ValueError, ep.EPError)):
            ep.ep_router(h, l, **kw)
    for bad in (l[:, :8], l.double().to(torch.float16), l.t(), l.cpu()):
        with pytest.raises((ValueError, TypeError)):
            ep.ep_router(h, bad)
    big = handle(2048, 1)
    with pytest.raises(ep.EPError):
        ep.ep_router(big, torch.zeros((1, 2048), device=DEV), num_groups=64, kept_groups=2)
    with pytest.raises(ValueError):
        ep.ep_router_grad(h, l, torch.zeros((3, 2), dtype=torch.int64, device=DEV), torch.zeros((2, 2), device=DEV))
    h.check()


def test_captured_and_replayed():
    g = gen(8)
    h = handle(256, 8)
    logits, dw = torch.randn((64, 256), generator=g, device=DEV), torch.randn((64, 8), generator=g, device=DEV)
    bias = torch.randn(256, generator=g, device=DEV) * 0.1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = ep.ep_router(h, logits, bias=bias, score="sigmoid", num_groups=8, kept_groups=4)
        dl = ep.ep_router_grad(h, logits, r["topk_idx"], dw, score="sigmoid")
    for _ in range(2):
        logits.copy_(torch.randn((64, 256), generator=g, device=DEV))
        graph.replay()
        want = ep.ep_router(h, logits, bias=bias, score="sigmoid", num_groups=8, kept_groups=4)
        assert torch.equal(r["topk_idx"], want["topk_idx"]) and torch.equal(r["topk_weights"], want["topk_weights"])
        assert torch.equal(dl, ep.ep_router_grad(h, logits, want["topk_idx"], dw, score="sigmoid"))
    h.check()
