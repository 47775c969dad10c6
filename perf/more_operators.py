"""Operators around the experts: the router in front of a dispatch, products with an epilogue, a layer for a few tokens.

Three operators, each in a plain form (elementary torch operations in 32 bits, rounded once at the end; the router's
keys in 64, since close ones decide which experts are chosen) and as this package's calls:

  router   logits to the experts of every token and their weights, and the logits' gradient (ep_router,
           ep_router_grad)
  product  rows grouped by expert times bf16 weights, with bias, activation (gated or not), routing weight and
           residual in the epilogue, and the epilogue's gradient (ep_grouped_gemm_act, ep_act_grad); one group makes a
           dense product
  layer    a whole mixture-of-experts layer for at most 64 tokens, with bf16 or FP8 weights (ep_moe_layer)

Set `own` to True to make `run` call the package.  Rows of expert e are [begin[e], begin[e] + count[e]).
"""
import math

import torch

own = False

GROUP = 128  # weights of one FP8 scale: 128 x 128
DEV = "cuda"


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a training batch (8 ranks x 4096 tokens, 256 experts): sigmoid scores, selection bias, 4 of 8 groups
        dict(name="router_train", op="router", form="forward", ranks=8, tokens=4096, experts=256, topk=8, score="sigmoid",
             dtype="fp32", biased=True, groups=8, kept=4, normalize=True),
        # the gradient of a softmax router of the same batch
        dict(name="router_grad", op="router", form="grad", ranks=8, tokens=4096, experts=256, topk=8, score="softmax",
             dtype="fp32", biased=False, groups=1, kept=1, normalize=True),
        # a decode step: latency
        dict(name="router_decode", op="router", form="forward", ranks=8, tokens=4, experts=32, topk=4, score="softmax",
             dtype="bf16", biased=False, groups=1, kept=1, normalize=False),
        # training, the experts' up projection with its gated activation and routing weights, kept for the backward pass
        dict(name="product_gated_train", op="product", form="forward", ranks=8, tokens=2048, topk=8, experts=64, n=4096,
             k=7168, act="silu", gated=True, biased=False, weighted=True, residual=False, keep=True, out="bf16"),
        # a dense shared expert's down projection of an odd batch, bias and residual stream added
        dict(name="product_dense_residual", op="product", form="forward", ranks=1, tokens=8187, topk=1, experts=1, n=7168,
             k=2048, act="none", gated=False, biased=True, weighted=False, residual=True, keep=False, out="bf16"),
        # the router's logits: few columns, kept in fp32
        dict(name="product_logits", op="product", form="forward", ranks=1, tokens=4096, topk=1, experts=1, n=256, k=7168,
             act="none", gated=False, biased=False, weighted=False, residual=False, keep=False, out="fp32"),
        # a decode step of bf16 experts with biases
        dict(name="product_decode", op="product", form="forward", ranks=8, tokens=4, topk=4, experts=32, n=1024, k=1024,
             act="gelu", gated=True, biased=True, weighted=False, residual=False, keep=False, out="bf16"),
        # training, the epilogue's gradient: gate and up, the biases, the routing weights
        dict(name="product_gated_grad", op="product", form="grad", ranks=8, tokens=1021, topk=4, experts=32, n=2048, k=8,
             act="silu", gated=True, biased=True, weighted=True, residual=False, keep=True, out="bf16"),
        # one token through a layer of FP8 experts: the weights of 8 experts
        dict(name="layer_one_token", op="layer", weights="fp8", ranks=1, tokens=1, experts=64, topk=8, hidden=7168, width=2048,
             shared=False, masked=False),
        # a decode step of a small bf16 layer (8 ranks x 2 tokens), a shared expert's output added
        dict(name="layer_small", op="layer", weights="bf16", ranks=8, tokens=2, experts=32, topk=4, hidden=1024, width=512,
             shared=True, masked=False),
        # a few tokens, sizes that are no multiple of anything, some slots without an expert
        dict(name="layer_odd", op="layer", weights="bf16", ranks=1, tokens=5, experts=40, topk=6, hidden=2056, width=1000,
             shared=False, masked=True),
        # the most tokens: every expert of an FP8 layer is read
        dict(name="layer_most_tokens", op="layer", weights="fp8", ranks=8, tokens=8, experts=64, topk=8, hidden=7168,
             width=2048, shared=True, masked=False),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["router", "product", "product", "layer", "layer"])
    ranks = rng.choice([1, 2, 4, 8, 16])
    if op == "router":
        experts = ranks * rng.choice([1, 3, 8, 16, 20])
        groups = rng.choice([1, 1, 2, 4]) if experts % 4 == 0 and experts >= 16 else 1
        return dict(op=op, form=rng.choice(["forward", "grad"]), ranks=ranks, tokens=_log_int(rng, 1, 32768 // ranks),
                    experts=experts, topk=min(experts // groups, rng.choice([1, 2, 4, 6, 8])),
                    score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["fp32", "bf16"]), biased=rng.random() < 0.5,
                    groups=groups, kept=max(1, groups // 2), normalize=rng.random() < 0.5)
    if op == "product":
        form = rng.choice(["forward", "forward", "grad"])
        dense = rng.random() < 0.4
        ranks = 1 if dense else ranks
        experts = 1 if dense else ranks * rng.choice([1, 2, 4, 5, 8])
        topk = min(experts, rng.choice([1, 2, 4, 6, 8]))
        tokens = _log_int(rng, 1, 16384 // ranks)
        gated = rng.random() < 0.5
        n, k = _log_int(rng, 64, 4096, 16), _log_int(rng, 64, 7168, 8)
        limit = 2.0 * 8 * 2048 * 8 * 4096 * 7168
        while 2.0 * ranks * tokens * topk * n * k > limit or experts * n * k > 64 * 4096 * 7168:
            n, tokens = max(64, n // 32 * 16), max(1, tokens // 2)
        out = "bf16" if gated or form == "grad" else rng.choice(["bf16", "bf16", "fp32"])
        return dict(op=op, form=form, ranks=ranks, tokens=tokens, topk=topk, experts=experts, n=n, k=k,
                    act=rng.choice(["silu", "gelu", "relu"] if gated else ["none", "silu", "gelu", "relu"]), gated=gated,
                    biased=rng.random() < 0.5, weighted=rng.random() < 0.5, residual=rng.random() < 0.5 and form == "forward",
                    keep=form == "grad" or rng.random() < 0.5, out=out)
    ranks = rng.choice([1, 2, 4, 8])
    experts = ranks * rng.choice([1, 3, 8])
    fp8 = rng.random() < 0.5
    step = GROUP if fp8 else 8
    return dict(op=op, weights="fp8" if fp8 else "bf16", ranks=ranks, tokens=_log_int(rng, 1, 64 // ranks), experts=experts,
                topk=min(experts, rng.choice([1, 2, 4, 6, 8])), hidden=_log_int(rng, 256, 7168, step),
                width=_log_int(rng, 128, 2048, step), shared=rng.random() < 0.5, masked=rng.random() < 0.3)


# ------------------------------------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 6271 + 271)
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    """N(0, std^2), drawn in pieces so that the 32-bit draws stay small."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * std)
    return out


def _codes(g, shape):
    """e4m3 weights as a cast leaves them: a bell curve that reaches the format's largest values."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_((torch.randn(part.shape, generator=g, device=DEV) * 128).clamp_(-448, 448))
    return out


def _choices(g, case):
    """Distinct top-k experts of every token, [ranks * tokens][topk], some experts more popular than others."""
    n, E = case["ranks"] * case["tokens"], case["experts"]
    liked = torch.randn(E, generator=g, device=DEV) * 0.3
    noise = -torch.log(-torch.log(torch.rand((n, E), generator=g, device=DEV).clamp_(1e-9, 1 - 1e-7)))
    return torch.topk(liked + noise, case["topk"], dim=1).indices


def _handle(case, hidden):
    """The handle that a program keeps; the plain form has none."""
    if not own:
        return None
    from combine_get_dispatch_03_gb300 import ep
    return ep.Handle(ep.Config(num_ranks=case["ranks"], num_max_tokens=case["tokens"], hidden=hidden,
                               num_experts=case["experts"], num_topk=case["topk"]))


def prepare(case, seed):
    g = _generator(seed)
    return dict(_PREPARE[case["op"]](case, g), case=case)


def _prepare_router(case, g):
    R, T, E, K = case["ranks"], case["tokens"], case["experts"], case["topk"]
    dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    s = dict(logits=(torch.randn((R, T, E), generator=g, device=DEV) * 1.5 + torch.randn(E, generator=g, device=DEV) * 0.3).to(dtype))
    s["bias"] = torch.randn(E, generator=g, device=DEV) * 0.02 if case["biased"] else None
    if case["form"] == "grad":  # the forward pass's choice is in hand
        s["topk_idx"] = _plain_route(s, case)[0]
        s["dweights"] = torch.randn((R, T, K), generator=g, device=DEV)
    s["handle"] = _handle(case, 128)
    return s


def _prepare_product(case, g):
    E, n, k = case["experts"], case["n"], case["k"]
    idx = _choices(g, case)
    count = torch.bincount(idx.view(-1), minlength=E).to(torch.int32)
    rows, width = idx.numel(), n // 2 if case["gated"] else n
    s = dict(count=count, begin=(torch.cumsum(count, 0) - count).to(torch.int32), rows=rows, most=int(count.max()), width=width)
    s["weights"] = torch.rand(rows, generator=g, device=DEV) if case["weighted"] else None
    if case["form"] == "forward":
        s["x"], s["w"] = _normal(g, (rows, k)), _normal(g, (E, n, k), k ** -0.5)
        s["bias"] = torch.randn((E, n), generator=g, device=DEV) * 0.1 if case["biased"] else None
        s["residual"] = _normal(g, (rows, width)) if case["residual"] else None
    else:
        s["pre"], s["dy"] = _normal(g, (rows, n)), _normal(g, (rows, width))
    s["handle"] = _handle(case, 8)
    return s


def _prepare_layer(case, g):
    R, T, E, K, H, I = (case[v] for v in ("ranks", "tokens", "experts", "topk", "hidden", "width"))
    idx = _choices(g, case).view(R, T, K).contiguous()
    if case["masked"]:
        idx = torch.where(torch.rand((R, T, K), generator=g, device=DEV) < 0.1, -1, idx)
    s = dict(x=_normal(g, (R, T, H)), topk_idx=idx)
    s["topk_weights"] = torch.softmax(torch.randn((R, T, K), generator=g, device=DEV), -1)
    s["shared"] = _normal(g, (R, T, H)) if case["shared"] else None
    if case["weights"] == "fp8":
        s["w_up"], s["w_down"] = _codes(g, (E, 2 * I, H)), _codes(g, (E, H, I))
        # codes of about 128 times these scales are weights of about H^-0.5 and I^-0.5
        s["up_scales"] = (torch.rand((E, 2 * I // GROUP, H // GROUP), generator=g, device=DEV) + 0.5) / 128 * H ** -0.5
        s["down_scales"] = (torch.rand((E, H // GROUP, I // GROUP), generator=g, device=DEV) + 0.5) / 128 * I ** -0.5
    else:
        s["w_up"], s["w_down"] = _normal(g, (E, 2 * I, H), H ** -0.5), _normal(g, (E, H, I), I ** -0.5)
        s["up_scales"] = s["down_scales"] = None
    s["handle"] = _handle(case, H)
    return s


_PREPARE = dict(router=_prepare_router, product=_prepare_product, layer=_prepare_layer)


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _own_router(s):
    from combine_get_dispatch_03_gb300 import ep
    case, h = s["case"], s["handle"]
    if case["form"] == "grad":
        return ep.ep_router_grad(h, s["logits"], s["topk_idx"], s["dweights"], score=case["score"],
                                 normalize=case["normalize"], scale=2.5)
    return ep.ep_router(h, s["logits"], bias=s["bias"], score=case["score"], num_groups=case["groups"],
                        kept_groups=case["kept"], normalize=case["normalize"], scale=2.5)


def _own_product(s):
    from combine_get_dispatch_03_gb300 import ep
    case, h = s["case"], s["handle"]
    if case["form"] == "grad":
        return ep.ep_act_grad(h, s["dy"], s["pre"], s["count"], s["begin"], act=case["act"], gated=case["gated"],
                              row_weights=s["weights"], with_bias=case["biased"])
    return ep.ep_grouped_gemm_act(h, s["x"], s["w"], s["count"], s["begin"], bias=s["bias"], act=case["act"],
                                  gated=case["gated"], row_weights=s["weights"], residual=s["residual"],
                                  keep_pre=case["keep"], out_dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16)


def _own_layer(s):
    from combine_get_dispatch_03_gb300 import ep
    return ep.ep_moe_layer(s["handle"], s["x"], s["topk_idx"], s["topk_weights"], s["w_up"], s["w_down"],
                           up_scales=s["up_scales"], down_scales=s["down_scales"], bias_0=s["shared"])


_OWN = dict(router=_own_router, product=_own_product, layer=_own_layer)


def _plain_route(s, case):
    """(chosen experts, their scores in 64 bits)."""
    l = s["logits"].double()
    score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.exp(l - l.amax(-1, keepdim=True))
    if case["score"] == "softmax":
        score = score / score.sum(-1, keepdim=True)
    key = score if s["bias"] is None else score + s["bias"].double()
    G = case["groups"]
    if G > 1:
        parts = key.view(*key.shape[:2], G, -1)
        group = torch.sort(parts, dim=-1, descending=True).values[..., :2].sum(-1)
        best = torch.sort(group, dim=-1, descending=True, stable=True).indices[..., :case["kept"]]
        keep = torch.zeros_like(group, dtype=torch.bool).scatter_(-1, best, True)
        key = torch.where(keep[..., None], parts, -math.inf).view(key.shape)
    elif s["bias"] is None:
        key = l  # the order of the scores, without their rounding
    idx = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :case["topk"]].contiguous()
    return idx, torch.gather(score, -1, idx)


def _plain_router(s):
    case = s["case"]
    if case["form"] == "forward":
        idx, w = _plain_route(s, case)
        w = w.float()
        if case["normalize"]:
            w = w / w.sum(-1, keepdim=True)
        return dict(topk_idx=idx, topk_weights=w * 2.5)
    l, idx, dw = s["logits"].float(), s["topk_idx"], s["dweights"] * 2.5
    score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.exp(l - l.amax(-1, keepdim=True))
    if case["score"] == "softmax":
        score = score / score.sum(-1, keepdim=True)
    if case["normalize"]:
        chosen = torch.gather(score, -1, idx)
        total = chosen.sum(-1, keepdim=True)
        dw = (dw - (dw * chosen).sum(-1, keepdim=True) / total) / total
    ds = torch.zeros_like(l).scatter_(-1, idx, dw)
    if case["score"] == "sigmoid":
        dl = ds * score * (1 - score)
    else:
        dl = score * (ds - (ds * score).sum(-1, keepdim=True))
    return dl.to(s["logits"].dtype)


def _act(v, act):
    """(activation, its derivative)."""
    if act == "none":
        return v, torch.ones_like(v)
    if act == "relu":
        return v * (v > 0), (v > 0).to(v.dtype)
    if act == "silu":
        sig = 1 / (1 + torch.exp(-v))
        return v * sig, sig * (1 + v * (1 - sig))
    phi = 0.5 * torch.erfc(v * -(0.5 ** 0.5))
    return v * phi, phi + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))


def _row_group(s, E):
    """The expert of every row (packed groups)."""
    return torch.repeat_interleave(torch.arange(E, device=DEV), s["count"].long(), output_size=s["rows"])


def _plain_product(s):
    case = s["case"]
    weight = s["weights"][:, None] if s["weights"] is not None else 1.0
    if case["form"] == "grad":
        dy, v = s["dy"].float(), s["pre"].float()
        if case["gated"]:
            gate, up = v.chunk(2, 1)
            a, slope = _act(gate, case["act"])
            d = torch.cat([dy * weight * up * slope, dy * weight * a], 1)
            value = a * up
        else:
            value, slope = _act(v, case["act"])
            d = dy * weight * slope
        out = dict(d_pre=d.to(torch.bfloat16))
        out["d_row_weights"] = (dy * value).sum(1) if s["weights"] is not None else None
        out["d_bias"] = None
        if case["biased"]:
            at = torch.arange(s["most"], device=DEV)
            valid = at < s["count"][:, None]
            index = torch.where(valid, s["begin"][:, None] + at, 0)
            out["d_bias"] = torch.stack([(d[index[e]] * valid[e, :, None]).sum(0) for e in range(case["experts"])])
        return out
    at = torch.arange(s["most"], device=DEV)
    valid = at < s["count"][:, None]
    index = torch.where(valid, s["begin"][:, None] + at, 0)
    y = torch.bmm(s["x"].float()[index], s["w"].float().transpose(1, 2))
    if s["bias"] is not None:
        y += s["bias"][:, None]
    v = torch.empty((s["rows"], case["n"]), device=DEV)
    v[index[valid]] = y[valid]
    del y
    if case["gated"]:
        gate, up = v.chunk(2, 1)
        out = _act(gate, case["act"])[0] * up
    else:
        out = _act(v, case["act"])[0]
    out = out * weight
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return dict(out=out.to(torch.float32 if case["out"] == "fp32" else torch.bfloat16),
                pre=v.to(torch.bfloat16) if case["keep"] else None)


def _weights(w, scales):
    """Weights [...][n][k] in 32 bits."""
    if scales is None:
        return w.float()
    n, k = w.shape[-2:]
    return w.float() * scales.repeat_interleave(GROUP, -2)[..., :n, :].repeat_interleave(GROUP, -1)[..., :k]


def _plain_layer(s):
    case = s["case"]
    H, K, E, I = case["hidden"], case["topk"], case["experts"], case["width"]
    x, idx, w = s["x"].view(-1, H).float(), s["topk_idx"].view(-1, K), s["topk_weights"].view(-1, K)
    w = torch.where(idx >= 0, w, 0.0)
    y = torch.zeros_like(x)

    def expert(rows, up, up_scales, down, down_scales):
        gate, u = (rows @ _weights(up, up_scales).t()).split(I, 1)
        return (gate / (1 + torch.exp(-gate)) * u) @ _weights(down, down_scales).t()

    if idx.numel() < E:  # the chosen experts one by one
        for t in range(idx.shape[0]):
            for k in range(K):
                e = idx[t, k:k + 1].clamp_min(0)
                pick = [None if v is None else v.index_select(0, e)[0]
                        for v in (s["w_up"], s["up_scales"], s["w_down"], s["down_scales"])]
                y[t:t + 1] += w[t, k] * expert(x[t:t + 1], *pick)
    else:
        per_expert = torch.zeros((idx.shape[0], E), device=DEV).scatter_add_(1, idx.clamp_min(0), w)
        for e in range(E):
            pick = [None if v is None else v[e] for v in (s["w_up"], s["up_scales"], s["w_down"], s["down_scales"])]
            y += per_expert[:, e:e + 1] * expert(x, *pick)
    if s["shared"] is not None:
        y += s["shared"].view(-1, H).float()
    return y.to(torch.bfloat16).view(s["x"].shape)


_PLAIN = dict(router=_plain_router, product=_plain_product, layer=_plain_layer)


# ------------------------------------------------------------------------------------------------ work and truth

def work(case):
    tokens, E, K = case["ranks"] * case["tokens"], case["experts"], case["topk"]
    if case["op"] == "router":
        logits = tokens * E * (4 if case["dtype"] == "fp32" else 2)
        if case["form"] == "grad":
            return dict(bytes=2 * logits + tokens * K * 12, flops=12.0 * tokens * E)
        return dict(bytes=logits + tokens * K * 12, flops=6.0 * tokens * E)
    used = E * (1 - (1 - K / E) ** tokens)  # experts that get a row, about
    if case["op"] == "product":
        rows, n, k = tokens * K, case["n"], case["k"]
        width = n // 2 if case["gated"] else n
        meta = rows * 4 * case["weighted"] + E * n * 4 * case["biased"]
        if case["form"] == "grad":
            return dict(bytes=rows * (4 * n + 2 * width) + 2 * meta, flops=12.0 * rows * n)
        out = width * (4 if case["out"] == "fp32" else 2) + 2 * width * case["residual"] + 2 * n * case["keep"]
        return dict(bytes=rows * (2 * k + out) + used * n * k * 2 + meta, flops=2.0 * rows * n * k)
    H, I = case["hidden"], case["width"]
    each = 3 * H * I * (1 + 4 / GROUP / GROUP if case["weights"] == "fp8" else 2)
    return dict(bytes=used * each + tokens * H * (4 + 2 * case["shared"]) + tokens * K * 12, flops=6.0 * tokens * K * H * I)


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_router(case, s):
    E = case["experts"]
    l = s["logits"].double().view(-1, E)
    if case["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-l))
    else:
        p = torch.softmax(l, 1)
    K = case["topk"]
    idx = s["topk_idx"] if case["form"] == "grad" else _plain_route(s, case)[0]  # whole numbers, compared as such
    idx = idx.view(-1, K)
    c = p.gather(1, idx)
    if case["form"] == "forward":
        w = 2.5 * (c / c.sum(1, keepdim=True) if case["normalize"] else c)
        return dict(topk_idx=None, topk_weights=w.view(*s["logits"].shape[:2], K))
    g = s["dweights"].double().view(-1, K)
    if case["normalize"]:  # w_j = 2.5 c_j / S: dw_j/dc_i = 2.5 (delta_ij S - c_j) / S^2
        S = c.sum(1, keepdim=True)
        dc = 2.5 * (g * S - (g * c).sum(1, keepdim=True)) / (S * S)
    else:
        dc = 2.5 * g
    if case["score"] == "sigmoid":
        dl = torch.zeros_like(l).scatter_(1, idx, dc * c * (1 - c))
    else:  # dp_j/dl_i = p_j (delta_ij - p_i)
        dl = torch.zeros_like(l).scatter_(1, idx, dc * c) - p * (dc * c).sum(1, keepdim=True)
    return dl.view(s["logits"].shape)


def _exact_act(v, act):
    if act == "none":
        return v, torch.ones_like(v)
    if act == "relu":
        return torch.clamp(v, min=0), torch.where(v > 0, 1.0, 0.0).double()
    if act == "silu":
        return v / (1 + torch.exp(-v)), (1 + torch.exp(-v) * (1 + v)) / (1 + torch.exp(-v)) ** 2
    cdf = (1 + torch.erf(v / math.sqrt(2))) / 2
    return v * cdf, cdf + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)


def _exact_product(case, s):
    n, width = case["n"], s["width"]
    keep = case["form"] == "forward" and case["keep"]
    out = torch.zeros((s["rows"], n if case["form"] == "grad" else width), dtype=torch.float64, device=DEV)
    pre = torch.zeros((s["rows"], n), dtype=torch.float64, device=DEV) if keep else None
    d_bias = torch.zeros((case["experts"], n), dtype=torch.float64, device=DEV)
    d_weights = torch.zeros(s["rows"], dtype=torch.float64, device=DEV)
    at = 0
    for e, m in enumerate(s["count"].tolist()):
        rows = slice(at, at + m)
        at += m
        weight = s["weights"][rows].double()[:, None] if s["weights"] is not None else 1.0
        if case["form"] == "grad":
            v, dy = s["pre"][rows].double(), s["dy"][rows].double()
            a, slope = _exact_act(v[:, :width], case["act"])
            up = v[:, width:] if case["gated"] else 1.0
            out[rows, :width] = dy * weight * up * slope
            if case["gated"]:
                out[rows, width:] = dy * weight * a
            d_weights[rows] = (dy * a * up).sum(1)
            d_bias[e] = out[rows].sum(0)
            continue
        v = s["x"][rows].double() @ s["w"][e].double().t()
        if s["bias"] is not None:
            v = v + s["bias"][e].double()
        if keep:
            pre[rows] = v
        a = _exact_act(v[:, :width], case["act"])[0] * weight
        out[rows] = a * v[:, width:] if case["gated"] else a
        if s["residual"] is not None:
            out[rows] += s["residual"][rows].double()
    if case["form"] == "grad":
        return dict(d_pre=out, d_row_weights=d_weights if case["weighted"] else None, d_bias=d_bias if case["biased"] else None)
    return dict(out=out, pre=pre)


def _exact_layer(case, s):
    H, K, I = case["hidden"], case["topk"], case["width"]
    x, idx = s["x"].view(-1, H).double(), s["topk_idx"].view(-1, K)
    y = s["shared"].view(-1, H).double() if s["shared"] is not None else torch.zeros_like(x)

    def dense(w, scales, e):
        w = w[e].double()
        if scales is not None:
            n, k = w.shape
            w = (w.view(n // GROUP, GROUP, k // GROUP, GROUP) * scales[e].double()[:, None, :, None]).view(n, k)
        return w

    for e in sorted(set(idx.flatten().tolist()) - {-1}):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        v = x[t] @ dense(s["w_up"], s["up_scales"], e).t()
        a = v[:, :I] / (1 + torch.exp(-v[:, :I])) * v[:, I:]
        y.index_add_(0, t, s["topk_weights"].view(-1, K)[t, k].double()[:, None] * (a @ dense(s["w_down"], s["down_scales"], e).t()))
    return y.view(s["x"].shape)


_EXACT = dict(router=_exact_router, product=_exact_product, layer=_exact_layer)
