"""The expert operators: what the experts of a mixture-of-experts layer compute between a dispatch and a combine.

Four operators, each in a plain form (elementary torch operations in 32 bits, rounded once at the end) and as
this package's calls:

  product      rows grouped by expert times that expert's bf16 weights: forward, gradient of the rows, gradient
               of the weights (ep_grouped_gemm, ep_grouped_gemm_wgrad)
  product_fp8  the same product on e4m3 rows with one scale per 128 channels and e4m3 weights with one scale per
               128 x 128 block, from packed rows or in place from low-latency messages (ep_grouped_gemm_fp8)
  swiglu       the gated activation between an expert's two products, optionally cast to e4m3 with scales, and
               its gradient (ep_swiglu, ep_swiglu_grad)
  expert_rows  a normal dispatch's rows brought into expert order, and the sum back (ep_expert_layout,
               ep_expert_gather, ep_expert_reduce)

Set `own` to True to make `run` call the package.  Rows of expert e are [begin[e], begin[e] + count[e]).
"""
import math

import torch

own = False

GROUP = 128      # channels that share one FP8 scale
E4M3_MAX = 448.0
HEADER = 16      # bytes before the payload of a low-latency message
DEV = "cuda"


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # training, forward: the up projection of a large batch (8 ranks x 2048 tokens, top-8, hidden 7168)
        dict(name="product_train", op="product", form="forward", ranks=8, tokens=2048, topk=8, experts=64, n=4096, k=7168),
        # a decode step of bf16 experts: a row or two per expert, so the weights are all there is to read
        dict(name="product_decode", op="product", form="forward", ranks=8, tokens=2, topk=4, experts=32, n=2048, k=1024),
        # training, gradient of the rows of a ragged mid-sized batch
        dict(name="product_input_grad", op="product", form="input_grad", ranks=8, tokens=509, topk=4, experts=32, n=2048, k=4104),
        # training, gradient of the weights, kept in fp32 as a master gradient
        dict(name="product_weight_grad", op="product", form="weight_grad", ranks=8, tokens=1024, topk=8, experts=32, n=2048, k=7168),
        # prefill in FP8: packed rows of a normal dispatch, fp32 scales
        dict(name="fp8_prefill", op="product_fp8", layout="rows", scales="fp32", ranks=8, tokens=2048, topk=8, experts=64, n=4096, k=7168),
        # low-latency decode: message buffers of 8 ranks x 128 tokens read in place, UE8M0 scales
        dict(name="fp8_messages", op="product_fp8", layout="messages", scales="ue8m0", ranks=8, tokens=128, topk=8, experts=64, n=4096, k=7168),
        # one token through one dense FP8 layer (a single group), odd output width
        dict(name="fp8_one_token", op="product_fp8", layout="rows", scales="fp32", ranks=1, tokens=1, topk=1, experts=1, n=1000, k=2048),
        # between the two FP8 products of a prefill: activation, routing weight, cast to e4m3
        dict(name="swiglu_cast", op="swiglu", form="cast", weighted=True, ranks=8, tokens=2048, topk=8, experts=64, width=2048),
        # the activation's gradient in training, with the routing weights' gradient
        dict(name="swiglu_grad", op="swiglu", form="grad", weighted=True, ranks=8, tokens=1021, topk=4, experts=32, width=1024),
        # a decode step's activation: latency
        dict(name="swiglu_decode", op="swiglu", form="forward", weighted=False, ranks=8, tokens=4, topk=4, experts=32, width=1024),
        # received rows of a normal dispatch into expert order, with their routing weights
        dict(name="rows_gather", op="expert_rows", form="gather", fp8=False, ranks=8, tokens=2048, topk=8, experts=64, hidden=7168),
        # expert outputs summed back into receive rows, a ragged mid-sized batch
        dict(name="rows_reduce", op="expert_rows", form="reduce", fp8=False, ranks=8, tokens=509, topk=4, experts=32, hidden=2048),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["product", "product", "product_fp8", "product_fp8", "swiglu", "expert_rows"])
    ranks = rng.choice([1, 2, 4, 8, 16])
    experts = ranks * rng.choice([1, 2, 4, 5, 8])
    topk = min(experts, rng.choice([1, 2, 4, 6, 8]))
    tokens = _log_int(rng, 1, 2048 * 8 // ranks)
    case = dict(op=op, ranks=ranks, tokens=tokens, topk=topk, experts=experts)
    if op in ("product", "product_fp8"):
        if op == "product":
            case["form"] = rng.choice(["forward", "input_grad", "weight_grad"])
            k = _log_int(rng, 128, 7168, 8)
        else:
            case["layout"] = rng.choice(["rows", "messages"])
            case["scales"] = rng.choice(["fp32", "ue8m0"])
            k = _log_int(rng, 512, 7168, 512) if case["layout"] == "messages" else _log_int(rng, 128, 7168, 128)
            if case["layout"] == "messages":  # a low-latency buffer holds ranks * tokens rows for every expert
                case["tokens"] = min(tokens, 1024 // ranks)
        n = _log_int(rng, 64, 4096, 8)
        limit = 2.0 * 8 * 2048 * 8 * 4096 * 7168
        while 2.0 * ranks * case["tokens"] * topk * n * k > limit or experts * n * k > 64 * 4096 * 7168:
            n, case["tokens"] = max(64, n // 16 * 8), max(1, case["tokens"] // 2)
        return dict(case, n=_not_3072(n), k=_not_3072(k))
    if op == "swiglu":
        return dict(case, form=rng.choice(["cast", "forward", "grad"]), weighted=rng.random() < 0.5,
                    width=_not_3072(_log_int(rng, 128, 2048, 128)))
    fp8 = rng.random() < 0.5
    return dict(case, form="gather" if fp8 else rng.choice(["gather", "reduce"]), fp8=fp8,
                hidden=_not_3072(_log_int(rng, 128, 7168, 128 if fp8 else 8)))


def _not_3072(v):
    return 2944 if v == 3072 else v


# ------------------------------------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 12345)
    return g


def _normal(g, shape, std=1.0):
    """N(0, std^2) in bf16, drawn in pieces so that the 32-bit draws stay small."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * std)
    return out


def _codes(g, shape):
    """e4m3 payload as a cast leaves it: a bell curve that reaches the format's largest values."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_((torch.randn(part.shape, generator=g, device=DEV) * 128).clamp_(-E4M3_MAX, E4M3_MAX))
    return out


def _scales(g, shape, power_of_two):
    s = torch.rand(shape, generator=g, device=DEV) * 0.02 + 0.002
    return torch.exp2(torch.ceil(torch.log2(s))) if power_of_two else s


def _routing(g, case):
    """Distinct top-k experts of every token, [ranks * tokens][topk], some experts more popular than others."""
    n, E = case["ranks"] * case["tokens"], case["experts"]
    liked = torch.randn(E, generator=g, device=DEV) * 0.3
    noise = -torch.log(-torch.log(torch.rand((n, E), generator=g, device=DEV).clamp_(1e-9, 1 - 1e-7)))
    return torch.topk(liked + noise, case["topk"], dim=1).indices


def _groups(g, case):
    """Packed groups: per expert its rows' count and begin (device), the total and the longest (host)."""
    idx = _routing(g, case)
    count = torch.bincount(idx.view(-1), minlength=case["experts"]).to(torch.int32)
    begin = (torch.cumsum(count, 0) - count).to(torch.int32)
    return dict(count=count, begin=begin, rows=idx.numel(), most=int(count.max()))


def _handle(case, hidden, capacity):
    """The handle that a program keeps; the plain form has none."""
    if not own:
        return None
    from combine_get_dispatch_03_gb300 import ep
    return ep.Handle(ep.Config(num_ranks=case["ranks"], num_max_tokens=case["tokens"], hidden=hidden,
                               num_experts=case["experts"], num_topk=case["topk"], recv_capacity=capacity))


def prepare(case, seed):
    g = _generator(seed)
    return dict(_PREPARE[case["op"]](case, g), case=case)


def _prepare_product(case, g):
    s = _groups(g, case)
    E, n, k, form = case["experts"], case["n"], case["k"], case["form"]
    if form != "input_grad":
        s["x"] = _normal(g, (s["rows"], k))
    if form != "forward":
        s["dy"] = _normal(g, (s["rows"], n))
    if form != "weight_grad":
        s["w"] = _normal(g, (E, n, k), 0.02)
    s["handle"] = _handle(case, k, 0)
    return s


def _prepare_product_fp8(case, g):
    E, n, k = case["experts"], case["n"], case["k"]
    ue8m0 = case["scales"] == "ue8m0"
    s = _groups(g, case)
    if case["layout"] == "messages":
        # [ranks][experts per rank][ranks * tokens] messages: header, payload, scales
        R, EL, rows, G = case["ranks"], E // case["ranks"], case["ranks"] * case["tokens"], k // GROUP
        msgs = torch.zeros((R, EL, rows, HEADER + k + 4 * G), dtype=torch.uint8, device=DEV)
        msgs[..., HEADER:HEADER + k] = _codes(g, (R, EL, rows, k)).view(torch.uint8)
        scales = _scales(g, (R, EL, rows, G), ue8m0)
        if ue8m0:
            msgs[..., HEADER + k:HEADER + k + G] = (torch.log2(scales) + 127).to(torch.uint8)
        else:
            msgs[..., HEADER + k:] = scales.view(torch.uint8)
        s.update(msgs=msgs, out=torch.zeros((R, EL, rows, n), dtype=torch.bfloat16, device=DEV), begin=None)
    else:
        s.update(x=_codes(g, (s["rows"], k)), x_scales=_scales(g, (s["rows"], k // GROUP), ue8m0))
    s["w"] = _codes(g, (E, n, k))
    s["w_scales"] = _scales(g, (E, -(-n // GROUP), k // GROUP), ue8m0) * 0.01
    s["handle"] = _handle(case, k, 0)
    return s


def _prepare_swiglu(case, g):
    s = _groups(g, case)
    s["x"] = _normal(g, (s["rows"], 2 * case["width"]))
    s["dy"] = _normal(g, (s["rows"], case["width"])) if case["form"] == "grad" else None
    s["weights"] = torch.rand(s["rows"], generator=g, device=DEV) if case["weighted"] else None
    s["handle"] = _handle(case, 2 * case["width"], 0)
    return s


def _prepare_expert_rows(case, g):
    R, T, K, E, H = case["ranks"], case["tokens"], case["topk"], case["experts"], case["hidden"]
    idx, EL = _routing(g, case), E // R
    local = [torch.where(idx // EL == r, idx % EL, -1) for r in range(R)]
    here = [torch.nonzero((v >= 0).any(1)).view(-1) for v in local]
    num_recv = torch.tensor([v.numel() for v in here], dtype=torch.int32, device=DEV)
    cap = R * T  # the worst case, as a program without a look at the counts allocates it
    recv_topk_idx = torch.full((R, cap, K), -1, dtype=torch.int64, device=DEV)
    for r in range(R):
        recv_topk_idx[r, :here[r].numel()] = local[r][here[r]]
    s = dict(recv_topk_idx=recv_topk_idx, num_recv=num_recv, rows=R * T * K, cap=cap)
    if case["form"] == "gather":
        s["weights"] = torch.rand((R, cap, K), generator=g, device=DEV)
        s["x"] = _codes(g, (R, cap, H)) if case["fp8"] else _normal(g, (R, cap, H))
        s["x_scales"] = _scales(g, (R, cap, H // GROUP), False) if case["fp8"] else None
    else:
        # the layout of the forward pass is in hand; the sum writes the received rows, the rest stay as they are
        s["layout"] = _plain_layout(case, recv_topk_idx)
        s["y"] = _normal(g, (s["rows"], H))
        s["dweights"] = torch.randn(s["rows"], generator=g, device=DEV)
        s["out"] = torch.zeros((R, cap, H), dtype=torch.bfloat16, device=DEV)
        s["out_weights"] = torch.zeros((R, cap, K), device=DEV)
    s["handle"] = _handle(case, H, cap)
    return s


_PREPARE = dict(product=_prepare_product, product_fp8=_prepare_product_fp8, swiglu=_prepare_swiglu,
                expert_rows=_prepare_expert_rows)


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _own_product(s):
    from combine_get_dispatch_03_gb300 import ep
    form = s["case"]["form"]
    if form == "forward":
        return ep.ep_grouped_gemm(s["handle"], s["x"], s["w"], s["count"], s["begin"])
    if form == "input_grad":
        return ep.ep_grouped_gemm(s["handle"], s["dy"], s["w"], s["count"], s["begin"], w_transposed=True)
    return ep.ep_grouped_gemm_wgrad(s["handle"], s["dy"], s["x"], s["count"], s["begin"])


def _own_product_fp8(s):
    from combine_get_dispatch_03_gb300 import ep
    case, h = s["case"], s["handle"]
    if case["layout"] == "rows":
        return ep.ep_grouped_gemm_fp8(h, s["x"], s["x_scales"], s["w"], s["w_scales"], s["count"], s["begin"])
    x, scales, _ = ep.ll_views(s["msgs"], case["k"], True)
    if case["scales"] == "fp32":
        scales = scales.view(torch.float32)
    expected = case["ranks"] * case["tokens"] * case["topk"] // case["experts"]
    return ep.ep_grouped_gemm_fp8(h, x, scales, s["w"], s["w_scales"], s["count"], out=s["out"], expected_rows=expected)


def _own_swiglu(s):
    from combine_get_dispatch_03_gb300 import ep
    form, h = s["case"]["form"], s["handle"]
    if form == "grad":
        return ep.ep_swiglu_grad(h, s["dy"], s["x"], s["count"], s["begin"], row_weights=s["weights"])
    return ep.ep_swiglu(h, s["x"], s["count"], s["begin"], row_weights=s["weights"], cast_to_fp8=form == "cast")


def _own_expert_rows(s):
    from combine_get_dispatch_03_gb300 import ep
    h = s["handle"]
    if s["case"]["form"] == "reduce":
        return ep.ep_expert_reduce(h, s["y"], s["layout"]["slot_row"], num_recv=s["num_recv"],
                                   row_weights=s["dweights"], out=s["out"], out_topk_weights=s["out_weights"])
    lay = ep.ep_expert_layout(h, s["recv_topk_idx"], s["rows"], num_recv=s["num_recv"])
    out = ep.ep_expert_gather(h, s["x"], lay["slot_row"], s["rows"], num_recv=s["num_recv"], x_scales=s["x_scales"],
                              topk_weights=s["weights"])
    return dict(out, **lay)


_OWN = dict(product=_own_product, product_fp8=_own_product_fp8, swiglu=_own_swiglu, expert_rows=_own_expert_rows)


def _padded(s):
    """Row index [experts][most] of each group's rows, and which of them exist."""
    at = torch.arange(s["most"], device=DEV)
    valid = at < s["count"][:, None]
    return torch.where(valid, s["begin"][:, None] + at, 0), valid


def _plain_product(s):
    form = s["case"]["form"]
    index, valid = _padded(s)
    keep = valid[..., None]
    if form == "weight_grad":
        dy, x = s["dy"].float()[index] * keep, s["x"].float()[index] * keep
        return torch.bmm(dy.transpose(1, 2), x)
    rows = (s["x"] if form == "forward" else s["dy"]).float()
    w = s["w"].float()
    y = torch.bmm(rows[index], w.transpose(1, 2) if form == "forward" else w)
    out = torch.empty((s["rows"], y.shape[2]), dtype=torch.bfloat16, device=DEV)
    out[index[valid]] = y[valid].to(torch.bfloat16)
    return out


def _spread(scales, n, k):
    """One scale per 128 x 128 block -> one per element."""
    return scales.repeat_interleave(GROUP, -2)[..., :n, :].repeat_interleave(GROUP, -1)[..., :k]


def _message_parts(s):
    """Payload codes and 32-bit scales of a message buffer."""
    k = s["case"]["k"]
    codes = s["msgs"][..., HEADER:HEADER + k].contiguous().view(torch.float8_e4m3fn)
    tail = s["msgs"][..., HEADER + k:]
    if s["case"]["scales"] == "ue8m0":
        return codes, torch.exp2(tail[..., :k // GROUP].float() - 127)
    return codes, tail.contiguous().view(torch.float32)


def _plain_product_fp8(s):
    n, k, E = s["case"]["n"], s["case"]["k"], s["case"]["experts"]
    w = s["w"].float() * _spread(s["w_scales"], n, k)
    if s["case"]["layout"] == "rows":
        x = s["x"].float() * s["x_scales"].repeat_interleave(GROUP, -1)
        index, valid = _padded(s)
        y = torch.bmm(x[index], w.transpose(1, 2))
        out = torch.empty((s["rows"], n), dtype=torch.bfloat16, device=DEV)
        out[index[valid]] = y[valid].to(torch.bfloat16)
        return out
    codes, scales = _message_parts(s)
    most = max(s["most"], 1)
    x = codes.view(E, -1, k)[:, :most].float() * scales.view(E, -1, k // GROUP)[:, :most].repeat_interleave(GROUP, -1)
    valid = torch.arange(most, device=DEV) < s["count"][:, None]
    y = torch.bmm(x, w.transpose(1, 2)).to(torch.bfloat16)
    s["out"].view(E, -1, n)[:, :most][valid] = y[valid]
    return s["out"]


def _cast(v):
    """e4m3 codes and one scale per 128 channels."""
    groups = v.view(v.shape[0], -1, GROUP)
    amax = groups.abs().amax(-1, keepdim=True).clamp_min(1e-4)
    codes = (groups * (E4M3_MAX / amax)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(v.shape), (amax / E4M3_MAX).squeeze(-1)


def _plain_swiglu(s):
    form = s["case"]["form"]
    gate, up = s["x"].float().chunk(2, dim=1)
    sig = torch.sigmoid(gate)
    act = gate * sig
    weight = s["weights"][:, None] if s["weights"] is not None else 1.0
    if form == "grad":
        dy = s["dy"].float()
        dv = dy * weight
        dgate = dv * up * (sig * (1 + gate * (1 - sig)))
        out = dict(dx=torch.cat([dgate, dv * act], 1).to(torch.bfloat16))
        out["d_row_weights"] = (dy * act * up).sum(1) if s["weights"] is not None else None
        return out
    v = act * up * weight
    if form == "cast":
        codes, scales = _cast(v)
        return dict(out=codes, out_scales=scales)
    return dict(out=v.to(torch.bfloat16), out_scales=None)


def _plain_layout(case, recv_topk_idx):
    """Expert order: rank, local expert, receive row, top-k slot."""
    R, cap, K = recv_topk_idx.shape
    E, EL = case["experts"], case["experts"] // R
    rank = torch.arange(R, device=DEV)[:, None, None]
    expert = torch.where(recv_topk_idx >= 0, recv_topk_idx + rank * EL, E).view(-1)
    order = torch.sort(expert, stable=True)
    count = torch.bincount(expert, minlength=E + 1)[:E].to(torch.int32)
    rows = case["ranks"] * case["tokens"] * K
    slot_row = torch.full((R * cap * K,), -1, dtype=torch.int32, device=DEV)
    slot_row[order.indices[:rows]] = torch.arange(rows, dtype=torch.int32, device=DEV)
    return dict(group_count=count, group_begin=(torch.cumsum(count, 0) - count).to(torch.int32),
                slot_row=slot_row.view(R, cap, K))


def _plain_expert_rows(s):
    case = s["case"]
    if case["form"] == "gather":
        lay = _plain_layout(case, s["recv_topk_idx"])
        there = lay["slot_row"].view(-1)
        at = torch.nonzero(there >= 0).view(-1)
        slot = torch.empty(s["rows"], dtype=torch.int64, device=DEV)
        slot[there[at].long()] = at
        source = slot // case["topk"]
        flat = s["x"].view(-1, case["hidden"])
        out = flat.view(torch.uint8)[source].view(flat.dtype) if case["fp8"] else flat[source]
        scales = s["x_scales"].view(-1, case["hidden"] // GROUP)[source] if case["fp8"] else None
        return dict(lay, out=out, out_scales=scales, row_weights=s["weights"].view(-1)[slot])
    slot_row = s["layout"]["slot_row"]
    received = torch.arange(s["cap"], device=DEV) < s["num_recv"][:, None]
    at = slot_row[received].long()
    there = at >= 0
    at = at.clamp_min(0)
    s["out"][received] = (s["y"].float()[at] * there[..., None]).sum(1).to(torch.bfloat16)
    s["out_weights"][received] = torch.where(there, s["dweights"][at], 0.0)
    return dict(out=s["out"], out_topk_weights=s["out_weights"])


_PLAIN = dict(product=_plain_product, product_fp8=_plain_product_fp8, swiglu=_plain_swiglu,
              expert_rows=_plain_expert_rows)


# ------------------------------------------------------------------------------------------------ work and truth

def work(case):
    rows, E = case["ranks"] * case["tokens"] * case["topk"], case["experts"]
    tokens = case["ranks"] * case["tokens"]
    used = E * (1 - (1 - case["topk"] / E) ** tokens)  # experts that get a row, about
    if case["op"] == "product":
        n, k = case["n"], case["k"]
        weights = E * n * k * 4 if case["form"] == "weight_grad" else used * n * k * 2
        return dict(bytes=rows * (n + k) * 2 + weights, flops=2.0 * rows * n * k)
    if case["op"] == "product_fp8":
        n, k = case["n"], case["k"]
        per_scale = 1 if case["scales"] == "ue8m0" and case["layout"] == "messages" else 4
        return dict(bytes=rows * (k + k // GROUP * per_scale + 2 * n) + used * n * (k + k / GROUP / 32),
                    flops=2.0 * rows * n * k)
    if case["op"] == "swiglu":
        w = case["width"]
        out = {"forward": 2 * w, "cast": w + w // 32, "grad": 6 * w}[case["form"]]
        return dict(bytes=rows * (4 * w + out), flops=10.0 * rows * w)
    H, K, R = case["hidden"], case["topk"], case["ranks"]
    reached = tokens * R * (1 - (1 - 1 / R) ** K)  # receive rows, about
    row = H + H // 32 if case["fp8"] else 2 * H
    meta = reached * K * 8 + rows * 8
    return dict(bytes=(rows + reached) * row + meta, flops=float(rows * H))


def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, s)


def _each(s, case):
    """(expert, its first row, its rows) of every expert that has rows."""
    count = s["count"].tolist()
    at = 0
    for e in range(case["experts"]):
        if count[e]:
            yield e, at, count[e]
        at += count[e]


def _exact_product(case, s):
    form = case["form"]
    if form == "weight_grad":
        dw = torch.zeros((case["experts"], case["n"], case["k"]), dtype=torch.float64, device=DEV)
        for e, at, m in _each(s, case):
            dw[e] = s["dy"][at:at + m].double().t() @ s["x"][at:at + m].double()
        return dw
    rows = s["x"] if form == "forward" else s["dy"]
    out = torch.zeros((s["rows"], case["n"] if form == "forward" else case["k"]), dtype=torch.float64, device=DEV)
    for e, at, m in _each(s, case):
        w = s["w"][e].double()
        out[at:at + m] = rows[at:at + m].double() @ (w.t() if form == "forward" else w)
    return out


def _exact_product_fp8(case, s):
    n, k = case["n"], case["k"]
    messages = case["layout"] == "messages"
    if messages:
        EL, R = case["experts"] // case["ranks"], case["ranks"]
        out = torch.zeros((R, EL, s["msgs"].shape[2], n), dtype=torch.float64, device=DEV)
    else:
        out = torch.zeros((s["rows"], n), dtype=torch.float64, device=DEV)
    for e, at, m in _each(s, case):
        if messages:
            msg = s["msgs"][e // EL, e % EL, :m]
            x = msg[:, HEADER:HEADER + k].contiguous().view(torch.float8_e4m3fn).double()
            tail = msg[:, HEADER + k:].contiguous()
            scale = torch.pow(2.0, tail[:, :k // GROUP].double() - 127) if case["scales"] == "ue8m0" \
                else tail.view(torch.float32).double()
            to = out[e // EL, e % EL, :m]
        else:
            x, scale, to = s["x"][at:at + m].double(), s["x_scales"][at:at + m].double(), out[at:at + m]
        x = (x.view(m, -1, GROUP) * scale[:, :, None]).view(m, k)
        w = s["w"][e].double()
        for b in range(0, n, GROUP):
            block = w[b:b + GROUP]
            block.view(block.shape[0], -1, GROUP).mul_(s["w_scales"][e, b // GROUP].double()[None, :, None])
        to.copy_(x @ w.t())
    return out


def _exact_swiglu(case, s):
    x = s["x"].double()
    gate, up = x[:, :case["width"]], x[:, case["width"]:]
    weight = s["weights"].double()[:, None] if s["weights"] is not None else torch.ones((), device=DEV, dtype=torch.float64)
    sig = 1 / (1 + torch.exp(-gate))
    if case["form"] == "grad":
        dy = s["dy"].double()
        dgate = dy * weight * up * (sig + gate * sig * (1 - sig))
        dup = dy * weight * gate * sig
        dw = (dy * gate * sig * up).sum(1) if s["weights"] is not None else None
        return dict(dx=torch.cat([dgate, dup], 1), d_row_weights=dw)
    v = gate * sig * up * weight
    if case["form"] == "forward":
        return dict(out=v, out_scales=None)
    v = v.view(v.shape[0], -1, GROUP)
    amax = torch.clamp(v.abs().amax(2), min=1e-4)
    scale = amax / E4M3_MAX
    codes = (v / scale[:, :, None]).float().to(torch.float8_e4m3fn).double()
    return dict(out=codes.view(x.shape[0], -1), out_scales=scale)


def _exact_expert_rows(case, s):
    if case["form"] == "gather":
        return None  # whole numbers and copies
    y = torch.cat([s["y"].double(), torch.zeros((1, case["hidden"]), dtype=torch.float64, device=DEV)])
    dw = torch.cat([s["dweights"].double(), torch.zeros(1, dtype=torch.float64, device=DEV)])
    R, cap, K = s["layout"]["slot_row"].shape
    at = s["layout"]["slot_row"].long()
    for r in range(R):
        at[r, int(s["num_recv"][r]):] = -1
    out = torch.zeros((R, cap, case["hidden"]), dtype=torch.float64, device=DEV)
    for k in range(K):
        out += y[at[:, :, k]]
    return dict(out=out, out_topk_weights=dw[at])


_EXACT = dict(product=_exact_product, product_fp8=_exact_product_fp8, swiglu=_exact_swiglu,
              expert_rows=_exact_expert_rows)
