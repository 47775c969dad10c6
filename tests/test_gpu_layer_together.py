"""The router, the products with an epilogue, the dispatch and the combine, and the layer for a few tokens, as a program
uses them together: a training step against automatic differentiation in 64 bits, and decode steps.

Tolerances, fixed before the first run: values and gradients pass through chains of bf16 roundings, each at most 2^-8 of its
value and independent of the others; of d roundings in a row the whole (its norm) is off by less than d * 2^-8.  The step's
longest chains: nine for the output, fourteen for a gradient."""
import pytest
import torch

from combine_get_dispatch_03_gb300 import ep
from examples import moe_layer as M
from test_gpu_experts import DEV, gen, i32, randn

pytestmark = pytest.mark.gpu


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def setup(seed, R, T, E, K, H, I):
    g = gen(seed)
    h = ep.Handle(ep.Config(num_ranks=R, num_max_tokens=T, hidden=H, num_experts=E, num_topk=K, recv_capacity=R * T))
    one = ep.Handle(ep.Config(num_ranks=1, num_max_tokens=R * T, hidden=H, num_experts=1, num_topk=1))
    w = dict(gate=randn(g, (1, E, H), H ** -0.5), up=randn(g, (E, 2 * I, H), H ** -0.5), up_bias=torch.randn((E, 2 * I), generator=g, device=DEV) * 0.1,
             down=randn(g, (E, H, I), I ** -0.5), shared_up=randn(g, (1, I, H), H ** -0.5), shared_down=randn(g, (1, H, I), I ** -0.5),
             select=torch.randn(E, generator=g, device=DEV) * 0.02)
    return g, h, one, w


@pytest.mark.parametrize("score,groups,kept", [("softmax", 1, 1), ("sigmoid", 4, 2)])
def test_training_step(score, groups, kept):
    R, T, E, K, H, I = 4, 24, 16, 3, 256, 136
    g, h, one, w = setup(3, R, T, E, K, H, I)
    x, dy = randn(g, (R, T, H)), randn(g, (R, T, H))
    n = i32([R * T])
    kw = dict(score=score, scale=2.0)
    # forward
    logits = ep.ep_grouped_gemm_act(one, x.view(1, R * T, H), w["gate"], n, out_dtype=torch.float32)["out"].view(R, T, E)
    r = ep.ep_router(h, logits, bias=w["select"], num_groups=groups, kept_groups=kept, **kw)
    ep.ep_layout_notify(h, r["topk_idx"])
    d = ep.ep_dispatch(h, x, topk_idx=r["topk_idx"], topk_weights=r["topk_weights"], prepared=True)
    rows = R * T * K
    lay = ep.ep_expert_layout(h, d["recv_topk_idx"], rows)
    c, b = lay["group_count"], lay["group_begin"]
    q = ep.ep_expert_gather(h, d["recv_x"], lay["slot_row"], rows, topk_weights=d["recv_topk_weights"])
    f = ep.ep_grouped_gemm_act(h, q["out"], w["up"], c, b, bias=w["up_bias"], act="silu", gated=True, row_weights=q["row_weights"], keep_pre=True)
    back = ep.ep_expert_reduce(h, ep.ep_grouped_gemm(h, f["out"], w["down"], c, b), lay["slot_row"])["out"]
    s = ep.ep_grouped_gemm_act(one, x.view(1, R * T, H), w["shared_up"], n, act="gelu", keep_pre=True)
    shared = ep.ep_grouped_gemm_act(one, s["out"], w["shared_down"], n, residual=x.view(1, R * T, H))["out"].view(R, T, H)
    y = ep.ep_combine(h, back, bias_0=shared)["combined_x"]
    # backward
    drecv = ep.ep_dispatch(h, dy, cached=True)["recv_x"]
    ddown = ep.ep_expert_gather(h, drecv, lay["slot_row"], rows)["out"]
    dact = ep.ep_grouped_gemm(h, ddown, w["down"], c, b, w_transposed=True)
    a = ep.ep_act_grad(h, dact, f["pre"], c, b, act="silu", gated=True, row_weights=q["row_weights"], with_bias=True)
    grads = dict(down=ep.ep_grouped_gemm_wgrad(h, ddown, f["out"], c, b), up=ep.ep_grouped_gemm_wgrad(h, a["d_pre"], q["out"], c, b), up_bias=a["d_bias"])
    dq = ep.ep_grouped_gemm(h, a["d_pre"], w["up"], c, b, w_transposed=True)
    red = ep.ep_expert_reduce(h, dq, lay["slot_row"], row_weights=a["d_row_weights"])
    k = ep.ep_combine(h, red["out"], topk_weights=red["out_topk_weights"])
    dlogits = ep.ep_router_grad(h, logits, r["topk_idx"], k["combined_topk_weights"], **kw)
    dy1 = dy.view(1, R * T, H)
    ds = ep.ep_grouped_gemm(one, dy1, w["shared_down"], n, w_transposed=True)
    sa = ep.ep_act_grad(one, ds, s["pre"], n, act="gelu")
    grads["shared_down"] = ep.ep_grouped_gemm_wgrad(one, dy1, s["out"], n)
    grads["shared_up"] = ep.ep_grouped_gemm_wgrad(one, sa["d_pre"], x.view(1, R * T, H), n)
    dl = dlogits.view(1, R * T, E).to(torch.bfloat16)
    grads["gate"] = ep.ep_grouped_gemm_wgrad(one, dl, x.view(1, R * T, H), n)
    through_gate = ep.ep_grouped_gemm_act(one, dl, w["gate"].transpose(1, 2).contiguous(), n, residual=k["combined_x"].view(1, R * T, H))["out"]
    through_shared = ep.ep_grouped_gemm_act(one, sa["d_pre"], w["shared_up"].transpose(1, 2).contiguous(), n, residual=dy1)["out"]
    dx = through_gate.float() + through_shared.float()
    h.check()
    one.check()
    # the same in 64 bits, the choice held
    v = {key: t.double().requires_grad_(key != "select") for key, t in w.items()}
    xd = x.view(-1, H).double().requires_grad_()
    lg = xd @ v["gate"][0].t()
    p = torch.softmax(lg, 1) if score == "softmax" else torch.sigmoid(lg)
    idx = r["topk_idx"].view(-1, K)
    cw = p.gather(1, idx)
    cw = 2.0 * cw / cw.sum(1, keepdim=True)
    want = xd + torch.nn.functional.gelu(xd @ v["shared_up"][0].t()) @ v["shared_down"][0].t()
    for e in range(E):
        t, slot = torch.nonzero(idx == e, as_tuple=True)
        u = xd[t] @ v["up"][e].t() + v["up_bias"][e]
        o = (torch.nn.functional.silu(u[:, :I]) * u[:, I:]) @ v["down"][e].t() * cw[t, slot][:, None]
        want = want.index_add(0, t, o)
    want.backward(dy.view(-1, H).double())
    assert off(y.view(-1, H), want.detach()) < 9 * 2.0 ** -8
    for key, got in grads.items():
        assert off(got, v[key].grad) < 14 * 2.0 ** -8, key
    assert off(dx.view(-1, H), xd.grad) < 14 * 2.0 ** -8


@pytest.mark.parametrize("R,T", [(1, 1), (2, 4), (4, 16)])
def test_decode_steps(R, T):
    """Logits, router, shared expert and layer, in one graph, replayed; bf16 and FP8 weights, and the example's path."""
    E, K, H, I = 16, 4, 512, 256
    g, h, one, w = setup(R * T, R, T, E, K, H, I)
    x = randn(g, (R, T, H))
    n = i32([R * T])
    up, down = M.quantize(w["up"]), M.quantize(w["down"])

    def step(fp8):
        logits = ep.ep_grouped_gemm_act(one, x.view(1, R * T, H), w["gate"], n, out_dtype=torch.float32)["out"].view(R, T, E)
        r = ep.ep_router(h, logits, bias=w["select"], score="sigmoid", num_groups=4, kept_groups=2)
        s = ep.ep_grouped_gemm_act(one, x.view(1, R * T, H), w["shared_up"], n, act="gelu")["out"]
        shared = ep.ep_grouped_gemm_act(one, s, w["shared_down"], n, residual=x.view(1, R * T, H))["out"].view(R, T, H)
        weights = (up[0], down[0]) if fp8 else (w["up"], w["down"])
        scales = dict(up_scales=up[1], down_scales=down[1]) if fp8 else {}
        return r, ep.ep_moe_layer(h, x, r["topk_idx"], r["topk_weights"], *weights, bias_0=shared, **scales)

    for fp8 in (False, True):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r, y = step(fp8)
        for _ in range(2):
            x.copy_(randn(g, (R, T, H)))
            graph.replay()
            e, again = step(fp8)
            assert torch.equal(r["topk_idx"], e["topk_idx"]) and torch.equal(y, again)
            xd = x.view(-1, H).double()
            want = xd + torch.nn.functional.gelu(xd @ w["shared_up"][0].double().t()) @ w["shared_down"][0].double().t()
            wide = [(c.double().view(E, -1, 128, c.shape[2] // 128, 128) * sc.double()[:, :, None, :, None]).view(c.shape) for c, sc in (up, down)] \
                if fp8 else [w["up"].double(), w["down"].double()]
            for ex in range(E):
                t, slot = torch.nonzero(r["topk_idx"].view(-1, K) == ex, as_tuple=True)
                u = xd[t] @ wide[0][ex].t()
                o = (torch.nn.functional.silu(u[:, :I]) * u[:, I:]) @ wide[1][ex].t()
                want.index_add_(0, t, o * r["topk_weights"].view(-1, K)[t, slot].double()[:, None])
            assert off(y.view(-1, H), want) < 6 * 2.0 ** -8
    h.check()
    one.check()


# Waits that run out, as for the grouped products: one CTA or a few with a contraction of 2^18 take longer than the quarter
# of a millisecond after which a limit of a microsecond is noticed.  Every wait would be met later.
@pytest.mark.parametrize("ctas", [1, 3])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_layer_wait_that_runs_out(ctas, fp8):
    H, I = 1 << 18, 128
    h = ep.Handle(ep.Config(num_ranks=1, num_max_tokens=2, hidden=H, num_experts=1, num_topk=1, max_sms=ctas))
    one = torch.float8_e4m3fn if fp8 else torch.bfloat16
    x = torch.ones((1, 2, H), dtype=torch.bfloat16, device=DEV)
    up, down = torch.ones((1, 2 * I, H), device=DEV).to(one), torch.ones((1, H, I), device=DEV).to(one)
    kw = dict(up_scales=torch.full((1, 2 * I // 128, H // 128), 2.0 ** -18, device=DEV), down_scales=torch.ones((1, H // 128, I // 128), device=DEV)) if fp8 else {}
    if not fp8:
        up *= 2.0 ** -18
    idx, tw = torch.zeros((1, 2, 1), dtype=torch.int64, device=DEV), torch.ones((1, 2, 1), device=DEV)
    want = ep.ep_moe_layer(h, x, idx, tw, up, down, **kw)
    h.check()
    silu1 = torch.nn.functional.silu(torch.ones((), dtype=torch.float64)).to(torch.bfloat16).double()  # sums of 2^18 times 2^-18
    assert (want.double() - 128 * silu1).abs().max() <= 2.0 ** -8 * 128 * silu1
    ep.ep_selftest_wait_limit(h, 1000)
    ep.ep_moe_layer(h, x, idx, tw, up, down, **kw)
    assert h.status() == 3
    ep.ep_selftest_wait_limit(h)
    for _ in range(3):
        assert torch.equal(ep.ep_moe_layer(h, x, idx, tw, up, down, **kw), want)
    h.check()


@pytest.mark.parametrize("form", ["bf16", "gated"])  # fp32 sums are waited for every 512 rows: no wait is long
@pytest.mark.parametrize("ctas,bits", [(1, 18), (4, 20)])  # as many steps a CTA
def test_product_wait_that_runs_out(form, ctas, bits):
    """With four CTAs the contraction is cut, and the parts' tickets are as before afterwards."""
    k, n = 1 << bits, 16
    h = ep.Handle(ep.Config(num_ranks=1, num_max_tokens=2, hidden=8, num_experts=1, num_topk=1, max_sms=ctas))
    x, w = torch.ones((2, k), dtype=torch.bfloat16, device=DEV), torch.full((1, n, k), 2.0 ** -bits, dtype=torch.bfloat16, device=DEV)
    res, c = torch.ones((2, n // 2 if form == "gated" else n), dtype=torch.bfloat16, device=DEV), i32([2])
    kw = dict(residual=res, gated=form == "gated", act="relu")
    want = ep.ep_grouped_gemm_act(h, x, w, c, **kw)["out"]
    h.check()
    assert (want == 2).all()
    ep.ep_selftest_wait_limit(h, 1000)
    ep.ep_grouped_gemm_act(h, x, w, c, **kw)
    assert h.status() == 3
    ep.ep_selftest_wait_limit(h)
    for _ in range(3):
        assert torch.equal(ep.ep_grouped_gemm_act(h, x, w, c, **kw)["out"], want)
    h.check()
