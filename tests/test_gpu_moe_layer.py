"""The layer for a few tokens against a plain 64-bit form.

Tolerances, fixed before the first run.  With magnitudes M_g, M_u of gate and up (sums of |w| |x|), a tensor-core sum over m
is off by (m / 16 + 8) * 2^-22 of its magnitude; with FP8 weights the tokens' split leaves 2^-17 of a block's largest value, at most 2^-17 of
the row's largest, times the sum of |w|.  silu changes by at most 1.1 of what its argument does and adds 2^-19 of itself; gate * up
is rounded to bf16 (2^-8).  That error goes through |w_down|, the second sum adds its own, the weights 2^-22, and the output is rounded (2^-8)."""
import threading

import pytest
import torch

from combine_get_dispatch_03_gb300 import ep
from _parity import Guarded
from test_gpu_experts import DEV, gen, randn

pytestmark = pytest.mark.gpu


def layer_handle(R, T, H, E, K, max_sms=0):
    return ep.Handle(ep.Config(num_ranks=R, num_max_tokens=max(T, 1), hidden=H, num_experts=E, num_topk=K, max_sms=max_sms))


def choose(g, R, T, E, K):
    return torch.rand((R, T, E), generator=g, device=DEV).topk(K).indices


def weights(g, E, H, I, fp8):
    """(w_up, up_scales, w_down, down_scales) of unit gain."""
    if not fp8:
        return randn(g, (E, 2 * I, H), H ** -0.5), None, randn(g, (E, H, I), I ** -0.5), None

    def codes(n, k):
        c = (torch.randn((E, n, k), generator=g, device=DEV) * 128).clamp(-448, 448).to(torch.float8_e4m3fn)
        return c, (torch.rand((E, n // 128, k // 128), generator=g, device=DEV) + 0.5) / 128 * k ** -0.5
    return codes(2 * I, H) + codes(H, I)


def dense(w, scales, e):
    w = w[e].double()
    if scales is not None:
        w = w * scales[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    return w


def reference(x, idx, tw, w, bias=(), mask=None):
    """(result, tolerance) in 64 bits."""
    w_up, up_s, w_down, down_s = w
    R, T, H = x.shape
    E, I, K = w_up.shape[0], w_up.shape[1] // 2, idx.shape[2]
    fp8 = up_s is not None
    xd = x.reshape(-1, H).double()
    ok = (idx >= 0) & (idx < E)
    if mask is not None:
        m = torch.tensor(mask, dtype=torch.bool, device=DEV)
        ok = ok & ~m[:, None, None] & ~m[idx.clamp(0, E - 1) // (E // R)]
    i, ok, tw = idx.view(-1, K), ok.view(-1, K), tw.view(-1, K).double()
    y, tol = torch.zeros_like(xd), torch.zeros_like(xd)
    for e in i[ok].unique().tolist():
        t, k = torch.nonzero((i == e) & ok, as_tuple=True)
        up, down = dense(w_up, up_s, e), dense(w_down, down_s, e)
        v, m = xd[t] @ up.t(), xd[t].abs() @ up.abs().t()
        tv = (H / 16 + 8) * 2.0 ** -22 * m
        if fp8:
            tv = tv + 2.0 ** -17 * xd[t].abs().amax(1, keepdim=True) * up.abs().sum(1)
        s = v[:, :I] * torch.sigmoid(v[:, :I])
        ts = 1.1 * tv[:, :I] + 2.0 ** -19 * s.abs()
        a = s * v[:, I:]
        ta = ts * v[:, I:].abs() + s.abs() * tv[:, I:] + ts * tv[:, I:] + 2.0 ** -8 * a.abs() * (1 + 2.0 ** -8)
        if fp8:
            ta = ta + 2.0 ** -17 * a.abs().amax(1, keepdim=True)
        o, to = a @ down.t(), ta @ down.abs().t() + (I / 16 + 8) * 2.0 ** -22 * (a.abs() @ down.abs().t())
        p = tw[t, k][:, None]
        y.index_add_(0, t, p * o)
        tol.index_add_(0, t, p.abs() * (to + 2.0 ** -21 * o.abs()))
    for b in bias:
        y = y + b.view(-1, H).double()
        tol = tol + 2.0 ** -22 * (y.abs() + b.view(-1, H).double().abs())
    return y.view(x.shape), (tol * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs() + 1e-37).view(x.shape)


def within(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - want).abs() / tol).max())} x the tolerance"
    # roundings do not conspire: the whole is off by less than two of them (2^-8 each)
    if bool((want != 0).any()):
        assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -7


def run(h, x, idx, tw, w, **kw):
    out = Guarded(tuple(x.shape), torch.bfloat16)
    ep.ep_moe_layer(h, x, idx, tw, w[0], w[2], up_scales=w[1], down_scales=w[3], out=out.t, **kw)
    out.check()
    return out.t


SHAPES = [  # R, T, E, K, H, I
    (1, 1, 1, 1, 128, 128),
    (1, 1, 4, 2, 256, 384),
    (1, 3, 16, 4, 1024, 128),
    (2, 8, 8, 2, 512, 256),
    (1, 16, 8, 8, 384, 640),
    (1, 17, 5, 3, 256, 128),
    (8, 4, 32, 4, 1024, 512),
    (4, 16, 8, 8, 512, 384),
    (8, 8, 64, 6, 256, 256),
    (1, 64, 2, 1, 128, 256),
    (1, 2, 3, 3, 3968, 2176),
    (16, 1, 2048, 32, 128, 128),
    (2, 32, 2048, 32, 128, 128),
    (1, 9, 16, 3, 640, 128),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("biases", [0, 1, 2])
def test_layer(shape, fp8, biases):
    R, T, E, K, H, I = shape
    g = gen(H + I + T)
    h = layer_handle(R, T, H, E, K)
    w = weights(g, E, H, I, fp8)
    x, idx, tw = randn(g, (R, T, H)), choose(g, R, T, E, K), torch.softmax(torch.randn((R, T, K), generator=g, device=DEV), -1)
    bias = [randn(g, (R, T, H)) for _ in range(biases)]
    kw = {f"bias_{i}": b for i, b in enumerate(bias)}
    out = run(h, x, idx, tw, w, **kw)
    h.check()
    within(out, *reference(x, idx, tw, w, bias))
    for _ in range(3):  # the same bits, call after call
        assert torch.equal(run(h, x, idx, tw, w, **kw), out)
    h.check()


@pytest.mark.parametrize("R,T,E,K,H,I", [(1, 5, 7, 3, 264, 200), (1, 1, 3, 2, 8, 8), (2, 9, 6, 2, 136, 1000), (1, 40, 5, 4, 2056, 72),
                                         (1, 64, 4, 2, 72, 136), (1, 2, 2, 2, 4104, 8), (1, 13, 4, 4, 8, 264)])
def test_sizes_that_are_no_multiple(R, T, E, K, H, I):
    g = gen(H)
    h = layer_handle(R, T, H, E, K)
    w = weights(g, E, H, I, False)
    x, idx, tw = randn(g, (R, T, H)), choose(g, R, T, E, K), torch.rand((R, T, K), generator=g, device=DEV)
    out = run(h, x, idx, tw, w)
    h.check()
    within(out, *reference(x, idx, tw, w))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_slots_left_out_and_named_twice(fp8):
    R, T, E, K, H, I = 2, 6, 8, 4, 256, 128
    g = gen(3)
    h = layer_handle(R, T, H, E, K)
    w = weights(g, E, H, I, fp8)
    x, idx, tw = randn(g, (R, T, H)), choose(g, R, T, E, K), torch.rand((R, T, K), generator=g, device=DEV)
    b = randn(g, (R, T, H))
    idx[0, 0] = -1                       # a token without experts
    idx[0, 1, 1:] = -1
    idx[0, 2, 3] = idx[0, 2, 0]          # twice
    idx[1, 3] = 5                        # four times
    idx[1, 4, 0] = -1
    tw[0, 0] = float("nan")              # of slots without an expert: not read
    out = run(h, x, idx, tw, w, bias_0=b)
    h.check()
    again = tw.clone()
    again[0, 0] = 0
    within(out, *reference(x, idx, again, w, [b]))
    assert torch.equal(out[0, 0], b[0, 0])
    place = b.clone()                    # a bias may be the output
    ep.ep_moe_layer(h, x, idx, tw, w[0], w[2], up_scales=w[1], down_scales=w[3], bias_0=place, out=place)
    assert torch.equal(place, out)
    none = run(h, x, torch.full_like(idx, -1), tw, w, bias_1=b)
    h.check()
    assert torch.equal(none, b)
    assert (run(h, x, torch.full_like(idx, -1), tw, w) == 0).all()
    tw = again
    everyone = torch.full_like(idx, -1)
    everyone[..., 2] = 7                 # one expert for all tokens
    within(run(h, x, everyone, tw, w), *reference(x, everyone, tw, w))
    h.check()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_masked_ranks(fp8):
    R, T, E, K, H, I = 4, 3, 8, 4, 128, 256
    g = gen(9)
    h = layer_handle(R, T, H, E, K)
    w = weights(g, E, H, I, fp8)
    x, idx, tw = randn(g, (R, T, H)), choose(g, R, T, E, K), torch.rand((R, T, K), generator=g, device=DEV)
    for mask in ([0, 1, 0, 0], [1, 0, 0, 1], [1, 1, 1, 1]):
        ep.ep_clean_mask_buffer(h)
        for r, m in enumerate(mask):
            ep.ep_update_mask_buffer(h, r, bool(m))
        out = run(h, x, idx, tw, w)
        h.check()
        within(out, *reference(x, idx, tw, w, mask=mask))


def test_bad_experts_are_reported_and_left_out():
    g = gen(2)
    h = layer_handle(1, 4, 128, 8, 2)
    w = weights(g, 8, 128, 64, False)
    x, idx, tw = randn(g, (1, 4, 128)), choose(g, 1, 4, 8, 2), torch.rand((1, 4, 2), generator=g, device=DEV)
    for bad in (8, -2, 1 << 40, -(1 << 62)):
        wrong = idx.clone()
        wrong[0, 2, 1] = bad
        out = run(h, x, wrong, tw, w)
        assert h.status() == 7
        wrong[0, 2, 1] = -1
        assert torch.equal(out, run(h, x, wrong, tw, w))
        h.check()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T", [7, 33])
def test_special_values_stay_in_their_token(fp8, T):
    E, K, H, I = 6, 2, 256, 256
    g = gen(T)
    h = layer_handle(1, T, H, E, K)
    w = weights(g, E, H, I, fp8)
    x, idx, tw = randn(g, (1, T, H)), choose(g, 1, T, E, K), torch.rand((1, T, K), generator=g, device=DEV)
    clean = run(h, x, idx, tw, w)
    x2 = x.clone()
    x2[0, 2, 9], x2[0, 4, 200] = float("nan"), float("inf")
    out = run(h, x2, idx, tw, w)
    h.check()
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[2] = keep[4] = False
    assert torch.equal(out[0, keep], clean[0, keep])
    assert out[0, 2].isnan().all() and not out[0, 4].isfinite().any()
    # an expert that no token has may hold anything
    alone = torch.full_like(idx, 3)
    want = run(h, x, alone, tw, w)
    for t in (w[0], w[2]):
        t.view(torch.uint8)[torch.arange(E, device=DEV) != 3] = 0xff
    assert torch.equal(run(h, x, alone, tw, w), want)
    h.check()


def test_tokens_of_all_magnitudes_with_fp8_weights():
    """The split follows a block's magnitude: subnormal, tiny, huge and mixed tokens, and zeros."""
    E, K, H, I = 4, 2, 512, 256
    g = gen(14)
    h = layer_handle(1, 8, H, E, K)
    w = weights(g, E, H, I, True)
    x = randn(g, (1, 8, H)).float()
    for t, f in enumerate((1.0, 0.0, 1e-3, 1e-12, 1e3, 1e-38, 1.0, 1.0)):
        x[0, t] *= f
    x[0, 6, :128] *= 1e4      # one block far above the others
    x[0, 7, 5] = 3e4          # one outlier in a block
    x = x.to(torch.bfloat16)
    idx, tw = choose(g, 1, 8, E, K), torch.rand((1, 8, K), generator=g, device=DEV)
    out = run(h, x, idx, tw, w)
    h.check()
    assert (out[0, 1] == 0).all()
    want, tol = reference(x, idx, tw, w)
    bad = ~((out.double() - want).abs() <= tol)
    assert not bad.any()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("max_sms", [1, 2, 7, 64])
@pytest.mark.parametrize("T", [3, 40])
def test_any_number_of_ctas(fp8, max_sms, T):
    """One CTA has all the work, or several share a tile in every way."""
    E, K, H, I = 5, 2, 384, 256
    g = gen(max_sms)
    h = layer_handle(1, T, H, E, K, max_sms=max_sms)
    w = weights(g, E, H, I, fp8)
    x, idx, tw = randn(g, (1, T, H)), choose(g, 1, T, E, K), torch.rand((1, T, K), generator=g, device=DEV)
    out = run(h, x, idx, tw, w)
    h.check()
    within(out, *reference(x, idx, tw, w))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_captured_side_stream_and_other_calls_between(fp8):
    R, T, E, K, H, I = 2, 4, 16, 4, 512, 256
    g = gen(6)
    h = layer_handle(R, T, H, E, K)
    w = weights(g, E, H, I, fp8)
    x, tw = randn(g, (R, T, H)), torch.rand((R, T, K), generator=g, device=DEV)
    logits = torch.randn((R, T, E), generator=g, device=DEV)
    kw = dict(up_scales=w[1], down_scales=w[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # the first calls of the handle
        r = ep.ep_router(h, logits)
        y = ep.ep_moe_layer(h, x, r["topk_idx"], r["topk_weights"], w[0], w[2], bias_0=x, **kw)
        z = ep.ep_moe_layer(h, y, r["topk_idx"], r["topk_weights"], w[0], w[2], **kw)
    for _ in range(3):
        x.copy_(randn(g, (R, T, H)))
        logits.copy_(torch.randn((R, T, E), generator=g, device=DEV))
        graph.replay()
        e = ep.ep_router(h, logits)
        a = ep.ep_moe_layer(h, x, e["topk_idx"], e["topk_weights"], w[0], w[2], bias_0=x, **kw)
        assert torch.equal(y, a)
        assert torch.equal(z, ep.ep_moe_layer(h, a, e["topk_idx"], e["topk_weights"], w[0], w[2], **kw))
    idx = choose(g, R, T, E, K)
    want = ep.ep_moe_layer(h, x, idx, tw, w[0], w[2], **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = [ep.ep_moe_layer(h, x, idx, tw, w[0], w[2], stream=side, **kw) for _ in range(20)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, want) for a in again)
    ep.ep_ll_dispatch(h, x, idx)
    assert torch.equal(ep.ep_moe_layer(h, x, idx, tw, w[0], w[2], **kw), want)
    h.check()


def test_against_the_low_latency_path():
    """The same layer by dispatch, products and combine, in bf16: apart by the roundings between its calls."""
    R, T, E, K, H, I = 4, 8, 16, 4, 512, 256
    g = gen(8)
    h = layer_handle(R, T, H, E, K)
    w = weights(g, E, H, I, False)
    x, idx, tw = randn(g, (R, T, H)), choose(g, R, T, E, K), torch.softmax(torch.randn((R, T, K), generator=g, device=DEV), -1)
    y = ep.ep_moe_layer(h, x, idx, tw, w[0], w[2])
    d = ep.ep_ll_dispatch(h, x, idx, use_fp8=False)
    px, _, _ = ep.ll_views(d["recv_msgs"], H, False)
    a = ep.ep_grouped_gemm_act(h, px, w[0], d["packed_recv_count"], act="silu", gated=True, expected_rows=8)["out"]
    back = ep.ep_ll_combine(h, ep.ep_grouped_gemm(h, a, w[2], d["packed_recv_count"], expected_rows=8), idx, tw)
    h.check()
    # one rounding of the activation and of the output in each, one of the expert's output in the path: five of 2^-8 at most
    assert float((y.double() - back.double()).norm() / y.double().norm()) < 5 * 2.0 ** -8


def test_first_cuda_call_of_a_thread():
    g = gen(2)
    h = layer_handle(1, 4, 128, 8, 2)
    w = weights(g, 8, 128, 64, False)
    x, idx, tw = randn(g, (1, 4, 128)), choose(g, 1, 4, 8, 2), torch.rand((1, 4, 2), generator=g, device=DEV)
    want, out = run(h, x, idx, tw, w), torch.zeros_like(x)
    torch.cuda.synchronize()
    errors = []

    def call():
        try:
            ep.ep_moe_layer(h, x, idx, tw, w[0], w[2], out=out)
        except Exception as e:  # noqa: BLE001 -- shown by the thread that started this one
            errors.append(e)
    thread = threading.Thread(target=call)
    thread.start()
    thread.join()
    assert not errors, errors
    h.check()
    assert torch.equal(out, want)


def test_refusals():
    h = layer_handle(2, 40, 264, 4, 2)
    g = gen(1)
    w = weights(g, 4, 264, 128, False)

    def args(T):
        return randn(g, (2, T, 264)), choose(g, 2, T, 4, 2), torch.rand((2, T, 2), generator=g, device=DEV)

    assert ep.ep_moe_layer(h, *args(0), w[0], w[2]).shape == (2, 0, 264)
    assert ep.ep_moe_layer(h, *args(32), w[0], w[2]).shape == (2, 32, 264)
    for T in (33, 41):  # more than 64 in all; more than the handle's
        with pytest.raises(ep.EPError):
            ep.ep_moe_layer(h, *args(T), w[0], w[2])
    x, idx, tw = args(4)
    codes = [t.to(torch.float8_e4m3fn) for t in (w[0], w[2])]
    ones = [torch.ones((4, 2, 2), device=DEV), torch.ones((4, 2, 1), device=DEV)]
    with pytest.raises(ep.EPError):
        ep.ep_moe_layer(h, x, idx, tw, *codes, *ones)  # hidden 264 is no multiple of 128
    for call in (lambda: ep.ep_moe_layer(h, x, idx, tw, w[0], w[2].transpose(1, 2)),
                 lambda: ep.ep_moe_layer(h, x, idx, tw, w[0], w[2][:3]),
                 lambda: ep.ep_moe_layer(h, x, idx.int(), tw, w[0], w[2]),
                 lambda: ep.ep_moe_layer(h, x, idx, tw[:1], w[0], w[2]),
                 lambda: ep.ep_moe_layer(h, x, idx, tw, w[0], codes[1]),
                 lambda: ep.ep_moe_layer(h, x, idx, tw, w[0], w[2], bias_0=x[:, :2]),
                 lambda: ep.ep_moe_layer(h, x, idx, tw, w[0][:, :252].contiguous(), w[2][..., :126].contiguous())):
        with pytest.raises((ValueError, TypeError, ep.EPError)):
            call()
    h8 = layer_handle(1, 4, 256, 4, 2)
    w8 = weights(g, 4, 256, 128, True)
    x8, i8, t8 = randn(g, (1, 4, 256)), choose(g, 1, 4, 4, 2), torch.rand((1, 4, 2), generator=g, device=DEV)
    for up, down in ((None, None), (w8[1], None), (w8[1][:, :1], w8[3])):
        with pytest.raises((ValueError, ep.EPError)):
            ep.ep_moe_layer(h8, x8, i8, t8, w8[0], w8[2], up_scales=up, down_scales=down)
    L, st = ep.lib(), torch.cuda.current_stream().cuda_stream
    need = L.ep_moe_layer_workspace(h8.ptr, 4, 128)
    assert need > 0 and L.ep_moe_layer_workspace(h8.ptr, 65, 128) == -1
    ws, out = torch.zeros(need, dtype=torch.uint8, device=DEV), torch.zeros_like(x8)
    base = [h8.ptr, 4, 128, x8.data_ptr(), i8.data_ptr(), t8.data_ptr(), w8[0].data_ptr(), w8[1].data_ptr(), w8[2].data_ptr(),
            w8[3].data_ptr(), 1, None, None, out.data_ptr()]
    assert L.ep_moe_layer(*base, ws.data_ptr(), need - 1, st) == 1 and b"workspace" in L.ep_last_error()
    assert L.ep_moe_layer(*base, None, need, st) == 1
    assert L.ep_moe_layer(*base, ws.data_ptr(), need, st) == 0
    h.check()
    h8.check()
