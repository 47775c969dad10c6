"""Products with an epilogue and the epilogue's gradient against plain 64-bit forms.

Tolerances, fixed before the first run.  A sum v of products is off by tol_v = (k / 16 + 8) * 2^-22 of its sum of
magnitudes (test_gpu_experts.py), and 2^-23 of |v| with the bias.  An activation changes by at most 1.13 of what its argument does
(gelu; silu 1.1) and adds 2^-19 of its own value (exp and reciprocal 2^-22 each, erfc four units, an argument of up to 8
squared in exp 2^-19); a product with an up value, a weight, a residual 2^-23 each; the output's rounding is 2^-8 (bf16) or 2^-24.
A gradient: 2^-18 of the magnitudes of its terms for the derivative, and its rounding; sums of m of them m * 2^-24 of their
magnitudes more."""
import math

import pytest
import torch

from combine_get_dispatch_03_gb300 import ep
from _parity import Guarded
from test_gpu_experts import COUNTS, DEV, gen, handle, i32, packed, randn

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu"]


def act64(v, act):
    """(value, derivative) in 64 bits."""
    if act == "none":
        return v, torch.ones_like(v)
    if act == "relu":
        return v.clamp(min=0), (v > 0).double()
    if act == "silu":
        s = torch.sigmoid(v)
        return v * s, s * (1 + v * (1 - s))
    c = 0.5 * torch.erfc(-v / math.sqrt(2))
    return v * c, c + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)


def within(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - want).abs() / tol).max())} x the tolerance"


def check_forward(counts, n, k, act, gated, with_bias, weighted, with_residual, keep, dtype, expected, pad=0, gap=2, max_sms=0):
    E, width = len(counts), n // 2 if gated else n
    begin, rows = packed(counts, gap=gap)
    g = gen(n * 7 + k)
    x = torch.full((rows, k), float("nan"), dtype=torch.bfloat16, device=DEV)  # rows of no group
    for b, c in zip(begin, counts):
        x[b:b + c] = randn(g, (c, k))
    w = randn(g, (E, n, k), 2 * k ** -0.5)
    bias = torch.randn((E, n), generator=g, device=DEV) if with_bias else None
    weights = torch.rand(rows, generator=g, device=DEV) if weighted else None
    rows_pad = pad // 8 * 8  # of bf16 rows: multiples of 16 bytes
    residual = randn(g, (rows, width + rows_pad))[:, :width] if with_residual else None
    out, pre = Guarded((rows, width + pad), dtype), Guarded((rows, n + rows_pad), torch.bfloat16)
    h = handle(E, max_sms=max_sms)
    r = ep.ep_grouped_gemm_act(h, x, w, i32(counts), i32(begin), bias=bias, act=act, gated=gated, row_weights=weights,
                               residual=residual, pre=pre.t[:, :n] if keep else None, out=out.t[:, :width], expected_rows=expected)
    h.check()
    out.check()
    pre.check()
    assert (r["pre"] is not None) == keep
    used = torch.zeros(rows, dtype=torch.bool, device=DEV)
    eps = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    for e, (b, c) in enumerate(zip(begin, counts)):
        used[b:b + c] = True
        xe, we = x[b:b + c].double(), w[e].double().t()
        v, tol = xe @ we, (k / 16 + 8) * 2.0 ** -22 * (xe.abs() @ we.abs())
        if with_bias:
            v = v + bias[e].double()
            tol = tol + 2.0 ** -23 * v.abs()
        if keep:
            within(pre.t[b:b + c, :n], v, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * v.abs() + 1e-37)
        gate, up, tol_gate, tol_up = v[:, :width], 1.0, tol[:, :width], 0.0
        if gated:
            up, tol_up = v[:, width:], tol[:, width:]
        a, _ = act64(gate, act)
        tol = 1.13 * tol_gate + 2.0 ** -19 * a.abs()
        if gated:
            tol = tol * up.abs() + a.abs() * tol_up + tol * tol_up + 2.0 ** -23 * (a * up).abs()
            a = a * up
        if weighted:
            p = weights[b:b + c].double()[:, None]
            a, tol = a * p, tol * p + 2.0 ** -23 * (a * p).abs()
        if with_residual:
            a = a + residual[b:b + c].double()
            tol = tol + 2.0 ** -23 * (a.abs() + residual[b:b + c].double().abs())
        within(out.t[b:b + c, :width], a, tol * (1 + eps) + eps * a.abs() + 1e-37)
    assert (out.t[~used].contiguous().view(torch.uint8) == out.fill).all(), "a row outside every group was written"
    assert (out.t[:, width:].contiguous().view(torch.uint8) == out.fill).all()
    if keep:
        assert (pre.t[~used].contiguous().view(torch.uint8) == pre.fill).all()


@pytest.mark.parametrize("n,k", [(16, 8), (64, 64), (144, 136), (1008, 72), (528, 1032)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}g{sum(c)}")
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("expected", [1, 100000], ids=["single", "pair"])
def test_all_parts(counts, n, k, gated, expected):
    check_forward(counts, n, k, "silu", gated, True, True, True, True, torch.bfloat16, expected)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("parts", [0, 1, 2, 4, 8], ids=["alone", "bias", "weights", "residual", "pre"])
@pytest.mark.parametrize("pad", [0, 8])
def test_each_part_and_activation(act, gated, parts, pad):
    check_forward([33, 0, 200, 7], 272, 328, act, gated, bool(parts & 1), bool(parts & 2), bool(parts & 4), bool(parts & 8),
                  torch.bfloat16, 0, pad=pad)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n,pad", [(8, 0), (72, 4), (256, 0), (1000, 12)])
@pytest.mark.parametrize("expected", [1, 100000], ids=["single", "pair"])
def test_fp32_output(act, n, pad, expected):
    check_forward([130, 0, 31, 300], n, 136, act, False, True, True, True, n == 72, torch.float32, expected, pad=pad)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n", [48, 272, 528])
@pytest.mark.parametrize("k", [256, 1032])
@pytest.mark.parametrize("expected", [40, 100000])
def test_many_tiles_a_cta(gated, n, k, expected):
    """Results through shared memory (k up to 512) and by lanes, ragged ends, several tiles a CTA."""
    check_forward([33, 0, 64, 9011, 31, 1, 1300], n, k, "gelu", gated, True, True, True, True, torch.bfloat16, expected, max_sms=20)


@pytest.mark.parametrize("counts", [[1], [16], [130], [300, 0, 5]], ids=lambda c: f"{len(c)}g{sum(c)}")
@pytest.mark.parametrize("n,k", [(16, 1024), (272, 2056), (1008, 1544), (256, 7168)])
@pytest.mark.parametrize("form", ["bf16", "gated", "fp32"])
@pytest.mark.parametrize("max_sms", [0, 5])
def test_contraction_in_parts(counts, n, k, form, max_sms):
    """Few tiles and a long contraction: parts of it meet in a workspace."""
    check_forward(counts, n, k, "silu" if form == "gated" else "gelu", form == "gated", True, True, True, form != "fp32",
                  torch.float32 if form == "fp32" else torch.bfloat16, 0, pad=8, gap=0, max_sms=max_sms)


def test_contraction_in_parts_repeats_and_is_optional():
    """The same bits call after call, captured and on a side stream; without a workspace it is not cut."""
    g = gen(40)
    rows, n, k = 70, 264, 4104
    x, w, res = randn(g, (rows, k)), randn(g, (1, n, k), k ** -0.5), randn(g, (rows, n))
    h, c = handle(1), i32([rows])
    want = ep.ep_grouped_gemm_act(h, x, w, c, residual=res, act="gelu")["out"]
    for _ in range(20):
        assert torch.equal(ep.ep_grouped_gemm_act(h, x, w, c, residual=res, act="gelu")["out"], want)
    place = res.clone()
    ep.ep_grouped_gemm_act(h, x, w, c, residual=place, act="gelu", out=place)
    assert torch.equal(place, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [ep.ep_grouped_gemm_act(h, x, w, c, residual=res, act="gelu")["out"] for _ in range(3)]
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(o, want) for o in outs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = ep.ep_grouped_gemm_act(h, x, w, c, residual=res, act="gelu", stream=side)["out"]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, want)
    L, st = ep.lib(), torch.cuda.current_stream().cuda_stream
    need = L.ep_grouped_gemm_act_workspace(h.ptr, rows, n, k, 0, 0)
    assert need > 0 and L.ep_grouped_gemm_act_workspace(h.ptr, 100000, 4096, k, 0, 0) == 0
    whole, ws = torch.empty_like(want), torch.empty(need, dtype=torch.uint8, device=DEV)
    args = [h.ptr, rows, n, k, c.data_ptr(), None, x.data_ptr(), 2 * k, w.data_ptr(), None, 3, 0, None, res.data_ptr(), 2 * n, None, 0,
            whole.data_ptr(), 0, 2 * n, 0]
    assert L.ep_grouped_gemm_act(*args, ws.data_ptr(), need - 1, st) == 1 and b"workspace" in L.ep_last_error()
    assert L.ep_grouped_gemm_act(*args, None, 0, st) == 0
    h.check()
    # where none is needed, what is given is not looked at
    short = [*args]
    short[3], short[7] = 512, 2 * k
    assert L.ep_grouped_gemm_act_workspace(h.ptr, rows, n, 512, 0, 0) == 0
    w_short, out_short = w[:, :, :512].contiguous(), torch.empty_like(want)
    short[8], short[17] = w_short.data_ptr(), out_short.data_ptr()
    assert L.ep_grouped_gemm_act(*short, ws.data_ptr(), 1, st) == 0
    h.check()
    # both are sums of the same products, each off by (k / 16 + 8) 2^-22 of unit magnitudes at most, and rounded
    assert ((whole.double() - want.double()).abs() <= 2 * 1.13 * (k / 16 + 8) * 2.0 ** -22 * 16 + 2.0 ** -7 * want.double().abs()).all()


def test_dense_product_in_place_and_side_stream():
    """One expert is a dense product; the residual may be the output itself."""
    g = gen(1)
    rows, n, k = 517, 264, 520
    x, w, res = randn(g, (rows, k)), randn(g, (1, n, k), 0.05), randn(g, (rows, n))
    h = handle(1)
    c = i32([rows])
    want = ep.ep_grouped_gemm_act(h, x, w, c, residual=res, act="relu")["out"]
    stream = res.clone()
    ep.ep_grouped_gemm_act(h, x, w, c, residual=stream, act="relu", out=stream)
    assert torch.equal(stream, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = ep.ep_grouped_gemm_act(h, x, w, c, residual=res, act="relu", stream=side)["out"]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, want)
    assert ep.ep_grouped_gemm_act(h, x[:0], w, i32([0]), residual=res[:0])["out"].shape == (0, n)
    h.check()


def test_plain_form_gives_the_plain_products_bits():
    """Nothing in the epilogue: ep_grouped_gemm."""
    counts = [300, 0, 45, 129]
    begin, rows = packed(counts)
    g = gen(2)
    x, w = randn(g, (rows, 328)), randn(g, (4, 272, 328), 0.1)
    h = handle(4)
    c, b = i32(counts), i32(begin)
    for expected in (1, 100000):
        assert torch.equal(ep.ep_grouped_gemm_act(h, x, w, c, b, expected_rows=expected)["out"],
                           ep.ep_grouped_gemm(h, x, w, c, b, expected_rows=expected))
    h.check()


def test_message_buffers():
    """Rows without begins (low-latency messages of bf16, in place), outputs in their shape."""
    R, EL, cap, k, n = 2, 2, 40, 72, 144
    g = gen(6)
    msgs = torch.zeros((R, EL, cap, 16 + 2 * k), dtype=torch.uint8, device=DEV)
    x = randn(g, (R, EL, cap, k))
    msgs[..., 16:] = x.view(torch.uint8)
    w = randn(g, (4, n, k), 0.1)
    count = i32([[5, 0], [40, 1]])
    h = handle(4, R)
    view = msgs[..., 16:].view(torch.bfloat16)
    out = torch.full((R, EL, cap, n // 2), 3.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_grouped_gemm_act(h, view, w, count, act="silu", gated=True, out=out, expected_rows=5)
    h.check()
    for e, c in enumerate(count.flatten().tolist()):
        v = x[e // EL, e % EL, :c].double() @ w[e].double().t()
        want = act64(v[:, :n // 2], "silu")[0] * v[:, n // 2:]
        # 72 products of magnitudes up to a few units: 2^-7 covers the rounding and 2^-17 of sums of magnitude 10
        within(out[e // EL, e % EL, :c], want, 2.0 ** -8 * want.abs() + 2.0 ** -13)
        assert (out[e // EL, e % EL, c:] == 3).all()


def test_special_values_stay_in_their_rows():
    counts, n, k = [130, 66], 144, 136
    begin, rows = packed(counts)
    g = gen(12)
    x, w = randn(g, (rows, k)), randn(g, (2, n, k), 0.1)
    bias, weights, res = torch.randn((2, n), generator=g, device=DEV), torch.rand(rows, generator=g, device=DEV), randn(g, (rows, n // 2))
    h = handle(2)
    c, b = i32(counts), i32(begin)

    def run(x, weights, res):
        return ep.ep_grouped_gemm_act(h, x, w, c, b, bias=bias, act="gelu", gated=True, row_weights=weights, residual=res)["out"]

    clean = run(x, weights, res)
    x2, w2, r2 = x.clone(), weights.clone(), res.clone()
    x2[129, 5], w2[130], r2[131, 3] = float("nan"), float("nan"), float("nan")
    out = run(x2, w2, r2)
    assert torch.equal(out[:129], clean[:129]) and torch.equal(out[132:], clean[132:])
    assert out[129:131].isnan().all() and out[131].isnan().sum() == 1
    h.check()


@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(act):
    """The activation at every exponent: x = 1 and weights that are the argument."""
    v = torch.cat([torch.linspace(-12, 12, 4000), torch.logspace(-30, 4, 1000), -torch.logspace(-30, 4, 1000), torch.zeros(8)]).to(torch.bfloat16)
    n = v.numel()
    w = torch.zeros((1, n, 8), dtype=torch.bfloat16)
    w[0, :, 0] = v
    x = torch.zeros((1, 8), dtype=torch.bfloat16)
    x[0, 0] = 1
    h = handle(1)
    out = ep.ep_grouped_gemm_act(h, x.to(DEV), w.to(DEV), i32([1]), act=act, out_dtype=torch.float32)["out"][0]
    h.check()
    want, _ = act64(v.double().to(DEV), act)
    # below -88 exp(-v) and below -13 erfc pass what 32 bits hold: absolute
    assert ((out.double() - want).abs() <= 2.0 ** -18 * want.abs() + 1e-35).all()


GRADS = [(False, True), (True, True), (True, False), (False, False)]


@pytest.mark.parametrize("n", [16, 272, 1040])
@pytest.mark.parametrize("counts", COUNTS + [[3000, 1, 0, 700]], ids=lambda c: f"{len(c)}g{sum(c)}")
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("weighted,with_bias", GRADS)
def test_gradient(counts, n, act, gated, weighted, with_bias):
    E, width = len(counts), n // 2 if gated else n
    begin, rows = packed(counts, gap=1)
    g = gen(n)
    dy = torch.full((rows, width), float("nan"), dtype=torch.bfloat16, device=DEV)
    v = torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    for b, c in zip(begin, counts):
        dy[b:b + c], v[b:b + c] = randn(g, (c, width)), randn(g, (c, n), 2)
    weights = torch.rand(rows, generator=g, device=DEV) if weighted else None
    d_pre, d_w, d_b = Guarded((rows, n), torch.bfloat16), Guarded((rows,), torch.float32), Guarded((E, n), torch.float32)
    h = handle(E)
    ep.ep_act_grad(h, dy, v, i32(counts), i32(begin), act=act, gated=gated, row_weights=weights, d_pre=d_pre.t,
                   d_row_weights=d_w.t if weighted else None, d_bias=d_b.t if with_bias else None)
    h.check()
    for o in (d_pre, d_w, d_b):
        o.check()
    used = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for e, (b, c) in enumerate(zip(begin, counts)):
        used[b:b + c] = True
        vd, yd = v[b:b + c].double(), dy[b:b + c].double()
        p = weights[b:b + c].double()[:, None] if weighted else 1.0
        a, slope = act64(vd[:, :width], act)
        # magnitudes of the terms: a derivative of silu or gelu is a sum of two terms that may cancel
        if gated:
            up = vd[:, width:]
            want, mag = torch.cat([yd * p * up * slope, yd * p * a], 1), torch.cat([(yd * p * up).abs() * (slope.abs() + 1), (yd * p * a).abs()], 1)
            dw = yd * a * up
        else:
            want, mag = yd * p * slope, (yd * p).abs() * (slope.abs() + 1)
            dw = yd * a
        within(d_pre.t[b:b + c], want, 2.0 ** -18 * mag + 2.0 ** -8 * want.abs() + 1e-37)
        if weighted:
            within(d_w.t[b:b + c], dw.sum(1), (2.0 ** -18 + width * 2.0 ** -24) * dw.abs().sum(1) + 1e-37)
        if with_bias:
            within(d_b.t[e], want.sum(0), 2.0 ** -18 * mag.sum(0) + c * 2.0 ** -24 * want.abs().sum(0) + 1e-37)
    assert (d_pre.t[~used].view(torch.uint8) == d_pre.fill).all()
    if weighted:
        assert (d_w.t[~used].view(torch.uint8) == d_w.fill).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
def test_gradient_against_differences(act, gated):
    g = gen(21)
    rows, n = 40, 64
    width = n // 2 if gated else n
    v, dy, weights = randn(g, (rows, n)), randn(g, (rows, width)), torch.rand(rows, generator=g, device=DEV)
    h = handle(2)
    c, b = i32([25, 15]), i32([0, 25])
    r = ep.ep_act_grad(h, dy, v, c, b, act=act, gated=gated, row_weights=weights, with_bias=True)
    h.check()
    dv, dw = randn(g, (rows, n)).double(), torch.randn(rows, generator=g, device=DEV).double()
    db = torch.randn((2, n), generator=g, device=DEV).double()

    def f(s):
        x = v.double() + s * (dv + torch.cat([db[:1].expand(25, n), db[1:].expand(15, n)]))
        a, _ = act64(x[:, :width], act)
        y = (a * x[:, width:] if gated else a) * (weights.double() + s * dw)[:, None]
        return (y * dy.double()).sum()

    step = 2.0 ** -12  # off by step^2 / 6 of third derivatives of order 10: 1e-7 a term
    slope = (f(step) - f(-step)) / (2 * step)
    parts = [(r["d_pre"].double() * dv), (r["d_row_weights"].double() * dw), (r["d_bias"].double() * db)]
    assert abs(sum(p.sum() for p in parts) - slope) <= sum(2.0 ** -8 * p.abs().sum() for p in parts) + 1e-6 * rows * n


def test_gradient_without_activation_and_repeats():
    """Only the bias's gradient of a plain product: no kept values; the same bits call after call, under an SM cap too."""
    g = gen(4)
    counts = [1000, 0, 77, 3]
    begin, rows = packed(counts)
    dy = randn(g, (rows, 200))
    c, b = i32(counts), i32(begin)
    h = handle(4)
    first = ep.ep_act_grad(h, dy, None, c, b, with_bias=True)
    assert torch.equal(first["d_pre"], dy) and first["d_row_weights"] is None
    for other in (h, handle(4, max_sms=2)):
        assert torch.equal(ep.ep_act_grad(other, dy, None, c, b, with_bias=True)["d_bias"], first["d_bias"])
    v = randn(g, (rows, 200))
    want = ep.ep_act_grad(h, dy, v, c, b, act="silu")["d_pre"]
    place = v.clone()
    assert torch.equal(ep.ep_act_grad(h, dy, place, c, b, act="silu", d_pre=place)["d_pre"], want)
    empty = ep.ep_act_grad(h, dy[:0], v[:0], i32([0] * 4), i32([0] * 4), act="silu", with_bias=True)
    assert (empty["d_bias"] == 0).all()
    h.check()


@pytest.mark.parametrize("counts,begin,rows", [([100] * 8, [0] * 8, 100), ([3, 2], [0, 2], 4)])
def test_more_rows_than_there_are_write_nothing(counts, begin, rows):
    E, n, k = len(counts), 64, 64
    h = handle(E)
    c, b = i32(counts), i32(begin)
    zero = torch.zeros((rows, k), dtype=torch.bfloat16, device=DEV)
    out, pre, d_b = Guarded((rows, n // 2), torch.bfloat16), Guarded((rows, n), torch.bfloat16), Guarded((E, n), torch.float32)
    ep.ep_grouped_gemm_act(h, zero, torch.zeros((E, n, k), dtype=torch.bfloat16, device=DEV), c, b, gated=True, out=out.t, pre=pre.t)
    assert h.status() == 2
    ep.ep_act_grad(h, zero[:, :n // 2], zero[:, :n].contiguous(), c, b, gated=True, d_pre=pre.t, d_bias=d_b.t)
    assert h.status() == 2
    for o in (out, pre, d_b):
        o.check()
        assert (o.t.contiguous().view(torch.uint8) == o.fill).all()


@pytest.mark.parametrize("counts,begin,rows", [([4, 100], [0, 4], 60), ([4, 5], [-1, 4], 64)])
def test_groups_that_do_not_fit_are_reported_and_clamped(counts, begin, rows):
    g = gen(4)
    x, w = randn(g, (rows, 64)), randn(g, (2, 64, 64))
    out = Guarded((rows, 64), torch.bfloat16)
    h = handle(2)
    ep.ep_grouped_gemm_act(h, x, w, i32(counts), i32(begin), act="relu", out=out.t)
    assert h.status() == 2
    out.check()
    d = Guarded((rows, 64), torch.bfloat16)
    ep.ep_act_grad(h, x, x, i32(counts), i32(begin), act="relu", d_pre=d.t, with_bias=True)
    assert h.status() == 2
    d.check()


def test_refusals():
    h = handle(2)
    c = i32([4, 4])
    x, w = torch.zeros((8, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 64, 64), dtype=torch.bfloat16, device=DEV)
    odd = torch.zeros((8, 66), dtype=torch.bfloat16, device=DEV)[:, :64]
    bad = [dict(act="tanh"), dict(gated=True, out_dtype=torch.float32), dict(bias=torch.zeros((2, 63), device=DEV)),
           dict(row_weights=torch.zeros(7, device=DEV)), dict(residual=x[:7]), dict(residual=odd), dict(out=odd), dict(pre=odd),
           dict(expected_rows=-1)]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, ep.EPError)):
            ep.ep_grouped_gemm_act(h, x, w, c, i32([0, 4]), **kw)
    with pytest.raises(ep.EPError):
        ep.ep_grouped_gemm_act(h, odd, w, c, i32([0, 4]))       # rows that are not 16 bytes apart
    with pytest.raises(ep.EPError):
        ep.ep_grouped_gemm_act(h, x, w[:, :56].contiguous(), c, i32([0, 4]), gated=True)  # 28 gates
    for kw in (dict(act="silu"), dict(gated=True), dict(d_row_weights=torch.zeros(8, device=DEV))):
        with pytest.raises(ep.EPError):
            ep.ep_act_grad(h, x, None, c, i32([0, 4]), **kw)     # needs the kept values
    with pytest.raises((ValueError, ep.EPError)):
        ep.ep_act_grad(h, x, x[:, :56], c, i32([0, 4]), act="silu")
    L, st = ep.lib(), torch.cuda.current_stream().cuda_stream
    d_b = torch.zeros((2, 64), device=DEV)
    need = L.ep_act_grad_workspace(h.ptr, 8, 64)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    args = [h.ptr, 8, 64, c.data_ptr(), None, x.data_ptr(), 128, x.data_ptr(), 128, 0, 0, None, None, 0, None, d_b.data_ptr()]
    assert L.ep_act_grad(*args, ws.data_ptr(), need - 1, st) == 1 and b"workspace" in L.ep_last_error()
    assert L.ep_act_grad(*args, None, need, st) == 1
    assert L.ep_act_grad(*args, ws.data_ptr(), need, st) == 0
    h.check()


def test_captured_training_step():
    """Forward and backward of an expert's products in one graph, replayed on new rows."""
    g = gen(30)
    counts = [70, 0, 33, 129]
    begin, rows = packed(counts)
    H, I = 136, 72
    h = handle(4)
    c, b = i32(counts), i32(begin)
    x, dy = randn(g, (rows, H)), randn(g, (rows, H))
    up, down = randn(g, (4, 2 * I, H), 0.1), randn(g, (4, H, I), 0.1)
    bias = torch.randn((4, 2 * I), generator=g, device=DEV) * 0.1

    def step():
        f = ep.ep_grouped_gemm_act(h, x, up, c, b, bias=bias, act="silu", gated=True, keep_pre=True)
        y = ep.ep_grouped_gemm_act(h, f["out"], down, c, b, residual=x)["out"]
        da = ep.ep_grouped_gemm(h, dy, down, c, b, w_transposed=True)
        r = ep.ep_act_grad(h, da, f["pre"], c, b, act="silu", gated=True, with_bias=True)
        return [y, r["d_bias"], ep.ep_grouped_gemm_wgrad(h, r["d_pre"], x, c, b), ep.ep_grouped_gemm(h, r["d_pre"], up, c, b, w_transposed=True)]

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(2):
        x.copy_(randn(g, (rows, H)))
        dy.copy_(randn(g, (rows, H)))
        graph.replay()
        for a, e in zip(outs, step()):
            assert torch.equal(a, e)
    h.check()
