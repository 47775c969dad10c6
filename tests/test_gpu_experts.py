"""The expert products against plain 64-bit forms: ragged groups, odd sizes, strides, in-place messages, gradients.

Tolerances, fixed before the first run.  A product of bf16 (or e4m3) values is exact in fp32; adding m of them in
fp32, in any order and even cut off instead of rounded, is off by at most m * 2^-23 of the sum of magnitudes per
addition kept, and one rounding to bf16 (8 significant bits) by 2^-8 of the result.  With 16 products added per step of the tensor
cores the sum's part is taken as (m / 16 + 8) * 2^-22 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from combine_get_dispatch_03_gb300 import ep
from _parity import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"


def handle(E, R=1, hidden=512, tokens=64, K=1, cap=0, alignment=1, max_sms=0):
    return ep.Handle(ep.Config(num_ranks=R, num_max_tokens=tokens, hidden=hidden, num_experts=E, num_topk=K,
                               recv_capacity=cap, expert_alignment=alignment, max_sms=max_sms))


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def packed(counts, gap=0, order=None):
    """Begins of groups laid out one after another (in `order`), `gap` rows apart; and the rows in all."""
    begin, at = [0] * len(counts), gap
    for e in (order if order is not None else range(len(counts))):
        begin[e] = at
        at += counts[e] + gap
    return begin, at


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def close(got, want, magnitude, m, out_eps=2.0 ** -8):
    """got against want (64 bits) with the tolerance of the file's head."""
    got, want = got.double(), want.double()
    tol = out_eps * want.abs() + (m / 16 + 8) * 2.0 ** -22 * magnitude * (1 + out_eps) + 1e-37
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((got - want).abs() / tol).max())} x the tolerance"


COUNTS = [
    [1],
    [5, 0, 1, 0],
    [0, 0, 0],
    [128, 127, 129, 31, 32, 33, 0, 64],
    [257, 0, 300, 1],
    [0] * 61 + [2, 0, 515],
]


@pytest.mark.parametrize("n,k", [(8, 8), (64, 64), (72, 136), (1000, 72), (264, 1032), (520, 2048)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}g{sum(c)}")
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("expected", [1, 100000], ids=["single", "pair"])  # both tile heights on every shape
def test_grouped_gemm(counts, n, k, transposed, expected):
    E = len(counts)
    begin, rows = packed(counts, gap=3)
    g = gen(n * 31 + k)
    x = torch.full((rows, k), float("nan"), dtype=torch.bfloat16, device=DEV)  # rows of no group hold NaN
    for b, c in zip(begin, counts):
        x[b:b + c] = randn(g, (c, k))
    w = randn(g, (E, k, n) if transposed else (E, n, k), 0.1)
    out = Guarded((rows, n), torch.bfloat16)
    h = handle(E)
    ep.ep_grouped_gemm(h, x, w, i32(counts), i32(begin), w_transposed=transposed, out=out.t, expected_rows=expected)
    h.check()
    out.check()
    raw = out.t.view(torch.uint8)
    used = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for e, (b, c) in enumerate(zip(begin, counts)):
        used[b:b + c] = True
        we = w[e].double() if transposed else w[e].double().t()
        xe = x[b:b + c].double()
        close(out.t[b:b + c], xe @ we, xe.abs() @ we.abs(), k)
    assert (raw[~used] == out.fill).all(), "a row outside every group was written"


@pytest.mark.parametrize("n,k", [(8, 8), (64, 64), (72, 136), (1000, 72), (136, 1032)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}g{sum(c)}")
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weight_gradient(counts, n, k, dtype):
    E = len(counts)
    begin, rows = packed(counts, gap=2)
    g = gen(n * 17 + k)
    x = torch.full((rows, k), float("inf"), dtype=torch.bfloat16, device=DEV)
    dy = torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    for b, c in zip(begin, counts):
        x[b:b + c], dy[b:b + c] = randn(g, (c, k)), randn(g, (c, n))
    out = Guarded((E, n, k), dtype)
    h = handle(E)
    ep.ep_grouped_gemm_wgrad(h, dy, x, i32(counts), i32(begin), out=out.t)
    h.check()
    out.check()
    for e, (b, c) in enumerate(zip(begin, counts)):
        ye, xe = dy[b:b + c].double(), x[b:b + c].double()
        if c == 0:
            assert (out.t[e] == 0).all(), "an expert without rows has a zero gradient"
        close(out.t[e], ye.t() @ xe, ye.abs().t() @ xe.abs(), c, 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8)


def test_weight_gradient_accumulates():
    counts = [70, 0, 9]
    begin, rows = packed(counts)
    g = gen(5)
    x, dy = randn(g, (rows, 200)), randn(g, (rows, 72))
    h = handle(3)
    once = ep.ep_grouped_gemm_wgrad(h, dy, x, i32(counts), i32(begin))
    start = torch.randn((3, 72, 200), generator=g, device=DEV)
    more = start.clone()
    ep.ep_grouped_gemm_wgrad(h, dy, x, i32(counts), i32(begin), out=more, accumulate=True)
    h.check()
    assert torch.equal(more, start + once)


@pytest.mark.parametrize("n,k", [(8, 8), (72, 136), (264, 1032)])
@pytest.mark.parametrize("counts", [[1], [5, 0, 1, 0], [128, 127, 129, 31], [900, 1100], [2000, 0, 1]], ids=lambda c: f"{len(c)}g{sum(c)}")
def test_weight_gradient_added_and_of_many_rows(counts, n, k):
    """Few and many rows an expert, written and added: the same sums, nothing beside them."""
    E = len(counts)
    begin, rows = packed(counts)
    g = gen(n + k)
    x, dy = randn(g, (rows, k)), randn(g, (rows, n))
    once, more = Guarded((E, n, k), torch.float32), Guarded((E, n, k), torch.float32)
    start = torch.randn((E, n, k), generator=g, device=DEV)
    more.t.copy_(start)
    h = handle(E)
    for out, accumulate in ((once, False), (more, True), (more, True)):
        ep.ep_grouped_gemm_wgrad(h, dy, x, i32(counts), i32(begin), out=out.t, accumulate=accumulate)
        h.check()
        out.check()
    for e, (b, c) in enumerate(zip(begin, counts)):
        ye, xe = dy[b:b + c].double(), x[b:b + c].double()
        close(once.t[e], ye.t() @ xe, ye.abs().t() @ xe.abs(), c, 2.0 ** -24)
    assert torch.equal(more.t, start + once.t + once.t)


def test_weight_gradient_added_to_special_values():
    g = gen(9)
    x, dy = randn(g, (50, 64)), randn(g, (50, 32))
    h = handle(2)
    c, b = i32([50, 0]), i32([0, 50])
    once = ep.ep_grouped_gemm_wgrad(h, dy, x, c, b)
    start = torch.zeros((2, 32, 64), device=DEV)
    start[:, 0, 0], start[:, 5, 3], start[:, 31, 63], start[:, 1, :] = float("inf"), float("nan"), float("-inf"), 3e38
    more = start.clone()
    ep.ep_grouped_gemm_wgrad(h, dy, x, c, b, out=more, accumulate=True)
    h.check()
    assert torch.equal(more.isnan(), (start + once).isnan())
    assert torch.equal(more.nan_to_num(nan=0.5), (start + once).nan_to_num(nan=0.5))


def test_products_are_each_others_gradients():
    """sum(dy * forward(x)) changes with x and w as the two gradients say (differences along a direction)."""
    counts = [40, 0, 133, 7]
    begin, rows = packed(counts)
    g = gen(9)
    n, k = 136, 264
    x, w, dy = randn(g, (rows, k)), randn(g, (4, n, k), 0.1), randn(g, (rows, n))
    h = handle(4)
    c, b = i32(counts), i32(begin)
    dx = ep.ep_grouped_gemm(h, dy, w, c, b, w_transposed=True).double()
    dw = ep.ep_grouped_gemm_wgrad(h, dy, x, c, b).double()
    h.check()

    def f(xx, ww):
        y = torch.cat([xx[i:i + m].double() @ ww[e].double().t() for e, (i, m) in enumerate(zip(begin, counts))])
        return (dy.double() * y).sum()

    vx, vw = randn(g, (rows, k)).double(), randn(g, (4, n, k)).double()
    step = 2.0 ** -10  # f is linear in each argument: the difference is exact up to 64-bit rounding
    ax = (f(x.double() + step * vx, w) - f(x.double() - step * vx, w)) / (2 * step)
    aw = (f(x, w.double() + step * vw) - f(x, w.double() - step * vw)) / (2 * step)
    # dx is rounded to bf16: off by at most 2^-8 of every term (the sum of magnitudes bounds it)
    assert abs((dx * vx).sum() - ax) <= 2.0 ** -8 * (dx * vx).abs().sum()
    assert abs((dw * vw).sum() - aw) <= 2.0 ** -16 * (dw * vw).abs().sum()


def codes(g, shape):
    return (torch.randn(shape, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)


def fp8_reference(x, xs, w, ws):
    """(result, sum of magnitudes) of one expert, in 64 bits."""
    n, k = w.shape
    xd = x.double() * xs.double().repeat_interleave(128, 1)
    wd = w.double() * ws.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    return xd @ wd.t(), xd.abs() @ wd.abs().t()


@pytest.mark.parametrize("n,k", [(8, 128), (64, 256), (72, 384), (1000, 512), (264, 1152), (520, 2048)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}g{sum(c)}")
@pytest.mark.parametrize("expected", [1, 100000], ids=["single", "pair"])
def test_grouped_gemm_fp8(counts, n, k, expected):
    E = len(counts)
    begin, rows = packed(counts, gap=1, order=list(reversed(range(E))))
    g = gen(n * 13 + k)
    x = torch.full((rows, k), 0x7f, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # NaN codes
    xs = torch.full((rows, k // 128), float("nan"), device=DEV)
    for b, c in zip(begin, counts):
        x.view(torch.uint8)[b:b + c] = codes(g, (c, k)).view(torch.uint8)
        xs[b:b + c] = torch.rand((c, k // 128), generator=g, device=DEV) + 0.01
    w = codes(g, (E, n, k))
    ws = torch.rand((E, -(-n // 128), k // 128), generator=g, device=DEV) * 0.01
    out = Guarded((rows, n), torch.bfloat16)
    h = handle(E)
    ep.ep_grouped_gemm_fp8(h, x, xs, w, ws, i32(counts), i32(begin), out=out.t, expected_rows=expected)
    h.check()
    out.check()
    used = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for e, (b, c) in enumerate(zip(begin, counts)):
        used[b:b + c] = True
        want, magnitude = fp8_reference(x[b:b + c], xs[b:b + c], w[e], ws[e])
        close(out.t[b:b + c], want, magnitude, k)
    assert (out.t.view(torch.uint8)[~used] == out.fill).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_round", "fp8_ue8m0"])
def test_low_latency_messages_in_place(fmt):
    """LL dispatch -> product straight from the message buffer, against the buffer's own contents."""
    R, EL, T, K, H, n = 4, 3, 19, 3, 512, 200
    E = R * EL
    g = gen(77)
    h = handle(E, R, H, 24, K)
    x = randn(g, (R, T, H))
    idx = torch.stack([torch.randperm(E - 1, generator=torch.Generator().manual_seed(i))[:K] for i in range(R * T)])
    idx = idx.view(R, T, K).to(DEV)  # the last expert gets nothing
    fp8 = fmt != "bf16"
    d = ep.ep_ll_dispatch(h, x, idx, use_fp8=fp8, round_scale=fmt == "fp8_round", use_ue8m0=fmt == "fp8_ue8m0")
    px, scales, _ = ep.ll_views(d["recv_msgs"], H, fp8)
    cnt = d["packed_recv_count"]
    rows = R * 24
    out = torch.full((R, EL, rows, n), 7.0, dtype=torch.bfloat16, device=DEV)
    if not fp8:
        w = randn(g, (E, n, H), 0.1)
        ep.ep_grouped_gemm(h, px, w, cnt, out=out, expected_rows=R * T * K // E)
    else:
        w, ws = codes(g, (E, n, H)), torch.rand((E, 2, H // 128), generator=g, device=DEV) * 0.01
        s = scales if fmt == "fp8_ue8m0" else scales.view(torch.float32)
        ep.ep_grouped_gemm_fp8(h, px, s, w, ws, cnt, out=out)
    h.check()
    counts = cnt.view(-1).tolist()
    assert counts[-1] == 0 and sum(counts) == R * T * K
    for e, c in enumerate(counts):
        r, j = divmod(e, EL)
        if fp8:
            xs = torch.exp2(scales[r, j, :c, :H // 128].double() - 127) if fmt == "fp8_ue8m0" \
                else scales.view(torch.float32)[r, j, :c]
            want, magnitude = fp8_reference(px[r, j, :c], xs, w[e], ws[e])
        else:
            xe, we = px[r, j, :c].double(), w[e].double().t()
            want, magnitude = xe @ we, xe.abs() @ we.abs()
        close(out[r, j, :c], want, magnitude, H)
        assert (out[r, j, c:] == 7.0).all()


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}g{sum(c)}")
@pytest.mark.parametrize("expected", [1, 100000], ids=["few", "many"])
@pytest.mark.parametrize("n,k,pad,offset", [(72, 136, 2, 0), (520, 1032, 8, 2), (264, 72, 6, 6)])
def test_rows_four_bytes_apart(counts, expected, n, k, pad, offset):
    """Rows that are not 16 bytes apart, or do not begin at 16 bytes: the bits of the aligned call, both orientations."""
    begin, rows = packed(counts, gap=1)
    g = gen(k + pad)
    flat = randn(g, (rows * (k + pad) + offset,))
    x = flat[offset:].view(rows, k + pad)[:, :k]
    h = handle(len(counts))
    c, b = i32(counts), i32(begin)
    for transposed in (False, True):
        w = randn(g, (len(counts), k, n) if transposed else (len(counts), n, k), 0.1)
        want, out = (torch.full((rows, n), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        ep.ep_grouped_gemm(h, x.contiguous(), w, c, b, w_transposed=transposed, out=want, expected_rows=expected)
        ep.ep_grouped_gemm(h, x, w, c, b, w_transposed=transposed, out=out, expected_rows=expected)
        assert torch.equal(out, want)
    h.check()


@pytest.mark.parametrize("expected", [40, 300, 100000])  # single CTAs, pairs in bf16, pairs in both
@pytest.mark.parametrize("n,pad", [(8, 0), (72, 8), (136, 24), (264, 0), (200, 56)])
@pytest.mark.parametrize("form", ["forward", "transposed", "fp8"])
def test_many_tiles_a_cta(expected, n, pad, form):
    """Whole and ragged blocks of rows in turn, several tiles a CTA, rows of the result apart: against 64 bits, nothing
    written beside the result, and the bits of the call that expects few rows."""
    counts, k = [33, 0, 64, 30011, 31, 1, 1300], 256
    E = len(counts)
    begin, rows = packed(counts, gap=2)
    g = gen(n + expected)
    h = handle(E)
    c, b = i32(counts), i32(begin)
    if form == "fp8":
        x, w = codes(g, (rows, k)), codes(g, (E, n, k))
        xs = torch.rand((rows, k // 128), generator=g, device=DEV) + 0.01
        ws = torch.rand((E, -(-n // 128), k // 128), generator=g, device=DEV) * 0.01
    else:
        x, w = randn(g, (rows, k)), randn(g, (E, k, n) if form == "transposed" else (E, n, k), 0.1)

    def run(expect):
        out = Guarded((rows, n + pad), torch.bfloat16)
        if form == "fp8":
            ep.ep_grouped_gemm_fp8(h, x, xs, w, ws, c, b, out=out.t[:, :n], expected_rows=expect)
        else:
            ep.ep_grouped_gemm(h, x, w, c, b, w_transposed=form == "transposed", out=out.t[:, :n], expected_rows=expect)
        h.check()
        out.check()
        assert (out.t[:, n:].contiguous().view(torch.uint8) == out.fill).all()
        return out
    out = run(expected)
    used = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for e, (at, m) in enumerate(zip(begin, counts)):
        used[at:at + m] = True
        if form == "fp8":
            want, magnitude = fp8_reference(x[at:at + m], xs[at:at + m], w[e], ws[e])
        else:
            we, xe = w[e].double() if form == "transposed" else w[e].double().t(), x[at:at + m].double()
            want, magnitude = xe @ we, xe.abs() @ we.abs()
        close(out.t[at:at + m, :n], want, magnitude, k)
    assert (out.t[~used].view(torch.uint8) == out.fill).all(), "a row outside every group was written"
    assert torch.equal(run(1).t.view(torch.int16), out.t.view(torch.int16))


@pytest.mark.parametrize("k", [128, 384, 2944])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_fp8_messages_of_any_hidden_size(k, ue8m0):
    """Message buffers whose size is no multiple of 16 bytes, read in place."""
    R, EL, rows, n, G = 2, 3, 140, 136, k // 128
    g = gen(k)
    msgs = torch.zeros((R, EL, rows, 16 + k + 4 * G), dtype=torch.uint8, device=DEV)
    msgs[..., 16:16 + k] = codes(g, (R, EL, rows, k)).view(torch.uint8)
    if ue8m0:
        msgs[..., 16 + k:16 + k + G] = torch.randint(117, 130, (R, EL, rows, G), generator=g, device=DEV).to(torch.uint8)
    else:
        msgs[..., 16 + k:] = (torch.rand((R, EL, rows, G), generator=g, device=DEV) + 0.1).view(torch.uint8)
    px, scales, _ = ep.ll_views(msgs, k, True)
    counts = [140, 0, 1, 129, 33, 64]
    w, ws = codes(g, (6, n, k)), torch.rand((6, 2, G), generator=g, device=DEV) * 0.01
    s = scales if ue8m0 else scales.view(torch.float32)
    h = handle(6, R)
    out = ep.ep_grouped_gemm_fp8(h, px, s, w, ws, i32(counts))
    h.check()
    for e, c in enumerate(counts):
        r, j = divmod(e, EL)
        xs = torch.exp2(scales[r, j, :c, :G].double() - 127) if ue8m0 else s[r, j, :c]
        want, magnitude = fp8_reference(px[r, j, :c], xs, w[e], ws[e])
        close(out[r, j, :c], want, magnitude, k)


def test_strides_streams_and_repeats():
    """Strided rows in and out, a side stream, an SM cap: the same bits as the plain call, call after call."""
    counts = [3, 200, 0, 61]
    begin, rows = packed(counts)
    g = gen(3)
    k, n = 328, 144
    wide = randn(g, (rows, k + 24))
    x = wide[:, 8:8 + k]  # offset 16 bytes, stride k + 24
    w = randn(g, (4, n, k), 0.1)
    h = handle(4)
    c, b = i32(counts), i32(begin)
    want = ep.ep_grouped_gemm(h, x.contiguous(), w, c, b)
    out = torch.full((rows, n + 16), 5.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_grouped_gemm(h, x, w, c, b, out=out[:, 8:8 + n])
    assert torch.equal(out[:, 8:8 + n], want)
    assert (out[:, :8] == 5).all() and (out[:, 8 + n:] == 5).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [ep.ep_grouped_gemm(h, x, w, c, b) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, want) for a in again)
    small = handle(4, max_sms=3)
    assert torch.equal(ep.ep_grouped_gemm(small, x, w, c, b), want)
    h.check()
    small.check()


def test_special_values_stay_in_their_rows():
    """NaN and infinity in one row reach that row's outputs only; in the weight gradient that row's expert only."""
    counts, n, k = [130, 66], 72, 136
    begin, rows = packed(counts)
    g = gen(12)
    x, w = randn(g, (rows, k)), randn(g, (2, n, k), 0.1)
    h = handle(2)
    c, b = i32(counts), i32(begin)
    clean = ep.ep_grouped_gemm(h, x, w, c, b)
    x2 = x.clone()
    x2[129, 5], x2[130, 7] = float("nan"), float("inf")
    out = ep.ep_grouped_gemm(h, x2, w, c, b)
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[129:131] = False
    assert torch.equal(out[keep], clean[keep])
    assert out[129].isnan().all() and not out[130].isfinite().any()
    dy = randn(g, (rows, n))
    dw, dw2 = ep.ep_grouped_gemm_wgrad(h, dy, x, c, b), None
    x3 = x.clone()
    x3[129] = float("nan")  # the last row of expert 0, next to expert 1's first
    dw2 = ep.ep_grouped_gemm_wgrad(h, dy, x3, c, b)
    assert dw2[0].isnan().all() and torch.equal(dw2[1], dw[1])
    h.check()


@pytest.mark.parametrize("counts,begin,rows", [([4, 100], [0, 4], 60), ([4, 5], [0, 70], 64), ([4, -3], [0, 4], 64), ([4, 5], [-1, 4], 64)])
def test_groups_that_do_not_fit_are_reported_and_clamped(counts, begin, rows):
    g = gen(4)
    x, w = randn(g, (rows, 64)), randn(g, (2, 64, 64))
    out = Guarded((rows, 64), torch.bfloat16)
    h = handle(2)
    ep.ep_grouped_gemm(h, x, w, i32(counts), i32(begin), out=out.t)
    assert h.status() == 2
    out.check()
    good = [c if b >= 0 and c >= 0 and b + c <= rows else max(0, min(c, rows - b)) if b >= 0 else 0 for c, b in zip(counts, begin)]
    for e, (b, c) in enumerate(zip(begin, good)):
        if c:
            xe, we = x[b:b + c].double(), w[e].double().t()
            close(out.t[b:b + c], xe @ we, xe.abs() @ we.abs(), 64)
    ep.ep_grouped_gemm_wgrad(h, x, x, i32(counts), i32(begin))
    assert h.status() == 2


def test_many_experts_and_no_rows():
    E = 2048
    counts = [0] * E
    counts[0], counts[1033], counts[2047] = 2, 5, 1
    begin, rows = packed(counts)
    g = gen(8)
    x, w = randn(g, (rows, 64)), randn(g, (E, 16, 64))
    h = handle(E)
    out = ep.ep_grouped_gemm(h, x, w, i32(counts), i32(begin))
    for e in (0, 1033, 2047):
        b, c = begin[e], counts[e]
        xe, we = x[b:b + c].double(), w[e].double().t()
        close(out[b:b + c], xe @ we, xe.abs() @ we.abs(), 64)
    empty = ep.ep_grouped_gemm(h, x[:0], w, i32([0] * E), i32([0] * E))
    assert empty.shape == (0, 16)
    dw = ep.ep_grouped_gemm_wgrad(h, x[:0, :16], x[:0], i32([0] * E), i32([0] * E))
    assert dw.shape == (E, 16, 64) and (dw == 0).all()
    h.check()


# --------------------------------------------------------------------------------------------- gated activation

def swiglu_reference(x, width, weight):
    gate, up = x[:, :width].double(), x[:, width:].double()
    sig = 1 / (1 + torch.exp(-gate))
    p = weight.double()[:, None] if weight is not None else 1.0
    return gate, up, sig, p


# The hardware's exp and reciprocal are good to about 2^-21 each at |gate| < 16 (the argument's own rounding in
# exp grows with |gate|), the products add a few 2^-24: 2^-19 of the result; past |gate| = 16 the result of one
# side is below 2^-20 of the other inputs' scale and is held to an absolute 2^-30.
APPROX = 2.0 ** -19


@pytest.mark.parametrize("width", [8, 128, 136, 256, 512, 1032])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}g{sum(c)}")
@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu(counts, width, weighted):
    begin, rows = packed(counts, gap=1)
    g = gen(width)
    x = randn(g, (rows, 2 * width), 2.0)
    weight = torch.rand(rows, generator=g, device=DEV) if weighted else None
    out = Guarded((rows, width), torch.bfloat16)
    h = handle(len(counts))
    c, b = i32(counts), i32(begin)
    ep.ep_swiglu(h, x, c, b, row_weights=weight, out=out.t)
    h.check()
    out.check()
    gate, up, sig, p = swiglu_reference(x, width, weight)
    want = gate * sig * up * p
    used = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for bb, cc in zip(begin, counts):
        used[bb:bb + cc] = True
    tol = (2.0 ** -8 + APPROX) * want.abs() + 2.0 ** -30
    assert ((out.t.double() - want).abs() <= tol)[used].all()
    assert (out.t.view(torch.uint8)[~used] == out.fill).all()


@pytest.mark.parametrize("width", [128, 256, 384, 1024])
@pytest.mark.parametrize("round_scale", [False, True])
def test_swiglu_cast(width, round_scale):
    counts = [33, 0, 1, 100]
    begin, rows = packed(counts, gap=1)
    g = gen(width + 1)
    x = randn(g, (rows, 2 * width), 2.0)
    x[begin[2]] = 0  # a row of zeros takes the smallest scale
    weight = torch.rand(rows, generator=g, device=DEV)
    out, scales = Guarded((rows, width), torch.float8_e4m3fn), Guarded((rows, width // 128), torch.float32)
    h = handle(4)
    ep.ep_swiglu(h, x, i32(counts), i32(begin), row_weights=weight, cast_to_fp8=True, round_scale=round_scale,
                 out=out.t, out_scales=scales.t)
    h.check()
    out.check()
    scales.check()
    gate, up, sig, p = swiglu_reference(x, width, weight)
    v = (gate * sig * up * p).view(rows, -1, 128)
    scale = v.abs().amax(2).clamp_min(1e-4) / 448
    if round_scale:
        m, e = np.frexp(scale.cpu().numpy())  # log2 and pow of the device need not be exact at powers of two
        scale = torch.from_numpy(np.ldexp(1.0, np.where(m == 0.5, e - 1, e))).to(DEV)
    used = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for b, c in zip(begin, counts):
        used[b:b + c] = True
    got = scales.t.double()
    if round_scale:  # a power of two exactly, and the right one unless the maximum sits on a step within its error
        assert (torch.frexp(got)[0] == 0.5)[used].all()
        assert ((got == scale) | ((v.abs().amax(2) / 448 / got - 1).abs() < 2 * APPROX) |
                ((v.abs().amax(2) / 448 / got - 0.5).abs() < 2 * APPROX))[used].all()
    else:
        assert ((got - scale).abs() <= 2 * APPROX * scale)[used].all()
    # a code is the nearest e4m3 value: half a step of 2^-3 relative, or of 2^-9 near zero
    back = out.t.double().view(rows, -1, 128) * got[..., None]
    tol = (2.0 ** -4 + 2 * APPROX) * v.abs() + (2.0 ** -10 * (1 + APPROX)) * got[..., None] + 2.0 ** -30
    assert ((back - v).abs() <= tol)[used].all()
    assert (out.t.view(torch.uint8)[~used] == out.fill).all()


@pytest.mark.parametrize("width", [8, 128, 264, 1032])
@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu_gradient(width, weighted):
    counts = [33, 0, 1, 100]
    begin, rows = packed(counts, gap=1)
    g = gen(width + 2)
    x, dy = randn(g, (rows, 2 * width), 2.0), randn(g, (rows, width))
    weight = torch.rand(rows, generator=g, device=DEV) if weighted else None
    dx = Guarded((rows, 2 * width), torch.bfloat16)
    h = handle(4)
    r = ep.ep_swiglu_grad(h, dy, x, i32(counts), i32(begin), row_weights=weight, dx=dx.t)
    h.check()
    dx.check()
    gate, up, sig, p = swiglu_reference(x, width, weight)
    d = dy.double()
    slope = sig * (1 + gate * (1 - sig))
    want = torch.cat([d * p * up * slope, d * p * gate * sig], 1)
    # 1 - sig and 1 + gate * (1 - sig) cancel: their error is that of sig times |gate| + 1
    extra = torch.cat([(d * p * up * sig).abs() * (1 + gate.abs()), torch.zeros_like(d)], 1)
    used = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for b, c in zip(begin, counts):
        used[b:b + c] = True
    tol = (2.0 ** -8 + APPROX) * want.abs() + 2 * APPROX * extra + 2.0 ** -30
    assert ((dx.t.double() - want).abs() <= tol)[used].all()
    if weighted:
        terms = d * gate * sig * up
        err = (r["d_row_weights"].double() - terms.sum(1)).abs()
        assert (err <= (APPROX + width * 2.0 ** -24) * terms.abs().sum(1) + 2.0 ** -30)[used].all()
        # against differences in the row's weight: the output is linear in it
        step = (gate * sig * up * (p + 0.5) * d).sum(1) - (gate * sig * up * (p - 0.5) * d).sum(1)
        assert ((r["d_row_weights"].double() - step).abs() <= 2.0 ** -12 * terms.abs().sum(1) + 2.0 ** -30)[used].all()
    # against differences in x, along a direction
    v = randn(g, (rows, 2 * width)).double()
    eps = 2.0 ** -12

    def f(xx):
        gg, uu = xx[:, :width], xx[:, width:]
        return gg / (1 + torch.exp(-gg)) * uu * p * d

    slope_v = ((f(x.double() + eps * v) - f(x.double() - eps * v)) / (2 * eps)).sum(1)
    got = (dx.t.double() * v).sum(1)
    bound = (dx.t.double() * v).abs().sum(1) * 2.0 ** -7 + 2.0 ** -10
    assert ((got - slope_v).abs() <= bound)[used].all()


def test_swiglu_extreme_values():
    """Large gates saturate without NaN; NaN and infinity stay in their columns; -inf gates give NaN as in the formula."""
    g = torch.tensor([200.0, -200.0, 88.5, -88.5, 0.0, 3e38, -3e38, 1.0], device=DEV)
    x = torch.cat([g, torch.ones(8, device=DEV)])[None].to(torch.bfloat16)
    h = handle(1)
    out = ep.ep_swiglu(h, x, i32([1]), i32([0]))["out"].double()
    gd = x[0, :8].double()
    want = torch.where(gd > -100, gd / (1 + torch.exp(-gd)), torch.zeros_like(gd))
    assert ((out[0] - want).abs() <= 2.0 ** -8 * want.abs() + 1e-30).all()
    x2 = x.clone()
    x2[0, 1], x2[0, 11] = float("nan"), float("inf")
    bad = ep.ep_swiglu(h, x2, i32([1]), i32([0]))["out"][0]
    assert bad[1].isnan() and bad[3].isinf()
    keep = torch.tensor([0, 2, 4, 5, 6, 7], device=DEV)
    assert torch.equal(bad[keep].double(), out[0][keep])
    h.check()


# --------------------------------------------------------------------------------------------- expert order

def received(g, R, T, K, EL, cap, mask=0.0):
    """A dispatch's recv_topk_idx: random local experts, -1 elsewhere, rows past num_recv hold rubbish."""
    num = torch.randint(0, cap + 1, (R,), generator=torch.Generator().manual_seed(int(mask * 100) + R + K)).to(torch.int32)
    num[0] = cap
    if R > 1:
        num[1] = 0
    idx = torch.randint(-1, EL, (R, cap, K), generator=g, device=DEV)
    idx[torch.rand((R, cap, K), generator=g, device=DEV) < mask] = -1
    for r in range(R):
        idx[r, int(num[r]):] = 10 ** 12
    return idx, num


def layout_reference(idx, num, R, EL, K, alignment):
    idx, num = idx.cpu().numpy(), num.numpy()
    cap = idx.shape[1]
    count = [0] * (R * EL)
    where = []
    for r in range(R):
        for row in range(int(num[r])):
            for k in range(K):
                if idx[r, row, k] >= 0:
                    e = r * EL + int(idx[r, row, k])
                    where.append((r, row, k, e, count[e]))
                    count[e] += 1
    begin, at = [], 0
    for c in count:
        begin.append(at)
        at += -(-c // alignment) * alignment
    slot = torch.full((R, cap, K), -1, dtype=torch.int32)
    for r, row, k, e, i in where:
        slot[r, row, k] = begin[e] + i
    return count, begin, slot, at


LAYOUTS = [  # R, EL, K, cap, alignment, mask
    (1, 1, 1, 1, 1, 0.0),
    (2, 3, 2, 40, 1, 0.5),
    (4, 5, 3, 700, 8, 0.3),   # two chunks of slots per rank, the second one short
    (3, 1, 32, 65, 128, 0.0),
    (1, 2048, 4, 33, 1, 0.1),
    (32, 2, 2, 17, 4, 1.0),   # nothing to do at all
]


@pytest.mark.parametrize("R,EL,K,cap,alignment,mask", LAYOUTS)
def test_expert_layout(R, EL, K, cap, alignment, mask):
    g = gen(R * 100 + K)
    idx, num = received(g, R, cap, K, EL, cap, mask)
    count, begin, slot, rows = layout_reference(idx, num, R, EL, K, alignment)
    h = handle(R * EL, R, 64, max(cap, 1), K, cap, alignment)
    lay = ep.ep_expert_layout(h, idx, rows, num_recv=num.to(DEV))
    h.check()
    assert lay["group_count"].tolist() == count
    assert lay["group_begin"].tolist() == begin
    assert torch.equal(lay["slot_row"].cpu(), slot)
    if rows > 1 and sum(count):
        few = ep.ep_expert_layout(h, idx, rows // 2, num_recv=num.to(DEV))
        last = int(slot.max())
        assert h.status() == (2 if last >= rows // 2 else 0)
        assert torch.equal(few["slot_row"].cpu(), torch.where(slot < rows // 2, slot, -1))


def test_expert_layout_with_begins_past_every_row():
    """An alignment that pushes later experts' begins past 2^31: their slots have no row and the capacity is reported."""
    h = handle(4, 1, 64, 8, 1, 8, 2 ** 30)
    idx = torch.tensor([0, 1, 2, 3, 3, 2, 1, 0], dtype=torch.int64, device=DEV).view(1, 8, 1)
    lay = ep.ep_expert_layout(h, idx, 64, num_recv=i32([8]))
    assert h.status() == 2
    assert lay["group_count"].tolist() == [2, 2, 2, 2]
    assert lay["slot_row"].view(-1).tolist() == [0, -1, -1, -1, -1, -1, -1, 1]


def test_expert_layout_reports_bad_experts():
    h = handle(4, 2, 64, 8, 2, 8)
    idx = torch.zeros((2, 8, 2), dtype=torch.int64, device=DEV)
    idx[1, 3, 1] = 2
    lay = ep.ep_expert_layout(h, idx, 64, num_recv=i32([8, 8]))
    assert h.status() == 7
    assert int(lay["slot_row"][1, 3, 1]) == -1 and lay["group_count"].tolist() == [16, 0, 15, 0]


@pytest.mark.parametrize("R,EL,K,cap,alignment,mask", LAYOUTS)
@pytest.mark.parametrize("H,fp8", [(8, False), (264, False), (16392, False), (128, True), (1152, True)])
def test_expert_gather_and_reduce(R, EL, K, cap, alignment, mask, H, fp8):
    g = gen(R * 100 + H)
    idx, num = received(g, R, cap, K, EL, cap, mask)
    count, begin, slot, rows = layout_reference(idx, num, R, EL, K, alignment)
    rows = max(rows, 1)
    h = handle(R * EL, R, H, max(cap, 1), K, cap, alignment)
    num_d, slot_d = num.to(DEV), slot.to(DEV)
    x = codes(g, (R, cap, H)) if fp8 else randn(g, (R, cap, H))
    xs = torch.rand((R, cap, H // 128), generator=g, device=DEV) if fp8 else None
    tw = torch.rand((R, cap, K), generator=g, device=DEV)
    out = Guarded((rows, H), x.dtype)
    got = ep.ep_expert_gather(h, x, slot_d, rows, num_recv=num_d, x_scales=xs, topk_weights=tw, out=out.t)
    h.check()
    out.check()
    there = torch.nonzero(slot_d.view(-1) >= 0).view(-1)
    at = slot_d.view(-1)[there].long()
    source = there // K
    raw, xr = out.t.view(torch.uint8), x.view(R * cap, H).view(torch.uint8)
    assert torch.equal(raw[at], xr[source])
    assert torch.equal(got["row_weights"][at], tw.view(-1)[there])
    if fp8:
        assert torch.equal(got["out_scales"][at], xs.view(R * cap, -1)[source])
    untouched = torch.ones(rows, dtype=torch.bool, device=DEV)
    untouched[at] = False
    assert (raw[untouched] == out.fill).all()
    if fp8:
        return
    wide = randn(g, (rows, H + 8))
    y = wide[:, :H]
    rw = torch.randn(rows, generator=g, device=DEV)
    back, back_w = Guarded((R, cap, H), torch.bfloat16), Guarded((R, cap, K), torch.float32)
    ep.ep_expert_reduce(h, y, slot_d, num_recv=num_d, row_weights=rw, out=back.t, out_topk_weights=back_w.t)
    h.check()
    back.check()
    back_w.check()
    want = torch.zeros((R, cap, H), device=DEV)
    for k in range(K):  # fp32 additions in slot order: the same bits
        s = slot_d[:, :, k].long()
        want += torch.where((s >= 0)[..., None], y.float()[s.clamp_min(0)], 0.0)
    wrote = torch.arange(cap, device=DEV) < num_d[:, None]
    assert torch.equal(back.t[wrote], want.to(torch.bfloat16)[wrote])
    assert (back.t.view(torch.uint8)[~wrote] == back.fill).all()
    assert torch.equal(back_w.t[wrote], torch.where(slot_d >= 0, rw[slot_d.long().clamp_min(0)], 0.0)[wrote])
    assert (back_w.t.view(torch.uint8).view(R, cap, -1)[~wrote] == back.fill).all()


# --------------------------------------------------------------------------------------------- the layer they make up

def layer_reference(x, idx, w, w_up, w_down, dy):
    """Output and gradients of the layer in 64 bits, by differentiating the plain formula."""
    leaves = [v.detach().double().requires_grad_() for v in (x, w, w_up, w_down)]
    xd, wd, ud, dd = leaves
    R, T, H = x.shape
    flat, out = xd.view(R * T, H), torch.zeros((R * T, H), dtype=torch.float64, device=DEV)
    for e in range(w_up.shape[0]):
        tok, slot = torch.nonzero(idx.view(R * T, -1) == e, as_tuple=True)
        a = flat[tok] @ ud[e].t()
        gate, up = a.chunk(2, 1)
        v = gate / (1 + torch.exp(-gate)) * up * wd.view(R * T, -1)[tok, slot][:, None]
        out = out.index_add(0, tok, v @ dd[e].t())
    out = out.view(R, T, H)
    grads = torch.autograd.grad((out * dy.double()).sum(), leaves)
    return out.detach(), grads


def norm_error(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_moe_layer_trains_and_serves():
    """examples/moe_layer.py against 64 bits.  Each result passes at most eight roundings to bf16 (2^-8 of a value each,
    and a rounded gate or up value moves the activation by at most about twice that): 16 * 2^-8 in norm.  FP8 decode:
    three casts to e4m3 (2^-4 each at worst), 3 * 2^-4."""
    from examples import moe_layer as M
    R, T, H, E, K, I = 4, 37, 512, 12, 3, 256
    g = gen(41)
    x, dy = randn(g, (R, T, H)), randn(g, (R, T, H))
    w, idx = torch.softmax(torch.randn((R, T, E), generator=g, device=DEV), -1).topk(K)
    w, idx = w.contiguous(), idx.contiguous()
    idx[1, 5, 2] = -1  # a masked slot
    w_up, w_down = randn(g, (E, 2 * I, H), H ** -0.5), randn(g, (E, H, I), I ** -0.5)
    h = handle(E, R, H, T, K, R * T, 16)
    y, saved = M.forward(h, x, idx, w, w_up, w_down)
    got = M.backward(h, dy, saved, w_up, w_down)
    h.check()
    want_y, want = layer_reference(x, idx, w, w_up, w_down, dy)
    assert norm_error(y, want_y) < 16 * 2.0 ** -8
    for name, a, b in zip(("x", "topk_weights", "w_up", "w_down"), got, want):
        assert norm_error(a, b) < 16 * 2.0 ** -8, name
    yd = M.decode(h, x, idx, w, M.quantize(w_up), M.quantize(w_down))
    h.check()
    assert norm_error(yd, want_y) < 3 * 2.0 ** -4


def test_graph_replays_follow_new_inputs():
    """Products, activation and expert order captured once; replays read the counts, rows and weights that are there then."""
    E, rows, k, width = 4, 300, 256, 128
    g = gen(6)
    h = handle(E)
    x, w1, w2 = randn(g, (rows, k)), randn(g, (E, 2 * width, k), 0.1), randn(g, (E, k, width), 0.1)
    c, b = i32([10, 0, 200, 5]), i32([0, 10, 10, 210])

    def step():
        a = ep.ep_grouped_gemm(h, x, w1, c, b)
        v = ep.ep_swiglu(h, a, c, b)["out"]
        y = ep.ep_grouped_gemm(h, v, w2, c, b)
        return y, ep.ep_grouped_gemm_wgrad(h, y, v, c, b)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dw = step()
    for counts in ([10, 0, 200, 5], [0, 90, 1, 64], [0, 0, 0, 0], [300, 0, 0, 0]):
        c.copy_(i32(counts))
        b.copy_(i32(packed(counts)[0]))
        x.copy_(randn(g, (rows, k)))
        graph.replay()
        want_y, want_dw = step()
        h.check()
        n = sum(counts)
        assert torch.equal(y[:n], want_y[:n]) and torch.equal(dw, want_dw)


def test_overlapping_groups_are_reported():
    h = handle(64)
    x = torch.zeros((256, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((64, 64, 64), dtype=torch.bfloat16, device=DEV)
    c, b = i32([256] * 64), i32([0] * 64)
    out = torch.full((256, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_grouped_gemm(h, x, w, c, b, out=out)
    assert h.status() == 2 and (out == 3).all()
    act = torch.full((256, 32), 3.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_swiglu(h, x, c, b, out=act)
    assert h.status() == 2 and (act == 3).all()


# --------------------------------------------------------------------------------------------- refusals

def refused(code, words, f, *a, **kw):
    with pytest.raises(ep.EPError) as e:
        f(*a, **kw)
    assert e.value.status == code and words in str(e.value), str(e.value)


def test_refusals():
    h = handle(4, 2, 512, 8, 2, 16)
    low = handle(4, 2, 512, 8, 2, 0)
    c, b = i32([1, 0, 0, 0]), i32([0, 0, 0, 0])
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    f8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # noqa: E731
    f32 = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    g = ep.ep_grouped_gemm
    refused(1, "multiples of 8", g, h, bf(8, 60), bf(4, 64, 60), c, b)
    refused(1, "multiples of 8", g, h, bf(8, 64), bf(4, 12, 64), c, b)
    refused(1, "multiple of num_experts", g, h, bf(9, 64), bf(4, 64, 64), c)
    refused(1, "group_count", g, h, bf(8, 64), bf(4, 64, 64), None, b)
    refused(1, "4-byte", g, h, bf(8 * 64 + 1)[1:].view(8, 64), bf(4, 64, 64), c, b)
    refused(1, "multiples of 4", g, h, bf(8, 65)[:, :64], bf(4, 64, 64), c, b)
    refused(1, "16-byte aligned", g, h, bf(8, 64), bf(4 * 64 * 64 + 4)[4:].view(4, 64, 64), c, b)
    refused(1, "multiples of 4", g, h, bf(8, 64), bf(4, 64, 64), c, b, out=bf(8, 68)[:, :64])
    refused(1, "multiples of 16", ep.ep_grouped_gemm_wgrad, h, bf(8, 68)[:, :64], bf(8, 64), c, b)
    refused(1, "expected_rows", g, h, bf(8, 64), bf(4, 64, 64), c, b, expected_rows=-1)
    for bad in (bf(8, 72), f32(8, 64), torch.zeros((8, 64), dtype=torch.bfloat16)):
        with pytest.raises((TypeError, ValueError)):
            g(h, bad, bf(4, 64, 64), c, b)
    with pytest.raises(ValueError):
        g(h, bf(8, 64), bf(3, 64, 64), c, b)      # weights of three experts
    with pytest.raises(ValueError):
        g(h, bf(2, 4, 3, 64)[:, :, :2], bf(4, 64, 64), c, b)  # rows not evenly spaced
    with pytest.raises(ValueError):
        g(h, bf(64, 8).t(), bf(4, 64, 64), c, b)  # rows not contiguous inside
    with pytest.raises(TypeError):
        g(h, bf(8, 64), bf(4, 64, 64), c.long(), b)
    wg = ep.ep_grouped_gemm_wgrad
    refused(1, "accumulate needs", wg, h, bf(8, 64), bf(8, 64), c, b, out=bf(4, 64, 64), accumulate=True)
    with pytest.raises(ValueError):
        wg(h, bf(8, 64), bf(8, 64), c, b, accumulate=True)
    with pytest.raises(TypeError):
        wg(h, bf(8, 64), bf(8, 64), c, b, out=torch.zeros((4, 64, 64), dtype=torch.float16, device=DEV))
    q = ep.ep_grouped_gemm_fp8
    refused(5, "k % 128", q, h, f8(8, 64), f32(8, 0), f8(4, 64, 64), f32(4, 1, 0), c, b)
    with pytest.raises(ValueError):
        q(h, f8(8, 256), f32(8, 1), f8(4, 64, 256), f32(4, 1, 2), c, b)
    with pytest.raises(TypeError):
        q(h, f8(8, 256), bf(8, 2), f8(4, 64, 256), f32(4, 1, 2), c, b)
    s = ep.ep_swiglu
    refused(1, "multiple of 8", s, h, bf(8, 24), c, b)
    refused(5, "width % 128", s, h, bf(8, 128), c, b, cast_to_fp8=True, out=f8(8, 64), out_scales=f32(8, 0))
    refused(1, "go with cast_to_fp8", s, h, bf(8, 256), c, b, round_scale=True)
    with pytest.raises(ValueError):
        s(h, bf(8, 256), c, b, row_weights=f32(7))
    idx, n = torch.zeros((2, 16, 2), dtype=torch.int64, device=DEV), i32([1, 1])
    refused(8, "no normal dispatch", ep.ep_expert_layout, h, idx, 64)
    refused(1, "normal mode disabled", ep.ep_expert_layout, low, idx[:, :0].contiguous(), 64, num_recv=n)
    slot = torch.full((2, 16, 2), -1, dtype=torch.int32, device=DEV)
    refused(1, "go together", ep.ep_expert_gather, h, bf(2, 16, 512), slot, 64, num_recv=n, row_weights=f32(64))
    refused(1, "FP8 payload", ep.ep_expert_gather, h, f8(2, 16, 512), slot, 64, num_recv=n)
    refused(1, "go together", ep.ep_expert_reduce, h, bf(64, 512), slot, num_recv=n, row_weights=None,
            out_topk_weights=f32(2, 16, 2))
    with pytest.raises(ValueError):
        ep.ep_expert_reduce(h, bf(64, 256), slot, num_recv=n)
    h.check()
