"""The gradient of the products' epilogue with d_pre in pre's memory: the same bits as beside it."""
import pytest
import torch

from combine_get_dispatch_03_gb300 import ep
from test_gpu_experts import DEV, gen, handle, i32, packed, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [8, 200, 264, 1024, 2312])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("pad", [0, 8])
def test_gradient_in_place(width, gated, act, pad):
    """Several blocks of columns, several chunks of rows and a part of one, groups without rows, strided rows, all sums."""
    counts = [70, 0, 1, 133, 9]
    begin, rows = packed(counts, gap=3)
    g = gen(width)
    n = 2 * width if gated else width
    dy, weights = randn(g, (rows, width)), torch.rand(rows, generator=g, device=DEV)
    pre = randn(g, (rows, n + pad))
    h = handle(5)
    c, b = i32(counts), i32(begin)
    kw = dict(act=act, gated=gated, row_weights=weights, with_bias=True)
    want = ep.ep_act_grad(h, dy, pre[:, :n].clone(), c, b, **kw)
    for _ in range(3):
        both = pre.clone()
        got = ep.ep_act_grad(h, dy, both[:, :n], c, b, d_pre=both[:, :n], **kw)
        used = torch.zeros(rows, dtype=torch.bool, device=DEV)
        for at, m in zip(begin, counts):
            used[at:at + m] = True
        assert torch.equal(both[used, :n], want["d_pre"][used])
        assert torch.equal(both[~used], pre[~used]) and torch.equal(both[:, n:], pre[:, n:])
        assert torch.equal(got["d_row_weights"][used], want["d_row_weights"][used])
        assert torch.equal(got["d_bias"], want["d_bias"])
    h.check()
