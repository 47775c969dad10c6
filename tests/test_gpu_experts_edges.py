"""The expert operators at their edges: groups that overlap, waits that run out, calls from new threads, values at the
ends of the formats, and the paths that only some sizes take."""
import pytest
import torch

from combine_get_dispatch_03_gb300 import ep
from _parity import Guarded
from test_gpu_experts import DEV, handle, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["forward", "transposed", "fp8"])
@pytest.mark.parametrize("expected", [1, 100000], ids=["single", "pair"])
@pytest.mark.parametrize("counts,begin,rows", [
    ([100] * 8, [0] * 8, 100),             # one row tile each: no more tiles than groups apart would have
    ([256] * 64, [0] * 64, 256),
    ([3, 2], [0, 2], 4),                   # one row too many
    ([4, 1, 0], [0, 3, 9], 4),
    ([300, 0, 300, 300], [0, 0, 1, 2], 302),
], ids=["8x100", "64x256", "one", "one-with-empty", "4x300"])
def test_more_rows_than_there_are_write_nothing(counts, begin, rows, expected, form):
    """Whatever the tile height: EP_ERR_CAPACITY, and the output as it was."""
    E, n, k = len(counts), 72, 128
    h = handle(E)
    c, b = i32(counts), i32(begin)
    out = Guarded((rows, n), torch.bfloat16)

    def run(c):
        if form == "fp8":
            zero = torch.zeros((rows + E * n, k), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
            ep.ep_grouped_gemm_fp8(h, zero[:rows], torch.ones((rows, 1), device=DEV), zero[rows:].view(E, n, k),
                                   torch.ones((E, 1, 1), device=DEV), c, b, out=out.t, expected_rows=expected)
        else:
            zero = torch.zeros((rows + E * n, k), dtype=torch.bfloat16, device=DEV)
            w = zero[rows:].view((E, k, n) if form == "transposed" else (E, n, k))
            ep.ep_grouped_gemm(h, zero[:rows], w, c, b, w_transposed=form == "transposed", out=out.t, expected_rows=expected)
    run(c)
    assert h.status() == 2
    out.check()
    assert (out.t.view(torch.uint8) == out.fill).all()
    run(i32([rows] + [0] * (E - 1)))  # every row there is, once
    h.check()
    assert (out.t == 0).all()
