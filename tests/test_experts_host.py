"""The expert products' host side without a GPU: rows as views, and calls without a handle."""
import pytest
import torch

from combine_get_dispatch_03_gb300 import ep

CPU = torch.device("cpu")


def rows(t, *want):
    return ep._rows(t, "x", t.dtype, CPU, *want)[1:]


def test_rows_of_views():
    x = torch.zeros((6, 64), dtype=torch.bfloat16)
    assert rows(x) == (6, 64, 128)
    assert rows(x[:, :32]) == (6, 32, 128)
    assert rows(x[::2]) == (3, 64, 256)
    assert rows(x.view(2, 3, 64)) == (6, 64, 128)
    assert rows(x.view(2, 3, 64)[:, :, 8:16]) == (6, 8, 128)
    assert rows(x.view(2, 1, 3, 64)[..., :8]) == (6, 8, 128)
    assert rows(x[:1, :12]) == (1, 12, 32)  # one row: its stride is rounded up to what a call accepts
    assert rows(x[:0])[:2] == (0, 64)
    msgs = torch.zeros((2, 3, 5, 16 + 512 + 16), dtype=torch.uint8)
    px, scales, _ = ep.ll_views(msgs, 512, True)
    assert rows(px) == (30, 512, 544)
    assert rows(scales[..., :4]) == (30, 4, 544)
    assert rows(scales.view(torch.float32)) == (30, 4, 544)


@pytest.mark.parametrize("make", [
    lambda: torch.zeros((2, 3, 64))[:, :2],          # a gap between the two halves
    lambda: torch.zeros((8, 4)).t(),                 # elements of a row apart
    lambda: torch.zeros(8),                          # no rows
    lambda: torch.zeros((1, 8, 2))[:, :, 0],         # one row of strided elements
])
def test_rows_refuses(make):
    with pytest.raises(ValueError):
        rows(make())


def test_rows_checks_sizes_and_types():
    x = torch.zeros((6, 64))
    for want in ((5, None), (None, 63)):
        with pytest.raises(ValueError):
            rows(x, *want)
    with pytest.raises(TypeError):
        ep._rows(x, "x", torch.bfloat16, CPU)
    with pytest.raises(TypeError):
        ep._rows(None, "x", torch.bfloat16, CPU)


def test_calls_without_a_handle_are_refused():
    L = ep.lib()
    for rc in (L.ep_grouped_gemm(None, 0, 8, 8, None, None, None, 16, None, 0, None, 16, 0, None),
               L.ep_grouped_gemm_wgrad(None, 0, 8, 8, None, None, None, 16, None, 16, None, 2, 0, None),
               L.ep_grouped_gemm_fp8(None, 0, 8, 128, None, None, None, 128, None, 4, 0, None, None, None, 16, 0, None),
               L.ep_swiglu(None, 0, 8, None, None, None, 32, None, 0, 0, None, 16, None, None),
               L.ep_swiglu_grad(None, 0, 8, None, None, None, 16, None, 32, None, None, 32, None, None),
               L.ep_expert_layout(None, None, None, 0, None, None, None, None),
               L.ep_expert_gather(None, None, 0, None, None, None, None, 0, None, None, None, None),
               L.ep_expert_reduce(None, None, 16, None, None, None, 0, None, None, None)):
        assert rc == 1 and b"handle is NULL" in L.ep_last_error()
