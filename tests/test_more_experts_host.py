"""Host side of the router, the products with an epilogue and the layer for a few tokens, without a GPU."""
import pytest
import torch

from combine_get_dispatch_03_gb300 import ep


def test_calls_without_a_handle_are_refused():
    L = ep.lib()
    for rc in (L.ep_grouped_gemm_act(None, 0, 8, 8, None, None, None, 16, None, None, 0, 0, None, None, 0, None, 0, None, 0, 16, 0, None, 0, None),
               L.ep_act_grad(None, 0, 8, None, None, None, 16, None, 16, 0, 0, None, None, 0, None, None, None, 0, None),
               L.ep_router(None, 0, None, 2, None, None, 0, 1, 1, 1, 1.0, None, None, None),
               L.ep_router_grad(None, 0, None, 2, None, None, 0, 1, 1.0, None, None),
               L.ep_moe_layer(None, 0, 8, None, None, None, None, None, None, None, 0, None, None, None, None, 0, None)):
        assert rc == 1 and b"handle is NULL" in L.ep_last_error()
    assert L.ep_act_grad_workspace(None, 4, 8) == -1
    assert L.ep_moe_layer_workspace(None, 4, 8) == -1


class NoHandle:
    """Sizes without a device: what the binding refuses before it calls the library."""

    def __init__(self, **kw):
        self.cfg = ep.Config(**{**dict(num_ranks=2, num_max_tokens=4, hidden=256, num_experts=4, num_topk=2), **kw})
        self.device = torch.device("cpu")

    ptr = None


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("change,error", [
    (dict(x=zeros(8, 256)), ValueError),
    (dict(x=zeros(2, 4, 128)), ValueError),
    (dict(x=zeros(2, 4, 256, dtype=torch.float32)), TypeError),
    (dict(w_up=zeros(4, 63, 256)), ValueError),
    (dict(w_up=zeros(4, 64, 256, dtype=torch.float16)), TypeError),
    (dict(w_up=zeros(64, 256)), ValueError),
], ids=["rank", "hidden", "type", "odd", "weights", "dims"])
def test_layer_arguments(change, error):
    args = dict(x=zeros(2, 4, 256), w_up=zeros(4, 64, 256), w_down=zeros(4, 256, 32))
    args.update(change)
    with pytest.raises(error):
        ep.ep_moe_layer(NoHandle(), args["x"], torch.zeros((2, 4, 2), dtype=torch.int64), zeros(2, 4, 2, dtype=torch.float32),
                        args["w_up"], args["w_down"])


def test_router_and_product_arguments():
    h = NoHandle()
    with pytest.raises(TypeError):
        ep.ep_router(h, zeros(3, 4, dtype=torch.float16))
    with pytest.raises(ValueError):
        ep.ep_router(h, zeros(3, 5))
    c = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ep.ep_grouped_gemm_act(h, zeros(3, 8), zeros(4, 15, 8), c, gated=True)
    with pytest.raises(ValueError):
        ep.ep_grouped_gemm_act(h, zeros(3, 16), zeros(4, 16, 8), c)
    with pytest.raises(TypeError):
        ep.ep_grouped_gemm_act(h, zeros(3, 8), zeros(4, 16, 8), c, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="act must be one of"):
        ep._choice("tanh", ep.ACTS, "act")
