"""A mixture-of-experts layer on the dispatch / combine handle: training in bf16 and low-latency serving in FP8.

    python examples/moe_layer.py          # one training step and one decode step on random weights

Training (normal mode): layout and record -> dispatch -> expert order -> gather -> up product -> gated activation with
the routing weights -> down product -> reduce -> combine; the backward pass is the same path with every step's gradient
(a combine's gradient is a cached dispatch, a gather's a reduce, and the other way round).

Serving (low-latency mode): FP8 dispatch -> up product straight from the message buffer -> gated activation with the
FP8 cast -> down product -> combine with the routing weights.
"""
from __future__ import annotations

import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from combine_get_dispatch_03_gb300 import ep


def forward(h: ep.Handle, x, topk_idx, topk_weights, w_up, w_down):
    """x [R][T][H] bf16, topk_idx / topk_weights [R][T][K], w_up [E][2I][H] and w_down [E][H][I] bf16.

    Returns the layer's output [R][T][H] bf16 and what backward() needs."""
    c = h.cfg
    ep.ep_layout_notify(h, topk_idx)
    d = ep.ep_dispatch(h, x, topk_idx=topk_idx, topk_weights=topk_weights, prepared=True)
    rows = topk_idx.numel() + c.num_experts * (c.expert_alignment - 1)  # enough for any routing
    lay = ep.ep_expert_layout(h, d["recv_topk_idx"], rows)
    g = ep.ep_expert_gather(h, d["recv_x"], lay["slot_row"], rows, topk_weights=d["recv_topk_weights"])
    groups = (lay["group_count"], lay["group_begin"])
    up = ep.ep_grouped_gemm(h, g["out"], w_up, *groups)
    act = ep.ep_swiglu(h, up, *groups, row_weights=g["row_weights"])["out"]
    down = ep.ep_grouped_gemm(h, act, w_down, *groups)
    back = ep.ep_expert_reduce(h, down, lay["slot_row"])["out"]
    y = ep.ep_combine(h, back)["combined_x"]
    return y, dict(groups=groups, slot_row=lay["slot_row"], rows=rows, x=g["out"], weights=g["row_weights"], up=up, act=act)


def backward(h: ep.Handle, dy, saved, w_up, w_down):
    """dy [R][T][H] bf16, on the handle whose record forward() built: the gradients of x, topk_weights, w_up, w_down."""
    groups, slot_row = saved["groups"], saved["slot_row"]
    drecv = ep.ep_dispatch(h, dy, cached=True)["recv_x"]
    ddown = ep.ep_expert_gather(h, drecv, slot_row, saved["rows"])["out"]
    dact = ep.ep_grouped_gemm(h, ddown, w_down, *groups, w_transposed=True)
    dw_down = ep.ep_grouped_gemm_wgrad(h, ddown, saved["act"], *groups)
    g = ep.ep_swiglu_grad(h, dact, saved["up"], *groups, row_weights=saved["weights"])
    dw_up = ep.ep_grouped_gemm_wgrad(h, g["dx"], saved["x"], *groups)
    dx = ep.ep_grouped_gemm(h, g["dx"], w_up, *groups, w_transposed=True)
    back = ep.ep_expert_reduce(h, dx, slot_row, row_weights=g["d_row_weights"])
    c = ep.ep_combine(h, back["out"], topk_weights=back["out_topk_weights"])
    return c["combined_x"], c["combined_topk_weights"], dw_up, dw_down


def quantize(w):
    """bf16 weights [E][n][k] -> e4m3 codes and one fp32 scale per 128 x 128 block (done once, when a server loads them)."""
    E, n, k = w.shape
    nb = -(-n // 128)
    blocks = torch.zeros((E, nb * 128, k), dtype=torch.float32, device=w.device)
    blocks[:, :n] = w.float()
    blocks = blocks.view(E, nb, 128, k // 128, 128)
    scales = blocks.abs().amax((2, 4)).clamp_min(1e-4) / 448
    codes = (blocks / scales[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(E, nb * 128, k)[:, :n].contiguous(), scales


def decode(h: ep.Handle, x, topk_idx, topk_weights, up, down):
    """Low-latency step: x [R][T][H] bf16, T <= num_max_tokens; `up` and `down` are quantize()d weights."""
    c = h.cfg
    d = ep.ep_ll_dispatch(h, x, topk_idx, use_fp8=True, use_ue8m0=True)
    px, scales, _ = ep.ll_views(d["recv_msgs"], c.hidden, True)
    count = d["packed_recv_count"]
    expected = max(1, topk_idx.numel() // c.num_experts)
    a = ep.ep_grouped_gemm_fp8(h, px, scales, *up, count, expected_rows=expected)
    v = ep.ep_swiglu(h, a, count, cast_to_fp8=True)
    y = ep.ep_grouped_gemm_fp8(h, v["out"], v["out_scales"], *down, count, expected_rows=expected)
    return ep.ep_ll_combine(h, y, topk_idx, topk_weights)


def main():
    R, T, H, E, K, I = 8, 256, 1024, 32, 4, 512
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(0)

    def randn(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(torch.bfloat16)

    x, dy = randn(R, T, H), randn(R, T, H)
    topk_weights, topk_idx = torch.softmax(torch.randn((R, T, E), generator=g, device=dev), -1).topk(K)
    topk_idx, topk_weights = topk_idx.contiguous(), topk_weights.contiguous()
    w_up, w_down = randn(E, 2 * I, H, std=H ** -0.5), randn(E, H, I, std=I ** -0.5)
    h = ep.Handle(ep.Config(num_ranks=R, num_max_tokens=T, hidden=H, num_experts=E, num_topk=K, recv_capacity=R * T))
    y, saved = forward(h, x, topk_idx, topk_weights, w_up, w_down)
    grads = backward(h, dy, saved, w_up, w_down)
    h.check()
    print("training: output", tuple(y.shape), "gradients", [tuple(v.shape) for v in grads])
    t = 8
    yd = decode(h, x[:, :t].contiguous(), topk_idx[:, :t].contiguous(), topk_weights[:, :t].contiguous(),
                quantize(w_up), quantize(w_down))
    h.check()
    off = (yd.float() - y[:, :t].float()).norm() / y[:, :t].float().norm()
    print(f"decode: output {tuple(yd.shape)}, {float(off):.3f} from the bf16 layer (FP8 weights and activations)")


if __name__ == "__main__":
    main()
