"""A mixture-of-experts layer out of libep's calls: router, dispatch, experts,
combine.

`serve` is the low-latency form: tokens travel as E4M3 with ue8m0 scales and
the experts' weights are E4M3 with one scale per 128 x 128 block.  `forward` /
`backward` are a training step in bf16 over the contiguous layout, with the
gradients of the tokens, the router's logits and all expert weights.

    python examples/moe_layer.py        # runs both on small random data (needs a GB300)
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from combine_get_dispatch_gb300 import ep  # noqa: E402


def quantise_weights(w):
    """bf16 [..., N, K] -> E4M3 bytes and ue8m0 scales of 128 x 128 blocks, laid
    out once when weights are loaded."""
    *lead, N, K = w.shape
    b = w.float().reshape(*lead, N // 128, 128, K // 128, 128)
    amax = b.abs().amax((-3, -1)).clamp(min=1e-4)
    scale = torch.ceil(torch.log2(amax / 448)).clamp(-126, 127)
    q = (b * torch.exp2(-scale)[..., :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.reshape(w.shape).view(torch.uint8), (scale + 127).to(torch.uint8)


def serve(x, logits, k, w_in, w_out, max_tokens_per_rank, status):
    """x [R, T_r, H] bf16, logits [R, T_r, E]; w_in, w_out: quantise_weights of
    [E, 2, I, H] and [E, H, I].  Returns [R, T_r, H] bf16."""
    R, T_r, H = x.shape
    E, _, I, _ = w_in[0].shape
    dev = x.device
    idx = torch.empty((R, T_r, k), dtype=torch.int64, device=dev)
    weights = torch.empty((R, T_r, k), dtype=torch.float32, device=dev)
    ep.ep_gate_topk(logits, ep.EP_GATE_SOFTMAX_TOPK, idx, weights)
    b = ep.alloc_ll(R, T_r, H, E, k, max_tokens_per_rank, ep.EP_FP8_E4M3_UE8M0, device=dev)
    ws = ep.alloc_workspace(R, T_r, k, E, H, device=dev)
    ep.ep_ll_dispatch(x, idx, E, max_tokens_per_rank, ep.EP_FP8_E4M3_UE8M0, b["packed_recv_x"], b["packed_recv_scales"],
                      b["packed_recv_src_info"], b["layout_range"], b["recv_count"], b["combine_idx"], ws, status)
    lead = b["packed_recv_x"].shape[:-1]
    h = torch.empty((*lead, I), dtype=torch.uint8, device=dev)
    h_scales = torch.empty((*lead[:-1], I // 128, lead[-1]), dtype=torch.uint8, device=dev)
    y = torch.empty((*lead, H), dtype=torch.bfloat16, device=dev)
    ep.ep_expert_glu(b["packed_recv_x"], b["packed_recv_scales"], *w_in, b["recv_count"], None, ep.EP_ACT_SILU, h,
                     h_scales=h_scales, status=status)
    ep.ep_expert_linear(h, h_scales, *w_out, None, None, b["recv_count"], None, ep.EP_ACT_NONE, y, status=status)
    out = torch.empty_like(x)
    ep.ep_ll_combine(y, weights, b["combine_idx"], E, max_tokens_per_rank, out, status)
    return out


def forward(x, logits, k, w_in, w_out, cap_rows, status):
    """The layer in bf16 over the contiguous layout (w_in [E, 2, I, H], w_out
    [E, H, I]); returns the output and what the backward needs."""
    R, T_r, H = x.shape
    E, _, I, _ = w_in.shape
    dev = x.device
    s = {"x": x, "logits": logits, "w_in": w_in, "w_out": w_out, "cap": cap_rows}
    s["idx"] = torch.empty((R, T_r, k), dtype=torch.int64, device=dev)
    s["weights"] = torch.empty((R, T_r, k), dtype=torch.float32, device=dev)
    ep.ep_gate_topk(logits, ep.EP_GATE_SOFTMAX, s["idx"], s["weights"])
    s["lay"], s["nt"] = ep.alloc_layout(R, T_r, k, E, device=dev), ep.alloc_notify(R, E, device=dev)
    s["d"] = ep.alloc_dispatch(R, T_r, H, k, ep.EP_FP8_NONE, cap_rows, device=dev)
    s["ws"] = ep.alloc_workspace(R, T_r, k, E, H, device=dev)
    ep.ep_layout_notify_dispatch(x, s["idx"], E, ep.EP_FP8_NONE, 1, R * T_r, cap_rows, s["lay"], s["nt"], s["d"], s["ws"], status)
    s["counts"], s["psum"] = s["nt"]["expert_prefix"][R], s["nt"]["psum"]
    h = torch.empty((R, cap_rows, I), dtype=torch.bfloat16, device=dev)
    gu = torch.empty((R, cap_rows, 2, I), dtype=torch.bfloat16, device=dev)
    y = torch.empty((R, cap_rows, H), dtype=torch.bfloat16, device=dev)
    ep.ep_expert_glu(s["d"]["recv_x"], None, w_in, None, s["counts"], s["psum"], ep.EP_ACT_SILU, h, gu=gu, status=status)
    ep.ep_expert_linear(h, None, w_out, None, None, None, s["counts"], s["psum"], ep.EP_ACT_NONE, y, status=status)
    out = torch.empty_like(x)
    ep.ep_combine(y, s["weights"], s["d"]["combine_idx"], cap_rows, out, status)
    s.update(h=h, gu=gu, y=y)
    return out, s


def backward(d_out, s, status):
    """Gradients of x, logits, w_in and w_out for d_out [R, T_r, H] bf16."""
    R, T_r, H = d_out.shape
    E, _, I, _ = s["w_in"].shape
    k, cap, dev = s["idx"].shape[2], s["cap"], d_out.device
    # combine backwards is dispatch: every row gets its token's gradient, times the slot's weight
    g = ep.alloc_dispatch(R, T_r, H, k, ep.EP_FP8_NONE, cap, device=dev)
    ep.ep_dispatch(d_out, s["idx"], s["lay"]["slot_rank"], s["nt"]["expert_prefix"], s["psum"], E, ep.EP_FP8_NONE, cap,
                   g["recv_x"], None, g["recv_src_idx"], g["combine_idx"], s["ws"], status)
    rows = s["d"]["combine_idx"].reshape(-1).long()          # row of every slot, -1: unused
    used = rows >= 0
    safe = torch.where(used, rows, 0)
    d_rows, y_rows = g["recv_x"].reshape(-1, H), s["y"].reshape(-1, H)
    dots = (d_rows[safe].float() * y_rows[safe].float()).sum(-1)
    d_weights = torch.where(used, dots, torch.zeros_like(dots)).reshape(R, T_r, k)
    row_weight = torch.zeros(R * cap + 1, dtype=torch.float32, device=dev)
    row_weight[torch.where(used, rows, R * cap)] = s["weights"].reshape(-1)
    d_y = (d_rows.float() * row_weight[:-1, None]).to(torch.bfloat16).reshape(R, cap, H)
    d_h, d_w_out = torch.empty_like(s["h"]), torch.empty_like(s["w_out"])
    ep.ep_expert_linear_backward(d_y, None, s["h"], s["w_out"], s["counts"], s["psum"], ep.EP_ACT_NONE, None, d_h, d_w_out,
                                 status=status)
    d_rx, d_w_in = torch.empty_like(s["d"]["recv_x"]), torch.empty_like(s["w_in"])
    # gate and up are not needed after this: their gradients take their place
    ep.ep_expert_glu_backward(d_h, s["gu"], s["d"]["recv_x"], s["w_in"], s["counts"], s["psum"], ep.EP_ACT_SILU, s["gu"],
                              d_rx, d_w_in, status=status)
    # dispatch backwards is the plain sum of a token's rows
    d_x = torch.empty_like(d_out)
    ep.ep_rank_combine(d_rx, s["d"]["combine_idx"], cap, d_x, status)
    d_logits = torch.empty_like(s["logits"])
    ep.ep_gate_topk_backward(s["logits"], ep.EP_GATE_SOFTMAX, s["idx"], d_weights, d_logits, status)
    return d_x, d_logits, d_w_in, d_w_out


def main():
    torch.manual_seed(0)
    R, T_r, E, k, H, I = 4, 64, 32, 4, 1024, 512
    dev = "cuda"
    x = torch.randn((R, T_r, H), device=dev).bfloat16()
    logits = torch.randn((R, T_r, E), device=dev)
    w_in = (torch.randn((E, 2, I, H), device=dev) * H ** -0.5).bfloat16()
    w_out = (torch.randn((E, H, I), device=dev) * I ** -0.5).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out, saved = forward(x, logits, k, w_in, w_out, R * T_r * min(k, E // R), status)
    grads = backward(torch.randn_like(x), saved, status)
    fast = serve(x, logits, k, quantise_weights(w_in), quantise_weights(w_out), T_r, status)
    torch.cuda.synchronize()
    if ep.ep_read_status(status) != ep.EP_OK:
        raise SystemExit("a kernel reported " + ep.error_string(ep.ep_read_status(status)))
    print("forward", tuple(out.shape), "gradients", [tuple(g.shape) for g in grads], "serve", tuple(fast.shape))


if __name__ == "__main__":
    main()
