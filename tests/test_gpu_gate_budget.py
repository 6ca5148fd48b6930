"""The router's kernels under an SM budget (ep_set_num_sms): they stay within
it, and give the same bits as without."""
import pytest
import torch

from combine_get_dispatch_gb300 import ep
from test_gpu_expert_budget import bits, budget, on_budgets, two_sms_are_two  # noqa: F401

pytestmark = pytest.mark.gpu


def gate(backward):
    R, T, E, k = 1, 65536, 256, 8
    l = torch.randn((R, T, E), device="cuda")
    idx, w = torch.empty((R, T, k), dtype=torch.int64, device="cuda"), torch.randn((R, T, k), device="cuda")
    ep.ep_gate_topk(l, ep.EP_GATE_SOFTMAX, idx, torch.empty_like(w))
    d = torch.empty_like(l)
    if backward:
        return lambda: ep.ep_gate_topk_backward(l, ep.EP_GATE_SOFTMAX, idx, w, d)
    return lambda: ep.ep_gate_topk(l, ep.EP_GATE_SOFTMAX, idx, w)


@pytest.mark.parametrize("backward", [False, True])
def test_gate_keeps_to_the_budget(budget, backward):
    two_sms_are_two(budget, gate(backward))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(64, 4), (256, 8), (512, 16)])
def test_gate_bits(budget, E, k, dtype):
    l = torch.randn((1, 3001, E), device="cuda").to(dtype)
    g = torch.randn((1, 3001, k), device="cuda")

    def call():
        idx, w, d = torch.empty((1, 3001, k), dtype=torch.int64, device="cuda"), torch.empty_like(g), torch.empty_like(l)
        ep.ep_gate_topk(l, ep.EP_GATE_SOFTMAX, idx, w)
        ep.ep_gate_topk_backward(l, ep.EP_GATE_SOFTMAX, idx, g, d)
        return bits(idx, w, d)

    on_budgets(budget, call)
