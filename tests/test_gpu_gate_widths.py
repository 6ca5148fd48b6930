"""The router at the widths and k that no other test reaches: more than 12
choices of up to 256 experts, and the gradient of more than 8 choices of up to
128.  References and tolerances are those of test_gpu_gate.py."""
import math

import pytest
import torch

from combine_get_dispatch_gb300 import ep
from test_gpu_gate import draw, reference, reference_grad, run_gate

pytestmark = pytest.mark.gpu

INF = math.inf


def neighbours(E, k, dtype):
    """Random tokens, tokens of few distinct values, and tokens that take different ways beside one another."""
    rows = torch.cat((draw(1, 24, E, torch.float32, seed=E + k), draw(1, 25, E, torch.float32, seed=E - k, ties=True)), 1)
    rows[0, 1::8] = 2.5                                # every expert ties
    rows[0, 2::8] = -INF
    rows[0, 3::8, 1:] = -INF                           # one expert left
    rows[0, 4::8] = torch.linspace(-3, 3, E)
    rows[0, 5::16, :: max(1, E // 40)] = 5.0           # some forty equal largest
    rows[0, 13::16, E // 2] = INF
    rows[0, 6::16, :2] = math.nan
    return rows.to(dtype)


@pytest.mark.parametrize("score", ["softmax", "softmax_topk"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(13, 13), (16, 16), (64, 16), (40, 13), (63, 14), (100, 14), (125, 16), (128, 16),
                                 (200, 13), (255, 15), (256, 16)])
def test_many_choices(E, k, dtype, score):
    l = neighbours(E, k, dtype)
    idx, w = run_gate(l.cuda(), k, score)
    ref_idx, ref_w = reference(l, k, score)
    assert torch.equal(idx.cpu(), ref_idx)
    assert torch.isfinite(w).all()
    assert ((w.cpu().double() - ref_w).abs() <= 6e-6 * ref_w + 1e-37).all()


@pytest.mark.parametrize("score", ["softmax", "softmax_topk"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(9, 9), (16, 16), (65, 11), (100, 12), (128, 16), (129, 9), (255, 16), (256, 10)])
def test_gradient_of_many_choices(E, k, dtype, score):
    l = draw(1, 37, E, dtype, seed=5 * E + k)
    l[0, 3] = -INF
    l[0, 4, 1:] = -INF
    idx, _ = reference(l, k, score)
    g = torch.randn((1, 37, k), generator=torch.Generator().manual_seed(6))
    out, st = torch.full_like(l, 3.0).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_gate_topk_backward(l.cuda(), ep.GATE_SCORES[score], idx.cuda(), g.cuda(), out, st)
    ref, mag = reference_grad(l, idx, g, score)
    tol = 2e-5 * mag + (0 if dtype == torch.float32 else 2.0 ** -8 * ref.abs()) + 1e-40
    assert ((out.cpu().double() - ref).abs() <= tol).all()
    assert ep.ep_read_status(st) == ep.EP_OK


@pytest.mark.parametrize("E,k,dtype", [(64, 16, torch.float32), (64, 16, torch.bfloat16), (250, 16, torch.float32),
                                       (128, 13, torch.bfloat16)])
def test_unaligned_logits(E, k, dtype):
    """Logits that start off a 16-byte boundary are read value by value: the same bits."""
    l = neighbours(E, k, dtype).cuda()
    idx, w = run_gate(l, k, "softmax")
    room = torch.empty(l.numel() + 1, dtype=dtype, device="cuda")
    odd = room[1:].view(l.shape)
    odd.copy_(l)
    idx2, w2 = run_gate(odd, k, "softmax")
    assert torch.equal(idx, idx2) and torch.equal(w, w2)
