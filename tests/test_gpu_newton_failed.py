"""The optimiser's step after a wait that ran out in one of its products: weights are
not updated from what that product left.

A product that gives up says so in the last word of the workspace; here the host writes it while
the products run (on two SMs, some 100 ms)."""
import time

import pytest
import torch

from combine_get_dispatch_gb300 import ep
from test_gpu_expert_budget import budget  # noqa: F401

pytestmark = pytest.mark.gpu

STEPS = [(3.4445, -4.7750, 2.0315)] * 5


def test_weights_stay_where_a_product_failed(budget):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(1)
    g = torch.randn((32, 1416, 2048), generator=gen, device="cuda").bfloat16()
    w = torch.randn(g.shape, generator=gen, device="cuda")
    m, ws = torch.zeros_like(w), ep.alloc_orthogonalize_workspace(g.shape)
    failed = ws[-256:].view(torch.int32)[:1]
    got_w, got16 = w.clone(), torch.full_like(g, 7.0)
    ep.ep_muon_update(g[:1], m[:1].clone(), w[:1].clone(), got16[:1].clone(), STEPS, ws, lr=0.1)   # loads the kernels
    budget(2)
    stream, side = torch.cuda.Stream(), torch.cuda.Stream()
    one, ended = torch.ones(1, dtype=torch.int32).pin_memory(), torch.cuda.Event()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        ep.ep_muon_update(g, m, got_w, got16, STEPS, ws, lr=0.1, nesterov=False)
        ended.record()
    time.sleep(0.02)   # the word is cleared by the first kernel as it begins
    with torch.cuda.stream(side):
        failed.copy_(one, non_blocking=True)
    side.synchronize()
    assert not ended.query(), "the call was over before"
    torch.cuda.synchronize()
    assert torch.equal(got_w, w) and bool((got16 == 7).all()) and torch.equal(m, g.float())
    # the next call starts anew, whatever the word says
    budget(0)
    m.zero_()
    ep.ep_muon_update(g, m, got_w, got16, STEPS, ws, lr=0.1, nesterov=False)
    assert bool((got_w != w).any(-1).all()) and torch.equal(got16, got_w.bfloat16())
