"""The example layer -- router, dispatch, experts, combine, and its backward --
against a dense 64-bit layer.

Tolerances, as relative 2-norms.  Forward: h, y and the output are rounded to
bf16 once each (2^-8 at most, 2^-9 / sqrt(3) of the norm on average): 3 roundings,
bounded by 2^-8 sqrt(3) < 0.007.  Gradients pass some twice as many: 0.014; the
router's is a difference of two dot products of about equal size: 0.03.  E4M3:
tokens, weights and h are rounded to 4 significant bits (2^-4 at most, 0.026 of
the norm on average), through scales of a power of two: 4 such roundings, below
0.12."""
import os
import sys

import pytest
import torch

from combine_get_dispatch_gb300 import ep

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def dense(x, logits, k, w_in, w_out, topk_softmax):
    """The layer by every token through every expert it chose; differentiable."""
    R, T_r, H = x.shape
    E = logits.shape[-1]
    p = torch.softmax(logits, -1)
    _, idx = torch.sort(logits.detach(), dim=-1, descending=True, stable=True)
    idx = idx[..., :k]
    w = torch.gather(p, -1, idx)
    if topk_softmax:
        w = w / w.sum(-1, keepdim=True)
    mix = torch.zeros_like(p).scatter(-1, idx, w).reshape(-1, E)
    xf = x.reshape(-1, H)
    out = torch.zeros_like(xf)
    for e in range(E):
        hit = (mix[:, e].detach() != 0).nonzero()[:, 0]
        g, u = xf[hit] @ w_in[e, 0].t(), xf[hit] @ w_in[e, 1].t()
        y = (torch.nn.functional.silu(g) * u) @ w_out[e].t()
        out = out.index_add(0, hit, mix[hit, e, None] * y)
    return out.reshape(x.shape)


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("R,T_r,E,k,H,I", [(4, 16, 16, 2, 256, 128), (2, 65, 8, 3, 384, 256), (8, 40, 64, 6, 512, 384)])
def test_layer_matches_dense(R, T_r, E, k, H, I):
    import moe_layer
    g = torch.Generator(device="cuda").manual_seed(E)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, logits = rand(R, T_r, H).bfloat16(), rand(R, T_r, E)
    w_in, w_out = (rand(E, 2, I, H) * H ** -0.5).bfloat16(), (rand(E, H, I) * I ** -0.5).bfloat16()
    d_out = rand(R, T_r, H).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, saved = moe_layer.forward(x, logits, k, w_in, w_out, R * T_r * min(k, E // R), status)
    got = moe_layer.backward(d_out, saved, status)
    args = [t.double().requires_grad_() for t in (x, logits, w_in, w_out)]
    ref = dense(args[0], args[1], k, args[2], args[3], False)
    ref.backward(d_out.double())
    assert rel(out, ref.detach()) < 0.007
    for name, a, b, tol in zip(("x", "logits", "w_in", "w_out"), got, args, (0.014, 0.03, 0.014, 0.014)):
        assert rel(a, b.grad) < tol, name
    fast = moe_layer.serve(x, logits, k, moe_layer.quantise_weights(w_in), moe_layer.quantise_weights(w_out), T_r, status)
    ref = dense(x.double(), logits.double(), k, w_in.double(), w_out.double(), True)
    assert rel(fast, ref) < 0.12
    assert ep.ep_read_status(status) == ep.EP_OK


def test_example_runs():
    import moe_layer
    moe_layer.main()
