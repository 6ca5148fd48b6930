"""The activations of the expert calls by themselves, relative to their own
value: rows of x are unit vectors, so that every sum is one weight, exactly.

Tolerances for |z| <= 12.  GELU is z Phi(z), and the tail of Phi an exponential of
-z^2 / 2 >= -72, whose argument three roundings of 2^-24 put off by 72 x 3 x 2^-24
< 2^-16, times a factor within 2^-19; SiLU divides by 1 + exp(-z), whose exponential
is within 2 + 1.2 |z| ulp < 2^-18.  The slopes add z exp(-z^2 / 2) / sqrt(2 pi), off by
as much.  So 2^-15 of the value (of the slope's two terms), and 2^-8 for the one
rounding to bf16."""
import math

import pytest
import torch

from combine_get_dispatch_gb300 import ep

pytestmark = pytest.mark.gpu

ROWS, N, K = 3, 2048, 8


def values():
    """N bf16 values from -12 to 12, the flanks of zero among them."""
    z = torch.linspace(-12, 12, N, device="cuda").bfloat16()
    z[:16] = torch.tensor([0.0, -0.0, 2.0 ** -60, -2.0 ** -60, 2.0 ** -9, -2.0 ** -9, 0.5, -0.5, 1.0, -1.0, -0.75, 3.5, -3.5,
                           -5.0, -5.25, -5.5]).bfloat16()
    return z


def act64(z, name):
    """Value, slope, and the sum of the slope's terms' magnitudes."""
    z = z.double()
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        t = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    else:
        c = 1 / (1 + torch.exp(-z))
        t = z * torch.exp(-z) / (1 + torch.exp(-z)) ** 2
    return z * c, c + t, c + t.abs()


def near(got, ref, terms=None):
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -15 * (ref if terms is None else terms).abs()
    off = (got.double() - ref).abs()
    assert bool((off <= tol).all()), f"off by {float((off / ref.abs().clamp(min=1e-300)).max()):.3g} of the value"


def tables():
    return (torch.tensor([ROWS], dtype=torch.int32, device="cuda"),
            torch.tensor([[0, ROWS]], dtype=torch.int64, device="cuda"))


def unit_rows():
    x = torch.zeros((1, ROWS, K), dtype=torch.bfloat16, device="cuda")
    x[..., 0] = 1
    return x


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_linear_value_and_slope(act):
    z, (c, ps) = values(), tables()
    v, s, terms = act64(z, act)
    w = torch.randn((1, N, K), device="cuda").bfloat16()
    w[0, :, 0] = z
    y = torch.empty((1, ROWS, N), dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_linear(unit_rows(), None, w, None, None, None, c, ps, ep.ACTS[act], y)
    near(y, v.expand(1, ROWS, N))
    pre, dpre = z.expand(1, ROWS, N).contiguous(), torch.empty_like(y)
    ep.ep_expert_linear_backward(torch.ones_like(y), pre, None, w, c, ps, ep.ACTS[act], dpre, None, None,
                                 dbias=torch.empty((1, N), dtype=torch.bfloat16, device="cuda"))
    near(dpre, s.expand(1, ROWS, N), terms)


@pytest.mark.parametrize("up", [1.0, 2.0 ** 40])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_value_and_slope(act, up):
    z, (c, ps) = values(), tables()
    v, s, terms = act64(z, act)
    w = torch.randn((1, 2, N, K), device="cuda").bfloat16()
    w[0, 0, :, 0] = z
    w[0, 1, :, 0] = up
    h = torch.empty((1, ROWS, N), dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_glu(unit_rows(), None, w, None, c, ps, ep.ACTS[act], h)
    near(h, up * v.expand(1, ROWS, N))
    gu = torch.stack((z, torch.full_like(z, up))).expand(1, ROWS, 2, N).contiguous()
    dgu, dw = torch.empty_like(gu), torch.empty((1, 2, N, K), dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_glu_backward(torch.ones_like(h), gu, unit_rows(), None, c, ps, ep.ACTS[act], dgu, None, dw)
    near(dgu[:, :, 0], up * s.expand(1, ROWS, N), up * terms)
    near(dgu[:, :, 1], v.expand(1, ROWS, N))
