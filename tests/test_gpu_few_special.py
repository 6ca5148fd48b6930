"""Infinities among the layer's weights and hidden numbers: they come out as the formula
has them, an infinity times a number that is not zero being one."""
import pytest
import torch

from combine_get_dispatch_gb300 import ep
from test_gpu_few import act64, call, make, wide

pytestmark = pytest.mark.gpu

INF = float("inf")


def layer64(s, act):
    H = s["x"].shape[-1]
    x, idx = s["x"].double().reshape(-1, H), s["idx"].reshape(-1, s["idx"].shape[-1])
    weights, out = s["weights"].double().reshape(idx.shape), torch.zeros_like(x)
    for e in sorted(set(idx.flatten().tolist()) - {-1}):
        t, j = (idx == e).nonzero(as_tuple=True)
        gu, down = wide(s["w_gu"], None, e), wide(s["w_down"], None, e)
        h = act64(x[t] @ gu[0].t(), act) * (x[t] @ gu[1].t())
        # a sum of products: a matrix product in 64 bits may skip or split where numbers are infinite
        out.index_add_(0, t, weights[t, j].unsqueeze(1) * (h.unsqueeze(1) * down.unsqueeze(0)).sum(-1))
    return out.reshape(s["x"].shape)


def same(a, b):
    """Infinities, their signs and NaN in the same places, and what is finite near."""
    a = a.double()
    assert torch.equal(a.isnan(), b.isnan())
    assert torch.equal(torch.where(a.isinf(), a, 0.0), torch.where(b.isinf(), b, 0.0))
    f = torch.isfinite(b)
    assert bool(((a - b)[f].abs() <= 0.01 * b[f].abs().max()).all())


@pytest.mark.parametrize("T", [1, 7, 20, 40, 64])
@pytest.mark.parametrize("act", ["silu", "relu"])
def test_infinite_weights(T, act):
    s = make(T, 1, T, 2, 4, 72, 200, "bf16")
    for e in range(4):
        for n, value in enumerate((INF, -INF, INF)):
            s["w_down"][e, 7 * n + e, 31 * n + 5 * e] = value
    s["w_down"][2, 50, 3], s["w_down"][2, 50, 4] = INF, -INF
    # (times relu's zeros they are NaN)
    want = layer64(s, act)
    assert bool(want.isinf().any())
    same(call(s, act), want)


@pytest.mark.parametrize("T", [1, 3, 12, 48])
def test_hidden_numbers_that_bf16_holds(T):
    """h = 6, -6, 2^-100, an infinity: its second word is nothing, and does not show."""
    s = make(1, 1, T, 1, 1, 16, 16, "bf16")
    for n in ("x", "idx", "w_gu", "w_down"):
        s[n].zero_()
    s["weights"].fill_(1.0)
    s["x"][..., 0] = 1.0
    gate, up, down = s["w_gu"][0, 0], s["w_gu"][0, 1], s["w_down"][0]
    gate[0, 0], up[0, 0] = 2.0, 3.0
    gate[1, 0], up[1, 0] = 2.0, -3.0
    gate[2, 0], up[2, 0] = 2.0 ** -50, 2.0 ** -50
    down[0, 0], down[1, 0], down[2, 1], down[3, 2], down[4, 2] = INF, -INF, INF, INF, -INF
    down[5, 0], down[5, 1], down[6, 2] = 1.0, 0.5, 2.0 ** 100
    down[7, 9] = INF                                # times a zero
    out = call(s, "relu")
    want = torch.tensor([INF, -INF, -INF, INF, -INF, 3.0, 1.0, float("nan")] + [0.0] * 8, device="cuda").bfloat16()
    assert torch.equal(out[0].nan_to_num(nan=77.0), want.nan_to_num(nan=77.0).expand(T, 16))
    gate[3, 0], up[3, 0] = 3e38, 1e38               # h is an infinity in 32 bits
    down[:, 3] = 1.0
    down[8, 3], down[9, 3], down[10, 3] = INF, -INF, 0.0
    out = call(s, "relu")
    want = torch.tensor([INF, float("nan"), float("nan"), INF, float("nan"), INF, INF, float("nan"), INF, -INF, float("nan")] + [INF] * 5, device="cuda").bfloat16()
    assert torch.equal(torch.nan_to_num(out[0], nan=77.0), torch.nan_to_num(want, nan=77.0).expand(T, 16))
    assert ep.ACTS["relu"] == ep.EP_ACT_RELU


@pytest.mark.parametrize("T", [1, 6, 40])
@pytest.mark.parametrize("size", [-126, -110, -60, 0, 60, 100, 106])
def test_e4m3_scales_against_tokens(T, size):
    """Tokens of 2^size against gate and up scales of about 2^-size: what the layer computes with is of ordinary size."""
    from test_gpu_few import reference
    s = make(T, 1, T, 2, 4, 256, 128, "e4m3")
    s["x"] = (s["x"].clamp(-3.9, 3.9).double() * 2.0 ** size).bfloat16()
    s["gu_scales"] = (s["gu_scales"].int() - size).clamp(0, 254).to(torch.uint8)
    out = call(s, "silu")
    want, off = reference(s, "silu")
    # (a token's two parts lie 2^-140 apart at the least, closer than bf16 numbers anywhere)
    d = (out.double() - want).abs()
    assert bool((d <= off).all()), float((d / off).max())


@pytest.mark.parametrize("T", [1, 6, 40])
@pytest.mark.parametrize("byte", [0, 20, 127, 240, 254])
def test_e4m3_zeros_under_any_scale(T, byte):
    """Blocks of zero weights, whatever their scale, add nothing to tokens of any size."""
    from test_gpu_few import reference
    s = make(T, 1, T, 2, 4, 384, 256, "e4m3")
    s["x"] *= 2.0 ** 12
    s["gu_scales"] -= 12
    for w, sc, at in ((s["w_gu"], s["gu_scales"], (slice(None), 1, 0, 1)), (s["w_gu"], s["gu_scales"], (2, 0, 1, 2)), (s["w_down"], s["down_scales"], (1, 2, 0))):
        *lead, n, k = at
        w[(*lead, slice(128 * n, 128 * n + 128), slice(128 * k, 128 * k + 128))] = 0
        sc[at] = byte
    out = call(s, "silu")
    want, off = reference(s, "silu")
    d = (out.double() - want).abs()
    assert bool((d <= off).all()), float((d / off).max())
