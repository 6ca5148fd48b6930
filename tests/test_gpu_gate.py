"""The router's top-k and its gradient against plain 64-bit definitions: ids
exactly (ties to the lower expert), weights and gradients to fp32 rounding.

Tolerances.  A weight is one exponential over a sum of at most E of them: expf
is within 2 ulp and its argument l - m is rounded once (an absolute error of
|l - m| 2^-24, so a relative one of the exponential, and the exponential is
below 2^-24 of the largest for |l - m| > 17); the sum of E <= 1024 positive
terms over 32 lanes rounds at most 37 times, the quotient once:
(17 + 4 + 37 + 17 + 4 + 2) 2^-24 < 6e-6 relative.  A gradient is a sum of at
most two products of such weights and the sum of k <= 16 products: 6e-6 of the
terms' magnitude, each taken with its sign dropped, three factors: 2e-5."""
import math

import pytest
import torch

from combine_get_dispatch_gb300 import ep

pytestmark = pytest.mark.gpu

INF = math.inf


def reference(logits, k, score):
    """(idx, weights float64) on the host, one row at a time."""
    R, T_r, E = logits.shape
    idx = torch.full((R, T_r, k), -1, dtype=torch.int64)
    w = torch.zeros((R, T_r, k), dtype=torch.float64)
    for r in range(R):
        for t in range(T_r):
            row = logits[r, t].double().tolist()
            order = sorted((e for e in range(E) if row[e] > -INF), key=lambda e: (-row[e], e))
            chosen = order[:k]
            if not chosen:
                continue
            m = row[chosen[0]]
            ex = {e: 1.0 if row[e] == m else math.exp(row[e] - m) for e in order}
            total = math.fsum(ex[e] for e in (order if score == "softmax" else chosen))
            for j, e in enumerate(chosen):
                idx[r, t, j] = e
                w[r, t, j] = ex[e] / total
    return idx, w


def reference_grad(logits, idx, grad, score):
    """(gradient, sum of the terms' magnitudes), float64, dense."""
    l = logits.double()
    ok = (idx >= 0).double()
    at = idx.clamp(min=0)
    finite = l > -INF
    m = torch.where(finite, l, torch.full_like(l, -1e300)).amax(-1, keepdim=True)
    ex = torch.where(finite, torch.exp(l - m), torch.zeros_like(l))
    part = torch.gather(ex, -1, at) * ok
    total = (ex if score == "softmax" else part).sum(-1, keepdim=True)
    total = torch.where(total == 0, torch.ones_like(total), total)
    w, g = part / total, grad.double() * ok
    inner, inner_abs = (w * g).sum(-1, keepdim=True), (w * g).abs().sum(-1, keepdim=True)
    p = ex / total if score == "softmax" else torch.zeros_like(ex).scatter_add_(-1, at, w)
    own = torch.zeros_like(ex).scatter_add_(-1, at, w * g)
    return own - p * inner, own.abs() + p * inner_abs


def run_gate(logits, k, score):
    R, T_r, _ = logits.shape
    idx = torch.full((R, T_r, k), -7, dtype=torch.int64, device="cuda")
    w = torch.full((R, T_r, k), 9.0, dtype=torch.float32, device="cuda")
    ep.ep_gate_topk(logits, ep.GATE_SCORES[score], idx, w)
    return idx, w


def draw(R, T_r, E, dtype, seed, ties=False):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((R, T_r, E), generator=g) * 2
    if ties:
        l = torch.round(l)   # few distinct values
    l = l.masked_fill(torch.rand((R, T_r, E), generator=g) < 0.1, -INF)
    return l.to(dtype)


@pytest.mark.parametrize("score", ["softmax", "softmax_topk"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,T_r,E,k", [(1, 1, 1, 1), (1, 3, 5, 5), (2, 17, 8, 2), (4, 16, 16, 2), (1, 33, 31, 7),
                                       (2, 9, 64, 8), (1, 20, 100, 6), (8, 13, 128, 6), (16, 9, 256, 8),
                                       (1, 11, 257, 16), (2, 5, 512, 16), (4, 4, 1000, 3), (1024, 1, 1024, 16)])
def test_gate_matches_definition(R, T_r, E, k, dtype, score):
    for ties in (False, True):
        l = draw(R, T_r, E, dtype, seed=E + k, ties=ties)
        idx, w = run_gate(l.cuda(), k, score)
        ref_idx, ref_w = reference(l, k, score)
        assert torch.equal(idx.cpu(), ref_idx)
        assert ((w.cpu().double() - ref_w).abs() <= 6e-6 * ref_w).all()


@pytest.mark.parametrize("score", ["softmax", "softmax_topk"])
def test_gate_special_values(score):
    low = torch.finfo(torch.float32).min
    rows = torch.tensor([
        [-INF] * 6,                                  # nothing to choose
        [-INF, -INF, 3.0, -INF, -INF, -INF],          # one expert left
        [math.nan] * 6,                              # nothing but NaN
        [math.nan, 1.0, math.nan, 2.0, -INF, 0.0],    # NaN beside numbers
        [low] * 6,                                   # the type's lowest value is a number
        [low, 0.0, low, -INF, low, 1.0],
        [INF, 0.0, INF, 1.0, -INF, 2.0],              # infinities share the weight
        [0.0, -0.0, 0.0, -0.0, 0.0, -0.0],            # signed zeros tie
        [1e-45, -1e-45, 0.0, 1e-40, -1e-40, 0.0],
        [88.0, -88.0, 200.0, -200.0, 199.0, 0.0],
    ]).reshape(1, -1, 6)
    idx, w = run_gate(rows.cuda(), 4, score)
    ref_idx, ref_w = reference(rows, 4, score)
    assert torch.equal(idx.cpu(), ref_idx)
    assert torch.isfinite(w).all()
    assert ((w.cpu().double() - ref_w).abs() <= 6e-6 * ref_w + 1e-37).all()


@pytest.mark.parametrize("score", ["softmax", "softmax_topk"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,T_r,E,k", [(1, 1, 1, 1), (2, 17, 8, 2), (1, 33, 31, 7), (2, 9, 64, 8), (8, 13, 128, 6),
                                       (16, 9, 256, 8), (1, 11, 257, 16), (2, 5, 512, 16), (1, 9, 1024, 16)])
def test_gate_backward_matches_formula(R, T_r, E, k, dtype, score):
    l = draw(R, T_r, E, dtype, seed=3 * E + k)
    l[0, 0] = -INF   # a token with no expert
    idx, _ = reference(l, k, score)
    g = torch.randn((R, T_r, k), generator=torch.Generator().manual_seed(5))
    out = torch.full_like(l, 3.0).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_gate_topk_backward(l.cuda(), ep.GATE_SCORES[score], idx.cuda(), g.cuda(), out, st)
    ref, mag = reference_grad(l, idx, g, score)
    tol = 2e-5 * mag + (0 if dtype == torch.float32 else 2.0 ** -8 * ref.abs()) + 1e-40
    assert ((out.cpu().double() - ref).abs() <= tol).all()
    assert ep.ep_read_status(st) == ep.EP_OK


@pytest.mark.parametrize("score", ["softmax", "softmax_topk"])
def test_gate_backward_matches_differences(score):
    """sum(grad * weights) moved along one logit at a time: central differences
    of the forward kernel.  Step 2^-6: the quotient's own error is step^2/6 of
    a third derivative below 2 (8e-5) and 2 * 6e-6 * |grad| k / (2 step)."""
    E, k, step = 24, 4, 2.0 ** -6
    l = torch.randn((1, 1, E), generator=torch.Generator().manual_seed(2)).cuda() * 2
    g = torch.randn((1, 1, k), generator=torch.Generator().manual_seed(3)).cuda()
    idx, _ = run_gate(l, k, score)
    out = torch.empty_like(l)
    ep.ep_gate_topk_backward(l, ep.GATE_SCORES[score], idx, g, out)
    for e in range(E):
        vals = []
        for sgn in (1, -1):
            m = l.clone()
            m[0, 0, e] += sgn * step
            i2, w2 = run_gate(m, k, score)
            dense = torch.zeros(E, dtype=torch.float64, device="cuda").scatter_(0, i2[0, 0], w2[0, 0].double())
            if set(i2[0, 0].tolist()) != set(idx[0, 0].tolist()):
                vals = None
                break
            vals.append(float((dense[idx[0, 0]] * g[0, 0].double()).sum()))
        if vals is not None:
            assert abs((vals[0] - vals[1]) / (2 * step) - float(out[0, 0, e])) < 2e-3


def test_gate_backward_refuses_bad_ids():
    l = torch.randn((1, 4, 8), device="cuda")
    idx = torch.tensor([[0, 1], [8, 2], [-2, 3], [5, -1]], device="cuda").reshape(1, 4, 2)
    g = torch.ones((1, 4, 2), device="cuda")
    out = torch.empty_like(l)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_gate_topk_backward(l, ep.EP_GATE_SOFTMAX_TOPK, idx, g, out, st)
    assert ep.ep_read_status(st) == ep.EP_ERR_INVALID_ARG
    clean = idx.masked_fill((idx < -1) | (idx >= 8), -1).cpu()
    ref, mag = reference_grad(l.cpu(), clean, g.cpu(), "softmax_topk")
    assert ((out.cpu().double() - ref).abs() <= 2e-5 * mag + 1e-40).all()


def test_gate_many_tokens_and_stream():
    """More tokens than one wave of warps, on a side stream; every token of a
    row-repeated batch has the same result."""
    l = draw(1, 7, 160, torch.float32, seed=1)
    big = l.repeat(1, 20011, 1).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    idx = torch.empty((1, big.shape[1], 6), dtype=torch.int64, device="cuda")
    w = torch.empty((1, big.shape[1], 6), dtype=torch.float32, device="cuda")
    ep.ep_gate_topk(big, ep.EP_GATE_SOFTMAX, idx, w, stream=s)
    s.synchronize()
    ref_idx, _ = reference(l, 6, "softmax")
    assert torch.equal(idx.view(20011, 7, 6).cpu(), ref_idx.expand(20011, 7, 6))
    assert torch.equal(w.view(20011, 7, 6), w[:, :7].expand(20011, 7, 6))


def test_gate_empty_batch_and_refusals():
    before = ep.ep_launch_count()
    i0 = torch.empty((2, 0, 2), dtype=torch.int64, device="cuda")
    w0 = torch.empty((2, 0, 2), dtype=torch.float32, device="cuda")
    ep.ep_gate_topk(torch.empty((2, 0, 8), device="cuda"), 0, i0, w0)
    l = torch.randn((2, 3, 8), device="cuda")
    i, w = (torch.empty((2, 3, 2), dtype=t, device="cuda") for t in (torch.int64, torch.float32))
    for bad in (lambda: ep.ep_gate_topk(l.half(), 0, i, w), lambda: ep.ep_gate_topk(l[..., ::2], 0, i, w),
                lambda: ep.ep_gate_topk(l, 0, i.int(), w), lambda: ep.ep_gate_topk(l, 0, i, w[:, :2]),
                lambda: ep.ep_gate_topk_backward(l, 0, i, w, l.bfloat16())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ep.EPError):
        ep.ep_gate_topk(l, 2, i, w)   # no such score
    with pytest.raises(ep.EPError):   # k > E
        ep.ep_gate_topk(l[..., :1].contiguous(), 0, i, w)
    with pytest.raises(ep.EPError):   # E not a multiple of R
        ep.ep_gate_topk(l[..., :7].contiguous(), 0, i, w)
    assert ep.ep_launch_count() == before


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(5, 3), (33, 1), (64, 8), (100, 4), (128, 8), (250, 7), (256, 8), (256, 12), (300, 8)])
def test_gate_unlike_neighbours(E, k, dtype):
    """Tokens side by side (an odd number of them) that take different ways: few and
    many candidates, all equal, switched off, infinite."""
    g = torch.Generator().manual_seed(E * 16 + k)
    rows = torch.randn((61, E), generator=g)
    rows[1::8] = 2.5                                  # every expert ties
    rows[2::8] = -INF
    rows[3::8, 1:] = -INF                             # one expert left
    rows[4::8] = torch.linspace(-3, 3, E)             # the largest in the last lanes
    rows[5::8] = torch.linspace(3, -3, E)
    rows[6::8, :: max(1, E // 40)] = 5.0              # some forty equal largest
    rows[7::16, E // 2] = INF
    rows[15::16, :2] = math.nan
    rows = rows.to(dtype)[None]
    for score in ("softmax", "softmax_topk"):
        idx, w = run_gate(rows.cuda(), k, score)
        ref_idx, ref_w = reference(rows, k, score)
        assert torch.equal(idx.cpu(), ref_idx)
        assert torch.isfinite(w).all()
        assert ((w.cpu().double() - ref_w).abs() <= 6e-6 * ref_w + 1e-37).all()
