"""The experts' products where their rings wrap and their offsets grow: many
tiles and long contractions on few SMs, hundreds of experts, rows past 2^31
elements.  Tolerances as in test_gpu_expert.py: n 2^-24 of the terms' magnitudes
for a sum of n, 2^-8 for the rounding to bf16."""
import numpy as np
import pytest
import torch

from combine_get_dispatch_gb300 import ep

pytestmark = pytest.mark.gpu


def near(got, ref, tol):
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"off by {float((err - tol).max()):.3g} over the tolerance"


def normal(counts, width, seed):
    """One rank's rows, segments back to back."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((1, int(sum(counts)), width), generator=g, device="cuda").bfloat16()


def tables(counts):
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    ps = torch.tensor([[0] + np.cumsum(counts).tolist()], dtype=torch.int64, device="cuda")
    return c, ps


@pytest.mark.parametrize("sms", [2, 0])
@pytest.mark.parametrize("counts,K,N", [([3000], 1000, 2056), ([700, 0, 513, 1, 1300], 1544, 776),
                                        ([2049] * 3, 72, 4104)])
def test_many_tiles(counts, K, N, sms):
    """One pair of SMs (then all) through some hundred tiles in every direction."""
    E = len(counts)
    g = torch.Generator(device="cuda").manual_seed(9)
    x, d = normal(counts, K, 1), normal(counts, N, 2)
    w = (torch.randn((E, N, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
    c, ps = tables(counts)
    y, dx, dw = torch.empty_like(d), torch.empty_like(x), torch.empty_like(w)
    ep.ep_set_num_sms(sms)
    try:
        ep.ep_expert_linear(x, None, w, None, None, None, c, ps, ep.EP_ACT_NONE, y)
        ep.ep_expert_linear_backward(d, None, x, w, c, ps, ep.EP_ACT_NONE, None, dx, dw)
        torch.cuda.synchronize()
    finally:
        ep.ep_set_num_sms(0)
    at = 0
    for e, n in enumerate(counts):
        xe, de, we = x[0, at:at + n].double(), d[0, at:at + n].double(), w[e].double()
        for got, a, b in ((y[0, at:at + n], xe, we.t()), (dx[0, at:at + n], de, we), (dw[e], de.t(), xe)):
            r = a @ b
            near(got, r, 2.0 ** -8 * r.abs() + a.shape[1] * 2.0 ** -24 * (a.abs() @ b.abs()) + 1e-30)
        at += n


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("E,N,most", [(3, 200, 2100), (24, 1096, 700), (56, 4104, 300)])
def test_bias_gradient_split(E, N, most, act):
    """An expert's rows summed by 8 CTAs, by 2 and by one; uneven segments, none and
    one row among them.  The slope of SiLU and its product are within 2^-18."""
    rng = np.random.default_rng(E)
    counts = rng.integers(0, most, E).tolist()
    counts[0], counts[1], counts[2] = 0, most, 1
    dy = normal(counts, N, 1)
    pre = normal(counts, N, 2) if act != "none" else None
    dpre = torch.empty_like(dy) if act != "none" else None
    c, ps = tables(counts)
    db = torch.full((E, N), -77.0, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((E, N, 8), dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_linear_backward(dy, pre, None, w, c, ps, ep.ACTS[act], dpre, None, None, dbias=db)
    at = 0
    for e, n in enumerate(counts):
        d, e_d = dy[0, at:at + n].double(), 0.0
        if pre is not None:
            z = pre[0, at:at + n].double()
            q = torch.sigmoid(z)
            e_d = 2.0 ** -18 * d.abs()
            d = d * (q * (1 + z * (1 - q)))
            near(dpre[0, at:at + n], d, 2.0 ** -8 * d.abs() + e_d)
        s = d.sum(0)
        near(db[e], s, 2.0 ** -8 * s.abs() + (n * 2.0 ** -24 * d.abs() + e_d).sum(0) + 1e-30)
        at += n


def test_a_thousand_experts():
    """1024 experts of 0 to 40 rows on 4 ranks, gated, forward and weights' gradient."""
    rng = np.random.default_rng(4)
    R, E, H, I = 4, 1024, 72, 40
    counts = rng.integers(0, 41, E) * (rng.random(E) < 0.7)
    per = counts.reshape(R, -1)
    ps = np.concatenate([np.zeros((R, 1), np.int64), np.cumsum(per, 1)], 1)
    cap = int(ps[:, -1].max()) + 7
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((R, cap, H), generator=g, device="cuda").bfloat16()
    w = (torch.randn((E, 2, I, H), generator=g, device="cuda") * H ** -0.5).bfloat16()
    c, psum = torch.tensor(per, dtype=torch.int32, device="cuda"), torch.tensor(ps, device="cuda")
    h, gu = torch.zeros((R, cap, I), dtype=torch.bfloat16, device="cuda"), torch.zeros((R, cap, 2, I), dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_glu(x, None, w, None, c, psum, ep.EP_ACT_SILU, h, gu=gu)
    dw = torch.full_like(w, 7.0)
    ep.ep_expert_linear_backward(gu.reshape(R, cap, 2 * I), None, x, None, c, psum, ep.EP_ACT_NONE, None, None,
                                 dw.view(E, 2 * I, H))
    for e in range(E):
        r, a = e // (E // R), int(ps[e // (E // R), e % (E // R)])
        xe = x[r, a:a + counts[e]].double()
        z = torch.einsum("nh,gih->ngi", xe, w[e].double())
        near(gu[r, a:a + counts[e]], z, 2.0 ** -8 * z.abs() + H * 2.0 ** -24 * torch.einsum("nh,gih->ngi", xe.abs(), w[e].double().abs()))
        d = gu[r, a:a + counts[e]].double().reshape(-1, 2 * I)
        ref = d.t() @ xe
        near(dw[e].reshape(2 * I, H), ref, 2.0 ** -8 * ref.abs() + 64 * 2.0 ** -24 * (d.abs().t() @ xe.abs()))
    free = torch.ones((R, cap), dtype=torch.bool, device="cuda")
    for e in range(E):
        r, a = e // (E // R), int(ps[e // (E // R), e % (E // R)])
        free[r, a:a + counts[e]] = False
    assert not h[free].any() and not gu[free].any()


def test_rows_past_two_billion_elements():
    """A segment that lies wholly past element 2^31 of its layout, in every
    direction, and nothing else written."""
    H, I, cap, n = 8192, 64, 300_000, 75
    start = cap - n - 3
    assert start * H > 2 ** 31
    x = torch.zeros((1, cap, H), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(6)
    x[0, start:start + n] = torch.randn((n, H), generator=g, device="cuda").bfloat16()
    w = (torch.randn((1, I, H), generator=g, device="cuda") * H ** -0.5).bfloat16()
    c = torch.tensor([n], dtype=torch.int32, device="cuda")
    ps = torch.tensor([[start, start + n]], dtype=torch.int64, device="cuda")
    y = torch.zeros((1, cap, I), dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_linear(x, None, w, None, None, None, c, ps, ep.EP_ACT_NONE, y)
    xe, we = x[0, start:start + n].double(), w[0].double()
    r = xe @ we.t()
    near(y[0, start:start + n], r, 2.0 ** -8 * r.abs() + H * 2.0 ** -24 * (xe.abs() @ we.abs().t()))
    dx, dw = torch.zeros_like(x), torch.empty_like(w)
    ep.ep_expert_linear_backward(y, None, x, w, c, ps, ep.EP_ACT_NONE, None, dx, dw)
    d = y[0, start:start + n].double()
    r = d @ we
    near(dx[0, start:start + n], r, 2.0 ** -8 * r.abs() + I * 2.0 ** -24 * (d.abs() @ we.abs()))
    r = d.t() @ xe
    near(dw[0], r, 2.0 ** -8 * r.abs() + n * 2.0 ** -24 * (d.abs().t() @ xe.abs()))
    assert not dx[0, :start].any() and not dx[0, start + n:].any() and not y[0, :start].any() and not y[0, start + n:].any()


def test_inputs_made_on_another_stream():
    """Rows and counts written by kernels of a side stream right before the call
    on that stream: the call comes up early and has to wait for them."""
    counts, H, I = [300, 45], 256, 264
    c, ps = tables(counts)
    src = normal(counts, H, 3)
    w = (torch.randn((2, 2, I, H), device="cuda") * H ** -0.5).bfloat16()
    want, h = (torch.zeros((1, 345, I), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ep.ep_expert_glu(src, None, w, None, c, ps, ep.EP_ACT_SILU, want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(20):
            x, c2 = torch.zeros_like(src), torch.zeros_like(c)
            h.zero_()
            torch.cuda._sleep(200_000)
            x.copy_(src)
            c2.copy_(c)
            ep.ep_expert_glu(x, None, w, None, c2, ps, ep.EP_ACT_SILU, h)
            h2 = h.clone()
            s.synchronize()
            assert torch.equal(h2.view(torch.int16), want.view(torch.int16))
