"""The experts' products over a receive layout, and their gradients, against
plain 64-bit products.

Tolerances, element by element.  Products of two bf16 (or E4M3) values are
exact in fp32 and a sum of n of them in any order is off by at most
n 2^-24 S, S the sum of the terms' magnitudes (tensor cores that align addends
before adding lose no more than one such unit per step); a power-of-two scale
is exact.  The output's rounding to bf16 (8 significant bits) adds at most
2^-8 of it.  Behind an activation the error is multiplied by its largest slope
(1.13 for SiLU and GELU) and the function itself is within 2^-18 of its value.
The products of the gradients take dgu / dpre as the calls return them, rounded
to bf16 (that is their definition): the references do the same, after checking
them."""
import math

import numpy as np
import pytest
import torch

from combine_get_dispatch_gb300 import ep

pytestmark = pytest.mark.gpu

POISON = -77.0
ACTS = ["relu", "silu", "gelu"]


def act64(z, name):
    if name == "silu":
        q = torch.sigmoid(z)
        return z * q, q * (1 + z * (1 - q))
    if name == "gelu":
        c = 0.5 * (1 + torch.erf(z / math.sqrt(2)))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    return z, torch.ones_like(z)


class Layout:
    """Segments of `counts` (one list per rank) in the normal (aligned, NaN
    between) or packed layout."""

    def __init__(self, counts, packed=False, align=1, slack=5, cap=None):
        self.counts = np.array(counts, dtype=np.int32)
        R, E_l = self.counts.shape
        self.R, self.E, self.packed = R, R * E_l, packed
        if packed:
            self.cap = cap if cap is not None else int(self.counts.max()) + slack
            self.lead = (R, E_l, self.cap)
            self.starts = np.arange(self.E) * self.cap
            self.psum = None
        else:
            al = -(-self.counts // align) * align
            ps = np.concatenate([np.zeros((R, 1), np.int64), np.cumsum(al, 1)], 1)
            self.cap = cap if cap is not None else int(ps[:, -1].max()) + slack
            self.lead = (R, self.cap)
            self.starts = (ps[:, :-1] + np.arange(R)[:, None] * self.cap).reshape(-1)
            self.psum = torch.from_numpy(ps.astype(np.int64)).cuda()
        self.dcounts = torch.from_numpy(self.counts).cuda()
        self.rows = int(np.prod(self.lead))
        self.free = torch.ones(self.rows, dtype=torch.bool)
        for a, n in self.each():
            self.free[a:a + n] = False
        self.free = self.free.cuda()

    def each(self):
        return [(int(a), int(n)) for a, n in zip(self.starts, self.counts.reshape(-1))]

    def randn(self, width, seed, std=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = (torch.randn((self.rows, width), generator=g, device="cuda") * std).bfloat16()
        t[self.free] = math.nan
        return t.reshape(*self.lead, width)

    def out(self, *width, dtype=torch.bfloat16):
        return torch.full((*self.lead, *width), POISON if dtype == torch.bfloat16 else 0x5A, dtype=dtype, device="cuda")

    def untouched(self, t):
        u = t.reshape(self.rows, -1)[self.free]
        return bool((u == (POISON if t.dtype == torch.bfloat16 else 0x5A)).all())


def weights(E, shape, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((E, *shape), generator=g, device="cuda") / math.sqrt(K)).bfloat16()


def near(got, ref, tol):
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"off by {float((err - tol).max()):.3g} over the tolerance"


LAYOUTS = {
    "dense_1": dict(counts=[[1]]),
    "dense_300": dict(counts=[[300]]),
    "ragged": dict(counts=[[0, 1, 127, 128], [129, 0, 5, 257]]),
    "aligned": dict(counts=[[3, 0, 130], [255, 64, 0], [1, 1, 1]], align=128),
    "packed": dict(counts=[[7, 0, 200], [256, 33, 1]], packed=True),
    "empty": dict(counts=[[0, 0], [0, 0]]),
}
# (inner or hidden, output or intermediate) widths around the tiles' edges
WIDTHS = [(8, 8), (64, 128), (72, 40), (200, 136), (256, 264), (1000, 520)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("H,I", WIDTHS)
@pytest.mark.parametrize("name", LAYOUTS)
def test_glu_forward(name, H, I, act):
    L = Layout(**LAYOUTS[name])
    x, w = L.randn(H, 1), weights(L.E, (2, I, H), H, 2)
    h, gu = L.out(I), L.out(2, I)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_expert_glu(x, None, w, None, L.dcounts, L.psum, ep.ACTS[act], h, gu=gu, status=st)
    h2 = L.out(I)
    ep.ep_expert_glu(x, None, w, None, L.dcounts, L.psum, ep.ACTS[act], h2)
    assert ep.ep_read_status(st) == ep.EP_OK
    assert torch.equal(h.view(torch.int16), h2.view(torch.int16))
    assert L.untouched(h) and L.untouched(gu)
    fx, fh, fg = x.reshape(L.rows, H), h.reshape(L.rows, I), gu.reshape(L.rows, 2, I)
    for e, (a, n) in enumerate(L.each()):
        xe, we = fx[a:a + n].double(), w[e].double()
        g, u = xe @ we[0].t(), xe @ we[1].t()
        sg, su = (H * 2.0 ** -24 * (xe.abs() @ we[i].abs().t()) for i in (0, 1))
        near(fg[a:a + n, 0], g, 2.0 ** -8 * g.abs() + sg)
        near(fg[a:a + n, 1], u, 2.0 ** -8 * u.abs() + su)
        v = act64(g, act)[0]
        near(fh[a:a + n], v * u, 2.0 ** -8 * (v * u).abs() + 1.13 * sg * (u.abs() + su) + v.abs() * su + 1e-30)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("H,I", WIDTHS)
@pytest.mark.parametrize("name", LAYOUTS)
def test_glu_backward(name, H, I, act):
    L = Layout(**LAYOUTS[name])
    x, w = L.randn(H, 1), weights(L.E, (2, I, H), H, 2)
    dh, gu = L.randn(I, 3), L.randn(2 * I, 4).reshape(*L.lead, 2, I)
    dgu, dx = L.out(2, I), L.out(H)
    dw = torch.full((L.E, 2, I, H), POISON, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_glu_backward(dh, gu, x, w, L.dcounts, L.psum, ep.ACTS[act], dgu, dx, dw)
    assert L.untouched(dgu) and L.untouched(dx)
    for e, (a, n) in enumerate(L.each()):
        at = slice(a, a + n)
        g, u = (gu.reshape(L.rows, 2, I)[at, i].double() for i in (0, 1))
        d = dh.reshape(L.rows, I)[at].double()
        v, s = act64(g, act)
        ref = torch.cat([d * u * s, d * v], 1)
        near(dgu.reshape(L.rows, -1)[at], ref, 2.0 ** -8 * ref.abs() + 2.0 ** -18 * torch.cat([(d * u).abs(), d.abs()], 1))
        check_gradients(dgu.reshape(L.rows, -1)[at].double(), x.reshape(L.rows, H)[at].double(),
                        w[e].reshape(2 * I, H).double(), dx.reshape(L.rows, H)[at], dw[e].reshape(2 * I, H))
    # in place of gu, and each gradient by itself, give the same bits
    own, dx2, dw2 = gu.clone(), L.out(H), torch.empty_like(dw)
    ep.ep_expert_glu_backward(dh, own, None, w, L.dcounts, L.psum, ep.ACTS[act], own, dx2, None)
    ep.ep_expert_glu_backward(dh, gu, x, None, L.dcounts, L.psum, ep.ACTS[act], dgu, None, dw2)
    assert torch.equal(dx.view(torch.int16), dx2.view(torch.int16))
    assert torch.equal(dw.view(torch.int16), dw2.view(torch.int16))


def check_gradients(d, x, w, dx, dw):
    """dx = d W, dw = d^T x of the d that the call returned."""
    n, N = d.shape
    r = d @ w
    near(dx, r, 2.0 ** -8 * r.abs() + N * 2.0 ** -24 * (d.abs() @ w.abs()) + 1e-30)
    r = d.t() @ x
    near(dw, r, 2.0 ** -8 * r.abs() + n * 2.0 ** -24 * (d.abs().t() @ x.abs()) + 1e-30)


@pytest.mark.parametrize("act,bias,residual", [("none", False, False), ("none", True, True), ("relu", True, False),
                                               ("silu", False, True), ("gelu", True, True)])
@pytest.mark.parametrize("K,N", WIDTHS)
@pytest.mark.parametrize("name", LAYOUTS)
def test_linear_forward(name, K, N, act, bias, residual):
    L = Layout(**LAYOUTS[name])
    x, w = L.randn(K, 1), weights(L.E, (N, K), K, 2)
    b = weights(L.E, (N,), 1, 5) if bias else None
    res = L.randn(N, 6) if residual else None
    y, pre = L.out(N), L.out(N)
    ep.ep_expert_linear(x, None, w, None, b, res, L.dcounts, L.psum, ep.ACTS[act], y, pre=pre)
    assert L.untouched(y) and L.untouched(pre)
    y2 = L.out(N) if res is None else res.clone()   # in place of the residual
    ep.ep_expert_linear(x, None, w, None, b, None if res is None else y2, L.dcounts, L.psum, ep.ACTS[act], y2)
    for e, (a, n) in enumerate(L.each()):
        at = slice(a, a + n)
        xe, we = x.reshape(L.rows, K)[at].double(), w[e].double()
        z = xe @ we.t() + (b[e].double() if bias else 0)
        sz = (K + 1) * 2.0 ** -24 * (xe.abs() @ we.abs().t() + (b[e].double().abs() if bias else 0))
        near(pre.reshape(L.rows, N)[at], z, 2.0 ** -8 * z.abs() + sz)
        v = act64(z, act)[0]
        r = v + (res.reshape(L.rows, N)[at].double() if residual else 0)
        near(y.reshape(L.rows, N)[at], r, 2.0 ** -8 * r.abs() + 1.13 * sz + 2.0 ** -18 * v.abs() + 1e-30)
        assert torch.equal(y.reshape(L.rows, N)[at].view(torch.int16), y2.reshape(L.rows, N)[at].view(torch.int16))


@pytest.mark.parametrize("act", ["none"] + ACTS)
@pytest.mark.parametrize("K,N", WIDTHS)
@pytest.mark.parametrize("name", LAYOUTS)
def test_linear_backward(name, K, N, act):
    L = Layout(**LAYOUTS[name])
    x, w = L.randn(K, 1), weights(L.E, (N, K), K, 2)
    dy = L.randn(N, 3)
    pre = L.randn(N, 4) if act != "none" else None
    dpre = L.out(N) if act != "none" else None
    dx = L.out(K)
    dw = torch.full((L.E, N, K), POISON, dtype=torch.bfloat16, device="cuda")
    db = torch.full((L.E, N), POISON, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_linear_backward(dy, pre, x, w, L.dcounts, L.psum, ep.ACTS[act], dpre, dx, dw, dbias=db)
    assert L.untouched(dx) and (dpre is None or L.untouched(dpre))
    for e, (a, n) in enumerate(L.each()):
        at = slice(a, a + n)
        d = dy.reshape(L.rows, N)[at].double()
        e_d = torch.zeros_like(d)
        if pre is not None:
            s = act64(pre.reshape(L.rows, N)[at].double(), act)[1]
            e_d = 2.0 ** -18 * d.abs()
            d = d * s
            near(dpre.reshape(L.rows, N)[at], d, 2.0 ** -8 * d.abs() + e_d)
        used = d if dpre is None else dpre.reshape(L.rows, N)[at].double()
        check_gradients(used, x.reshape(L.rows, K)[at].double(), w[e].double(), dx.reshape(L.rows, K)[at], dw[e])
        s = d.sum(0)
        near(db[e], s, 2.0 ** -8 * s.abs() + (n * 2.0 ** -24 * d.abs() + e_d).sum(0) + 1e-30)
    only = torch.empty_like(db)
    ep.ep_expert_linear_backward(dy, pre, None, w, L.dcounts, L.psum, ep.ACTS[act], dpre, None, None, dbias=only)
    assert torch.equal(only.view(torch.int16), db.view(torch.int16))


def test_gradients_match_differences():
    """Directional differences, in 64 bits, of sum(dh * h) and sum(dy * y): a
    step t along a random direction changes the sum by t <grad, direction> +
    O(t^3).  The kernels' gradients carry bf16 roundings, of 2^-8 at most each:
    gate and up as they were kept, the operand, the result.  Their signs are
    random, so <grad, direction> stays far within 2^-7 of the sum of the
    terms' magnitudes."""
    L = Layout(counts=[[40, 0, 9]])
    H, I = 96, 72
    x, w = L.randn(H, 1), weights(L.E, (2, I, H), H, 2)
    dh = L.randn(I, 3)
    h, gu = L.out(I), L.out(2, I)
    for act in ("silu", "gelu"):
        ep.ep_expert_glu(x, None, w, None, L.dcounts, L.psum, ep.ACTS[act], h, gu=gu)
        dgu, dx, dw = L.out(2, I), L.out(H), torch.empty_like(w)
        ep.ep_expert_glu_backward(dh, gu, x, w, L.dcounts, L.psum, ep.ACTS[act], dgu, dx, dw)
        vx, vw = torch.randn_like(x, dtype=torch.float64), torch.randn_like(w, dtype=torch.float64)

        def loss(t, sx, sw):
            total = 0.0
            for e, (a, n) in enumerate(L.each()):
                at = slice(a, a + n)
                xe = x.reshape(L.rows, H)[at].double() + t * sx * vx.reshape(L.rows, H)[at]
                we = w[e].double() + t * sw * vw[e]
                total += float((act64(xe @ we[0].t(), act)[0] * (xe @ we[1].t()) * dh.reshape(L.rows, I)[at].double()).sum())
            return total

        t = 1e-5
        ok = ~L.free
        terms = dx.reshape(L.rows, H)[ok].double() * vx.reshape(L.rows, H)[ok]
        assert abs((loss(t, 1, 0) - loss(-t, 1, 0)) / (2 * t) - float(terms.sum())) < 2.0 ** -7 * float(terms.abs().sum())
        terms = dw.double() * vw
        assert abs((loss(t, 0, 1) - loss(-t, 0, 1)) / (2 * t) - float(terms.sum())) < 2.0 ** -7 * float(terms.abs().sum())


def e4m3(shape, seed, lo, hi, K):
    """E4M3 bytes and random power-of-two scales (one byte per block)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn(shape, generator=g, device="cuda") * 90).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return q, lambda s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.uint8)


def dequant_rows(q, sc, L, K):
    blocks = sc.reshape(-1, K // 128, L.cap).permute(0, 2, 1).reshape(L.rows, K // 128)
    return q.reshape(L.rows, K).view(torch.float8_e4m3fn).double() * (2.0 ** (blocks.double() - 127)).repeat_interleave(128, 1)


FP8_WIDTHS = [(128, 128), (256, 384), (1152, 256), (2048, 640)]


@pytest.mark.parametrize("K,N", FP8_WIDTHS)
@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("out8", [False, True])
def test_glu_e4m3(name, K, N, out8):
    L = Layout(**LAYOUTS[name])
    x, sx = e4m3((*L.lead, K), 1, 115, 125, K)
    x.reshape(L.rows, K)[L.free] = 0x7F
    w, sw = e4m3((L.E, 2, N, K), 2, 110, 116, K)
    xs, ws = sx((*L.lead[:-1], K // 128, L.cap)), sw((L.E, 2, N // 128, K // 128))
    h = L.out(N, dtype=torch.uint8 if out8 else torch.bfloat16)
    hs = torch.full((*L.lead[:-1], N // 128, L.cap), 0x5A, dtype=torch.uint8, device="cuda") if out8 else None
    ep.ep_expert_glu(x, xs, w, ws, L.dcounts, L.psum, ep.EP_ACT_SILU, h, h_scales=hs)
    assert L.untouched(h)
    xd = dequant_rows(x, xs, L, K)
    hd = dequant_rows(h, hs, L, N) if out8 else h.reshape(L.rows, N)
    for e, (a, n) in enumerate(L.each()):
        wd = w[e].view(torch.float8_e4m3fn).double() * (2.0 ** (ws[e].double() - 127)).repeat_interleave(128, 1).repeat_interleave(128, 2)
        xe = xd[a:a + n]
        g, u = xe @ wd[0].t(), xe @ wd[1].t()
        sg, su = (K * 2.0 ** -24 * (xe.abs() @ wd[i].abs().t()) for i in (0, 1))
        v = act64(g, "silu")[0]
        ref = v * u
        err = 2.0 ** -18 * ref.abs() + 1.13 * sg * (u.abs() + su) + v.abs() * su
        if not out8:
            near(hd[a:a + n], ref, err + 2.0 ** -8 * ref.abs() + 1e-30)
        elif n:
            # a block's scale is a power of two at least amax / 448; half an E4M3 step is 2^-4 of a normal value and
            # 2^-10 of the scale below; a block at a power's edge may take the next one
            amax = ref.abs().reshape(n, -1, 128).amax(-1).clamp(min=1e-4)
            up = torch.exp2(torch.ceil(torch.log2(amax / 448 * (1 + 2.0 ** -12)))).repeat_interleave(128, 1)
            near(hd[a:a + n], ref, err * 1.07 + 2.0 ** -4 * ref.abs() + 2.0 ** -10 * up)
    if out8 and not L.packed and not L.free.all():
        flat = hs.reshape(-1, N // 128, L.cap).permute(0, 2, 1).reshape(L.rows, N // 128)
        assert bool((flat[L.free] == 0x5A).all())


@pytest.mark.parametrize("K,N", FP8_WIDTHS)
@pytest.mark.parametrize("name", LAYOUTS)
def test_linear_e4m3(name, K, N):
    L = Layout(**LAYOUTS[name])
    x, sx = e4m3((*L.lead, K), 1, 100, 140, K)
    x.reshape(L.rows, K)[L.free] = 0x7F
    w, sw = e4m3((L.E, N, K), 2, 100, 116, K)
    xs, ws = sx((*L.lead[:-1], K // 128, L.cap)), sw((L.E, N // 128, K // 128))
    b, res = weights(L.E, (N,), 1, 5), L.randn(N, 6)
    y = L.out(N)
    ep.ep_expert_linear(x, xs, w, ws, b, res, L.dcounts, L.psum, ep.EP_ACT_NONE, y)
    assert L.untouched(y)
    xd = dequant_rows(x, xs, L, K)
    for e, (a, n) in enumerate(L.each()):
        wd = w[e].view(torch.float8_e4m3fn).double() * (2.0 ** (ws[e].double() - 127)).repeat_interleave(128, 0).repeat_interleave(128, 1)
        xe = xd[a:a + n]
        r = xe @ wd.t() + b[e].double() + res.reshape(L.rows, N)[a:a + n].double()
        s = xe.abs() @ wd.abs().t() + b[e].double().abs() + res.reshape(L.rows, N)[a:a + n].double().abs()
        near(y.reshape(L.rows, N)[a:a + n], r, 2.0 ** -8 * r.abs() + (K + 2) * 2.0 ** -24 * s)


@pytest.mark.parametrize("packed", [False, True])
def test_segments_past_the_buffer_are_cut(packed):
    """counts that do not fit: rows up to cap_rows are computed, nothing past
    them is written, and the status word says so."""
    L = Layout(counts=[[20, 30], [10, 5]], packed=packed, slack=0)
    H, I = 64, 64
    x, w = L.randn(H, 1), weights(L.E, (2, I, H), H, 2)
    h, ref = L.out(I), L.out(I)
    ep.ep_expert_glu(x, None, w, None, L.dcounts, L.psum, ep.EP_ACT_SILU, ref)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    more = L.dcounts.clone()
    more[0, 1] += 1000    # the last segment of rank 0: reaches over the end
    ep.ep_expert_glu(x, None, w, None, more, L.psum, ep.EP_ACT_SILU, h, status=st)
    assert ep.ep_read_status(st) == ep.EP_ERR_CAPACITY
    ok = ~L.free
    assert torch.equal(h.reshape(L.rows, I)[ok].view(torch.int16), ref.reshape(L.rows, I)[ok].view(torch.int16))
    assert L.untouched(h)


def test_many_experts_side_stream_and_graph():
    """512 experts of 0..3 rows; on a side stream and replayed as a graph."""
    rng = np.random.default_rng(3)
    L = Layout(counts=rng.integers(0, 4, (2, 256)).tolist())
    H, I = 64, 72
    x, w = L.randn(H, 1), weights(L.E, (2, I, H), H, 2)
    want, h = L.out(I), L.out(I)
    ep.ep_expert_glu(x, None, w, None, L.dcounts, L.psum, ep.EP_ACT_RELU, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ep.ep_expert_glu(x, None, w, None, L.dcounts, L.psum, ep.EP_ACT_RELU, h, stream=s)
    s.synchronize()
    assert torch.equal(h.view(torch.int16), want.view(torch.int16))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ep.ep_expert_glu(x, None, w, None, L.dcounts, L.psum, ep.EP_ACT_RELU, h)
    for _ in range(2):
        h.fill_(POISON)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(h.view(torch.int16), want.view(torch.int16))
    fx, fh = x.reshape(L.rows, H), h.reshape(L.rows, I)
    for e, (a, n) in enumerate(L.each()):
        xe, we = fx[a:a + n].double(), w[e].double()
        g1, u = xe @ we[0].t(), xe @ we[1].t()
        sg, su = (H * 2.0 ** -24 * (xe.abs() @ we[i].abs().t()) for i in (0, 1))
        v = g1.clamp(min=0)
        near(fh[a:a + n], v * u, 2.0 ** -8 * (v * u).abs() + sg * (u.abs() + su) + v * su + 1e-30)


def test_sm_budget_gives_the_same_result():
    L = Layout(counts=[[300, 0, 77]])
    H, I = 200, 136
    x, w = L.randn(H, 1), weights(L.E, (2, I, H), H, 2)
    a, b = L.out(I), L.out(I)
    ep.ep_expert_glu(x, None, w, None, L.dcounts, L.psum, ep.EP_ACT_SILU, a)
    ep.ep_set_num_sms(3)
    try:
        ep.ep_expert_glu(x, None, w, None, L.dcounts, L.psum, ep.EP_ACT_SILU, b)
        torch.cuda.synchronize()
    finally:
        ep.ep_set_num_sms(0)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_refusals():
    before = ep.ep_launch_count()
    L = Layout(counts=[[3, 2]])
    H, I = 128, 128
    x, w, h = L.randn(H, 1), weights(L.E, (2, I, H), H, 2), L.out(I)
    c, ps, silu = L.dcounts, L.psum, ep.EP_ACT_SILU
    q, xs = torch.zeros_like(x, dtype=torch.uint8), torch.zeros((1, 1, L.cap), dtype=torch.uint8, device="cuda")
    wq, ws = torch.zeros_like(w, dtype=torch.uint8), torch.zeros((2, 2, 1, 1), dtype=torch.uint8, device="cuda")
    for bad in (
            lambda: ep.ep_expert_glu(x.float(), None, w, None, c, ps, silu, h),
            lambda: ep.ep_expert_glu(x, None, w[:, :1], None, c, ps, silu, h),
            lambda: ep.ep_expert_glu(x, None, w.transpose(2, 3), None, c, ps, silu, h),
            lambda: ep.ep_expert_glu(x, None, w, None, c.long(), ps, silu, h),
            lambda: ep.ep_expert_glu(x, None, w, None, c, None, silu, h),          # packed, but rows are not
            lambda: ep.ep_expert_glu(x, None, w, None, c, ps.int(), silu, h),
            lambda: ep.ep_expert_glu(x, None, w, None, c, ps, silu, h[..., :64]),
            lambda: ep.ep_expert_glu(x, None, w, ws, c, ps, silu, h),
            lambda: ep.ep_expert_glu(q, xs, wq, ws[:, :1], c, ps, silu, h),
            lambda: ep.ep_expert_glu_backward(h, None, x, w, c, ps, silu, h, None, None),
            lambda: ep.ep_expert_linear(x, None, w, None, None, None, c, ps, 0, h),
            lambda: ep.ep_expert_linear(x, None, w[:, 0].contiguous(), None, c, None, c, ps, 0, h),
            lambda: ep.ep_expert_linear_backward(h, None, x, w[:, 0].contiguous(), c, ps, silu, None, None, None)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (
            lambda: ep.ep_expert_glu(x, None, w, None, c, ps, ep.EP_ACT_NONE, h),
            lambda: ep.ep_expert_glu(x, None, w, None, c, ps, 9, h),
            lambda: ep.ep_expert_glu(q, xs.float(), wq, ws, c, ps, silu, h),       # fp32 scales
            lambda: ep.ep_expert_glu(x, None, w, None, c, ps, silu, q, h_scales=xs),  # E4M3 out of bf16 rows
            lambda: ep.ep_expert_glu(x[..., :4].contiguous(), None, w[..., :4].contiguous(), None, c, ps, silu, h),
            lambda: ep.ep_expert_linear(x, None, w[:, 0].contiguous(), None, None, None, c, ps, 7, h)):
        with pytest.raises(ep.EPError):
            bad()
    assert ep.ep_launch_count() == before
