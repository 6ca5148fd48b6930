"""The E4M3 products where their rings wrap: hundreds of tiles on two SMs and
on all, inner blocks that the stages do not divide, every activation, output
quantised or not, pre-activation kept.

Tolerances as in test_gpu_expert.py: K 2^-24 of the terms' magnitudes for a sum of
K, 2^-8 for a rounding to bf16; a rounding to E4M3 is half a step, 2^-4 of a
normal value and 2^-10 of the block's scale below, and a block whose largest
value is at a power's edge may have taken the next scale.  An activation multiplies
its argument's error by 1.13 at most and is itself within 2^-15 of its value."""
import numpy as np
import pytest
import torch

from combine_get_dispatch_gb300 import ep
from test_gpu_expert import Layout, act64, dequant_rows, e4m3, near, weights

pytestmark = pytest.mark.gpu

COUNTS = [[300, 0, 513], [1, 257, 700]]


def on_both(call):
    """The outputs of `call` on two SMs and on all: the same bits."""
    few = None
    for sms in (2, 0):
        ep.ep_set_num_sms(sms)
        try:
            out = call()
            torch.cuda.synchronize()
        finally:
            ep.ep_set_num_sms(0)
        for a, b in zip(few or out, out):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        few = out
    return few


def dequant_weights(w, ws):
    return w.view(torch.float8_e4m3fn).double() * (2.0 ** (ws.double() - 127)).repeat_interleave(128, -2).repeat_interleave(128, -1)


def value64(z, act):
    return 0.5 * z * torch.special.erfc(z * -0.5 ** 0.5) if act == "gelu" else act64(z, act)[0]


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("out8", [False, True])
@pytest.mark.parametrize("K,N,packed", [(384, 1280, False), (640, 1152, True), (1152, 256, False)])
def test_glu_many_tiles(K, N, packed, out8, act):
    L = Layout(COUNTS, packed=packed, align=1 if packed else 16)
    x, sx = e4m3((*L.lead, K), 1, 115, 120, K)
    x.reshape(L.rows, K)[L.free] = 0x7F
    w, sw = e4m3((L.E, 2, N, K), 2, 118, 121, K)
    xs, ws = sx((*L.lead[:-1], K // 128, L.cap)), sw((L.E, 2, N // 128, K // 128))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        h = L.out(N, dtype=torch.uint8 if out8 else torch.bfloat16)
        hs = torch.full((*L.lead[:-1], N // 128, L.cap), 0x5A, dtype=torch.uint8, device="cuda") if out8 else None
        ep.ep_expert_glu(x, xs, w, ws, L.dcounts, L.psum, ep.ACTS[act], h, h_scales=hs, status=st)
        return (h, hs) if out8 else (h,)

    out = on_both(call)
    assert ep.ep_read_status(st) == ep.EP_OK
    h = out[0]
    assert L.untouched(h)
    if out8:
        per_row = out[1].reshape(-1, N // 128, L.cap).permute(0, 2, 1).reshape(L.rows, N // 128)
        assert bool((per_row[L.free] == 0x5A).all())
    xd = dequant_rows(x, xs, L, K)
    hd = dequant_rows(h, out[1], L, N) if out8 else h.reshape(L.rows, N)
    for e, (a, n) in enumerate(L.each()):
        if n == 0:
            continue
        xe, wd = xd[a:a + n], dequant_weights(w[e], ws[e])
        g, u = xe @ wd[0].t(), xe @ wd[1].t()
        sg, su = (K * 2.0 ** -24 * (xe.abs() @ wd[i].abs().t()) for i in (0, 1))
        v = value64(g, act)
        ref = v * u
        err = 2.0 ** -15 * ref.abs() + 1.13 * sg * (u.abs() + su) + v.abs() * su + 1e-30
        if out8:
            amax = ref.abs().reshape(n, -1, 128).amax(-1).clamp(min=1e-4)
            scale = torch.exp2(torch.ceil(torch.log2(amax / 448)) + 1).repeat_interleave(128, 1)
            near(hd[a:a + n], ref, err * 1.07 + 2.0 ** -4 * ref.abs() + 2.0 ** -10 * scale)
        else:
            near(hd[a:a + n], ref, err + 2.0 ** -8 * ref.abs())


@pytest.mark.parametrize("act,bias,residual", [("none", False, False), ("none", True, True), ("relu", True, False),
                                               ("silu", False, True), ("gelu", True, True)])
@pytest.mark.parametrize("K,N,packed", [(384, 1408, True), (640, 2176, False), (1152, 256, False)])
def test_linear_many_tiles(K, N, packed, act, bias, residual):
    L = Layout(COUNTS, packed=packed, align=1 if packed else 16)
    x, sx = e4m3((*L.lead, K), 1, 115, 120, K)
    x.reshape(L.rows, K)[L.free] = 0x7F
    w, sw = e4m3((L.E, N, K), 2, 118, 121, K)
    xs, ws = sx((*L.lead[:-1], K // 128, L.cap)), sw((L.E, N // 128, K // 128))
    b = weights(L.E, (N,), 1, 5) if bias else None
    res = L.randn(N, 6) if residual else None

    def call():
        y, pre = L.out(N), L.out(N)
        ep.ep_expert_linear(x, xs, w, ws, b, res, L.dcounts, L.psum, ep.ACTS[act], y, pre=pre)
        y2 = L.out(N) if res is None else res.clone()   # without the kept sums, in place of the residual
        ep.ep_expert_linear(x, xs, w, ws, b, None if res is None else y2, L.dcounts, L.psum, ep.ACTS[act], y2)
        return y, pre, y2

    y, pre, y2 = on_both(call)
    assert L.untouched(y) and L.untouched(pre)
    xd = dequant_rows(x, xs, L, K)
    for e, (a, n) in enumerate(L.each()):
        at = slice(a, a + n)
        xe, wd = xd[at], dequant_weights(w[e], ws[e])
        z = xe @ wd.t() + (b[e].double() if bias else 0)
        sz = (K + 1) * 2.0 ** -24 * (xe.abs() @ wd.abs().t() + (b[e].double().abs() if bias else 0))
        near(pre.reshape(L.rows, N)[at], z, 2.0 ** -8 * z.abs() + sz)
        v = value64(z, act)
        r = v + (res.reshape(L.rows, N)[at].double() if residual else 0)
        near(y.reshape(L.rows, N)[at], r, 2.0 ** -8 * r.abs() + 1.13 * sz + 2.0 ** -15 * v.abs() + 1e-30)
        assert torch.equal(y.reshape(L.rows, N)[at].view(torch.int16), y2.reshape(L.rows, N)[at].view(torch.int16))


@pytest.mark.parametrize("out8", [False, True])
def test_nan_stays_in_its_row(out8):
    """A NaN byte among a row's inputs makes that row's outputs NaN and no other's."""
    L = Layout([[5, 140]])
    K, N = 256, 384
    x, sx = e4m3((*L.lead, K), 1, 115, 120, K)
    w, sw = e4m3((L.E, 2, N, K), 2, 118, 121, K)
    xs, ws = sx((*L.lead[:-1], K // 128, L.cap)), sw((L.E, 2, N // 128, K // 128))
    got = []
    for bad in (False, True):
        if bad:
            x[0, 3, 17] = x[0, 70, 200] = 0x7F
        h = L.out(N, dtype=torch.uint8 if out8 else torch.bfloat16)
        hs = torch.zeros((*L.lead[:-1], N // 128, L.cap), dtype=torch.uint8, device="cuda") if out8 else None
        ep.ep_expert_glu(x, xs, w, ws, L.dcounts, L.psum, ep.EP_ACT_RELU, h, h_scales=hs)
        got.append(h[0].view(torch.float8_e4m3fn).float() if out8 else h[0].float())
    hit = torch.zeros(L.cap, dtype=torch.bool, device="cuda")
    hit[3] = hit[70] = True
    assert torch.isnan(got[1][hit]).all()
    assert torch.equal(got[0][~hit].view(torch.int32), got[1][~hit].view(torch.int32))
