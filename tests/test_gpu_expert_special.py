"""Infinities and NaN in the rows of the experts' bf16 products, inside the
segments: they stay in their rows (in the weights' gradient: in their columns),
and every other output keeps its bits."""
import math

import pytest
import torch

from combine_get_dispatch_gb300 import ep
from test_gpu_expert import Layout, weights

pytestmark = pytest.mark.gpu

K, N = 200, 136


def bits_equal(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("act", ["none", "relu"])
def test_forward_rows(act):
    L = Layout([[3, 0, 300], [17, 1, 2]])
    x, w = L.randn(K, 1), weights(L.E, (N, K), K, 2)
    y0, y, pre = L.out(N), L.out(N), L.out(N)
    ep.ep_expert_linear(x, None, w, None, None, None, L.dcounts, L.psum, ep.ACTS[act], y0)
    rows = [1, 3 + 64, 3 + 299]   # of the first rank: a segment's middle, a tile's middle, a segment's end
    for r, v in zip(rows, (math.nan, math.inf, -math.inf)):
        x[0, r, 77] = v
    ep.ep_expert_linear(x, None, w, None, None, None, L.dcounts, L.psum, ep.ACTS[act], y, pre=pre)
    hit = torch.zeros(L.rows, dtype=torch.bool, device="cuda")
    hit[rows] = True
    assert bits_equal(y.reshape(L.rows, N)[~hit], y0.reshape(L.rows, N)[~hit])
    for r, e in zip(rows, (0, 2, 2)):
        z = x[0, r].double() @ w[e].double().t()
        want = z if act == "none" else torch.where(z < 0, 0.0, z)
        for got, ref in ((pre[0, r].double(), z), (y[0, r].double(), want)):
            assert torch.equal(torch.isnan(got), torch.isnan(ref))
            assert torch.equal(torch.isposinf(got), torch.isposinf(ref)) and torch.equal(torch.isneginf(got), torch.isneginf(ref))


def test_gradients():
    L = Layout([[3, 0, 300], [17, 1, 2]])
    x, w, dy = L.randn(K, 1), weights(L.E, (N, K), K, 2), L.randn(N, 3)

    def call():
        dx, dw, db = L.out(K), torch.empty_like(w), torch.empty((L.E, N), dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_linear_backward(dy, None, x, w, L.dcounts, L.psum, ep.EP_ACT_NONE, None, dx, dw, dbias=db)
        return dx, dw, db

    dx0, dw0, db0 = call()
    x[0, 3 + 200, 70] = math.nan      # column 70 of the third expert's weights' gradient
    dy[0, 3 + 299, 9] = math.inf      # row 302 of dx; row 9 of that gradient and of its bias
    dx, dw, db = call()
    hit = torch.zeros(L.rows, dtype=torch.bool, device="cuda")
    hit[3 + 299] = True
    assert bits_equal(dx.reshape(L.rows, K)[~hit], dx0.reshape(L.rows, K)[~hit])
    assert not torch.isfinite(dx[0, 3 + 299]).any()
    clean = torch.ones((N, K), dtype=torch.bool, device="cuda")
    clean[9], clean[:, 70] = False, False
    for e in range(L.E):
        if e == 2:
            assert not torch.isfinite(dw[e][~clean]).any() and bits_equal(dw[e][clean], dw0[e][clean])
            assert torch.isposinf(db[e, 9]) and bits_equal(db[e, :9], db0[e, :9]) and bits_equal(db[e, 10:], db0[e, 10:])
        else:
            assert bits_equal(dw[e], dw0[e]) and bits_equal(db[e], db0[e])
