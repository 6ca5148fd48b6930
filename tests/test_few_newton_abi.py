"""Refusals of ep_moe_few, ep_orthogonalize and ep_muon_update at the C boundary:
decided on the host, nothing launched (no GPU needed)."""
import ctypes

import pytest

from combine_get_dispatch_gb300 import ep

FAKE = 1 << 20   # never dereferenced: every call below is refused


def few(x=FAKE, idx=FAKE, weights=FAKE, wg=FAKE, gs=None, wd=FAKE, ds=None, mode=0, R=2, T_r=4, k=2, E=4, H=128, I=128, act=2, out=FAKE,
        ws=FAKE, size=1 << 30):
    return ep.load().ep_moe_few(x, idx, weights, wg, gs, wd, ds, mode, R, T_r, k, E, H, I, act, out, ws, size, None, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(idx=None), dict(weights=None), dict(wg=None), dict(wd=None), dict(out=None), dict(ws=None), dict(x=FAKE + 8),
    dict(wg=FAKE + 2), dict(wd=FAKE + 8), dict(out=FAKE + 4), dict(ws=FAKE + 8), dict(size=8 * 2 * 128 * 2 - 1), dict(mode=1, gs=FAKE, ds=FAKE),
    dict(mode=3), dict(mode=2), dict(mode=2, gs=FAKE), dict(mode=2, ds=FAKE), dict(gs=FAKE), dict(ds=FAKE),
    dict(mode=2, gs=FAKE, ds=FAKE, H=136), dict(mode=2, gs=FAKE, ds=FAKE, I=64), dict(H=12), dict(I=9), dict(H=0), dict(I=-8), dict(R=0), dict(R=3),
    dict(T_r=-1), dict(T_r=33), dict(R=1, T_r=65), dict(R=1024, T_r=1 << 22, E=1024), dict(k=0), dict(k=17), dict(E=0), dict(E=1025, R=1), dict(act=0),
    dict(act=4), dict(H=1 << 25), dict(E=256, H=1 << 23), dict(E=256, I=1 << 23)])
def test_few_refuses(bad):
    before = ep.ep_launch_count()
    assert few(**bad) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_launch_count() == before


def test_few_sizes():
    assert few(T_r=0) == ep.EP_OK
    size = ep.ep_moe_few_workspace_size
    assert size(1, 64, 16, 64, 2048) >= 1024 * 2048 * 2
    assert size(1, 0, 2, 4, 64) > 0
    for bad in ((0, 1, 1, 1, 8), (1, 65, 1, 1, 8), (1, 1, 17, 20, 8), (1, 1, 1, 1, 12), (2, 1, 1, 3, 8), (1, -1, 1, 1, 8)):
        assert size(*bad) == 0
    assert ep.EP_MOE_FEW_TOKENS == 64


def abc(*v):
    return (ctypes.c_float * len(v))(*v)


def ortho(g=FAKE, dtype=1, count=2, M=16, N=24, steps=1, coefficients=abc(3.0, -4.0, 2.0), eps=1e-7, out=FAKE, ws=FAKE, size=1 << 40):
    return ep.load().ep_orthogonalize(g, dtype, count, M, N, steps, coefficients, eps, out, ws, size, None, None)


def muon(g=FAKE, dtype=1, m=FAKE, w=FAKE, w16=FAKE, count=2, M=16, N=24, lr=0.1, scale=1.0, mu=0.9, nesterov=1, decay=0.0, steps=1,
         coefficients=abc(3.0, -4.0, 2.0), eps=1e-7, ws=FAKE, size=1 << 40):
    return ep.load().ep_muon_update(g, dtype, m, w, w16, count, M, N, lr, scale, mu, nesterov, decay, steps, coefficients, eps, ws, size, None, None)


NAN, INF = float("nan"), float("inf")
SHARED = [dict(g=None), dict(g=FAKE + 8), dict(dtype=2), dict(dtype=-1), dict(count=-1), dict(count=65536), dict(M=0), dict(N=0), dict(N=20), dict(N=-8),
          dict(M=(1 << 20) + 1), dict(N=(1 << 20) + 8), dict(count=65535, M=1 << 16), dict(steps=0), dict(steps=33), dict(coefficients=None),
          dict(coefficients=abc(NAN, 0.0, 0.0)), dict(coefficients=abc(1.0, 0.0, INF)), dict(eps=0.0), dict(eps=1e-13), dict(eps=-1.0), dict(eps=NAN),
          dict(eps=INF), dict(ws=None), dict(ws=FAKE + 4), dict(size=0), dict(size=64)]


@pytest.mark.parametrize("bad", SHARED + [dict(out=None), dict(out=FAKE + 2)])
def test_orthogonalize_refuses(bad):
    before = ep.ep_launch_count()
    assert ortho(**bad) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_launch_count() == before


@pytest.mark.parametrize("bad", SHARED + [dict(m=None), dict(w=None), dict(m=FAKE + 4), dict(w=FAKE + 8), dict(w16=FAKE + 2), dict(lr=NAN), dict(scale=INF),
                                          dict(mu=1.0), dict(mu=-0.5), dict(mu=NAN), dict(decay=INF)])
def test_muon_refuses(bad):
    before = ep.ep_launch_count()
    assert muon(**bad) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_launch_count() == before


def test_stack_sizes():
    size = ep.ep_orthogonalize_workspace_size
    assert ortho(count=0) == ep.EP_OK and muon(count=0) == ep.EP_OK
    assert size(2, 16, 24) > 0 and size(0, 16, 24) > 0
    assert size(64, 7168, 2048) >= 64 * 7168 * 2048 * 4   # no 32-bit wrap
    for bad in ((-1, 16, 24), (1, 0, 8), (1, 8, 12), (1, 1 << 21, 8), (65536, 8, 8)):
        assert size(*bad) == 0
