"""Refusals of the router's and the experts' entry points at the C boundary:
decided on the host, nothing launched (no GPU needed)."""
import pytest

from combine_get_dispatch_gb300 import ep

FAKE = 1 << 20   # never dereferenced: every call below is refused


def glu(mode=0, R=2, E=4, H=64, I=64, cap=8, act=2, counts=FAKE, x=FAKE, w=FAKE, h=FAKE, xs=None, ws=None, hs=None,
        gu=None, psum=FAKE):
    return ep.load().ep_expert_glu(x, xs, w, ws, mode, counts, psum, R, E, H, I, cap, act, h, hs, gu, None, None)


@pytest.mark.parametrize("bad", [
    dict(mode=1, xs=FAKE, ws=FAKE, H=128, I=128), dict(mode=3), dict(mode=2, H=128, I=128), dict(mode=2, xs=FAKE, ws=FAKE),
    dict(mode=2, xs=FAKE, ws=FAKE, H=128, I=128, gu=FAKE), dict(hs=FAKE), dict(R=0), dict(R=3), dict(E=2048, R=2),
    dict(R=1025, E=1025), dict(H=0), dict(H=60), dict(I=4), dict(cap=-1), dict(cap=1 << 30), dict(psum=None, cap=1 << 29),
    dict(H=1 << 25), dict(act=0), dict(act=4), dict(act=-1), dict(counts=None), dict(x=None), dict(w=None), dict(h=None),
    dict(x=FAKE + 8), dict(w=FAKE + 2), dict(h=FAKE + 4), dict(gu=FAKE + 8)])
def test_glu_refuses(bad):
    before = ep.ep_launch_count()
    assert glu(**bad) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_launch_count() == before


@pytest.mark.parametrize("R,E,psum", [(1, 1, FAKE), (2, 4, FAKE), (2, 4, None), (1024, 1024, None)])
def test_rows_stay_in_31_bits(R, E, psum):
    """One row more than 2^31 - 2^16 over all segments' buffers is refused."""
    cap = ((1 << 31) - (1 << 16)) // (E if psum is None else R) + 1
    assert glu(R=R, E=E, psum=psum, cap=cap) == ep.EP_ERR_INVALID_ARG
    assert glu(R=R, E=E, psum=psum, cap=0) == ep.EP_OK


def linear(R=1, E=1, K=64, N=64, cap=8, act=0, x=FAKE, w=FAKE, y=FAKE, bias=None, residual=None, pre=None):
    return ep.load().ep_expert_linear(x, None, w, None, 0, bias, residual, FAKE, FAKE, R, E, K, N, cap, act, y, pre, None, None)


@pytest.mark.parametrize("bad", [dict(K=12), dict(N=63), dict(act=5), dict(x=None), dict(y=None), dict(bias=FAKE + 2),
                                 dict(residual=FAKE + 8), dict(pre=FAKE + 1), dict(E=3, R=2)])
def test_linear_refuses(bad):
    assert linear(**bad) == ep.EP_ERR_INVALID_ARG


def test_backwards_refuse():
    L = ep.load()
    before = ep.ep_launch_count()
    g = lambda dh=FAKE, gu=FAKE, x=FAKE, w=FAKE, act=2, dgu=FAKE, dx=FAKE, dw=FAKE, H=64: L.ep_expert_glu_backward(  # noqa: E731
        dh, gu, x, w, FAKE, FAKE, 1, 1, H, 64, 8, act, dgu, dx, dw, None, None)
    for bad in (dict(dh=None), dict(gu=None), dict(x=None), dict(w=None), dict(act=0), dict(dgu=None), dict(dx=FAKE + 8),
                dict(dw=FAKE + 4), dict(H=9)):
        assert g(**bad) == ep.EP_ERR_INVALID_ARG, bad
    b = lambda dy=FAKE, pre=FAKE, x=FAKE, w=FAKE, act=2, dpre=FAKE, dx=FAKE, dw=FAKE, db=FAKE: L.ep_expert_linear_backward(  # noqa: E731
        dy, pre, x, w, FAKE, FAKE, 1, 1, 64, 64, 8, act, dpre, dx, dw, db, None, None)
    for bad in (dict(dy=None), dict(pre=None), dict(dpre=None), dict(x=None), dict(w=None), dict(act=7), dict(db=FAKE + 2)):
        assert b(**bad) == ep.EP_ERR_INVALID_ARG, bad
    assert ep.ep_launch_count() == before


def test_gate_refuses():
    L = ep.load()
    g = lambda l=FAKE, dt=0, R=1, T=4, E=8, k=2, sc=0, i=FAKE, w=FAKE: L.ep_gate_topk(l, dt, R, T, E, k, sc, i, w, None)  # noqa: E731
    for bad in (dict(l=None), dict(dt=2), dict(R=0), dict(R=3), dict(T=-1), dict(E=0), dict(E=2048), dict(k=0), dict(k=9),
                dict(E=32, k=17), dict(sc=2), dict(i=None), dict(w=None)):
        assert g(**bad) == ep.EP_ERR_INVALID_ARG, bad
    assert L.ep_gate_topk_backward(FAKE, 0, FAKE, None, 1, 4, 8, 2, 0, FAKE, None, None) == ep.EP_ERR_INVALID_ARG
    assert L.ep_gate_topk_backward(FAKE, 0, FAKE, FAKE, 1, 4, 8, 2, 0, None, None, None) == ep.EP_ERR_INVALID_ARG
