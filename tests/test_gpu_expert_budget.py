"""The experts' kernels under an SM budget (ep_set_num_sms):
they stay within it, and give the same bits as without."""
import numpy as np
import pytest
import torch

from combine_get_dispatch_gb300 import ep
from test_gpu_expert import Layout, weights

pytestmark = pytest.mark.gpu


@pytest.fixture
def budget():
    yield ep.ep_set_num_sms
    ep.ep_set_num_sms(0)


def time_of(call):
    """Milliseconds of the quickest of five."""
    call()
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


def bias_sum(act):
    rows, N = 32768, 2048
    c = torch.tensor([rows], dtype=torch.int32, device="cuda")
    ps = torch.tensor([[0, rows]], dtype=torch.int64, device="cuda")
    dy = torch.randn((1, rows, N), device="cuda", dtype=torch.bfloat16)
    pre = None if act == ep.EP_ACT_NONE else torch.randn_like(dy)
    dpre = None if act == ep.EP_ACT_NONE else torch.empty_like(dy)
    w, db = torch.zeros((1, N, 8), dtype=torch.bfloat16, device="cuda"), torch.empty((1, N), dtype=torch.bfloat16, device="cuda")
    return lambda: ep.ep_expert_linear_backward(dy, pre, None, w, c, ps, act, dpre, None, None, dbias=db)


def two_sms_are_two(budget, call):
    """On two SMs out of some 150, work that fills them all takes many times as long (8 is asked for)."""
    free = time_of(call)
    budget(2)
    few = time_of(call)
    assert few > 8 * free, f"{few:.3f} ms on two SMs, {free:.3f} ms on all"


@pytest.mark.parametrize("act", ["none", "silu"])
def test_bias_and_slope_keep_to_the_budget(budget, act):
    two_sms_are_two(budget, bias_sum(ep.ACTS[act]))


def bits(*ts):
    return [t.contiguous().view(torch.int16).clone() for t in ts if t is not None]


def on_budgets(budget, call):
    want = None
    for n in (0, 1, 2, 7, 40):
        budget(n)
        got = call()
        torch.cuda.synchronize()
        assert want is None or all(torch.equal(a, b) for a, b in zip(want, got))
        want = got


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("counts,K,N", [([[700, 0, 65]], 72, 200),                       # rows split over 8
                                        ([[40, 3], [0, 300]], 64, 8192),                # over 2
                                        ([np.arange(24).tolist()] * 2, 64, 4104)])       # one CTA a column group
def test_linear_bits(budget, counts, K, N, act):
    L = Layout(counts)
    x, w, dy = L.randn(K, 1), weights(L.E, (N, K), K, 2), L.randn(N, 3)
    b, pre = weights(L.E, (N,), 1, 5), L.randn(N, 4)
    plain = act == "none"

    def call():
        y, dpre, dx = L.out(N), None if plain else L.out(N), L.out(K)
        dw, db = torch.full_like(w, -77.0), torch.full_like(b, -77.0)
        ep.ep_expert_linear(x, None, w, None, b, None, L.dcounts, L.psum, ep.ACTS[act], y)
        ep.ep_expert_linear_backward(dy, None if plain else pre, x, w, L.dcounts, L.psum, ep.ACTS[act], dpre, dx, dw, dbias=db)
        assert L.untouched(y) and L.untouched(dx) and (plain or L.untouched(dpre))
        return bits(y, dpre, dx, dw, db)

    on_budgets(budget, call)


def test_no_rows_give_zero_bias_gradients(budget):
    """cap_rows 0 and experts without rows: zeros, under a budget too."""
    for n in (0, 1, 5):
        budget(n)
        for cap in (0, 16):
            c = torch.zeros(6, dtype=torch.int32, device="cuda")
            ps = torch.zeros((2, 4), dtype=torch.int64, device="cuda")
            dy = torch.full((2, cap, 200), float("nan"), dtype=torch.bfloat16, device="cuda")
            w = torch.zeros((6, 200, 8), dtype=torch.bfloat16, device="cuda")
            db = torch.full((6, 200), 7.0, dtype=torch.bfloat16, device="cuda")
            ep.ep_expert_linear_backward(dy, None, None, w, c, ps, ep.EP_ACT_NONE, None, None, None, dbias=db)
            assert not db.any()


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_glu_bits(budget, act):
    L = Layout([[300, 0, 77], [1, 513, 40]], align=16)
    H, I = 200, 136
    x, w, dh = L.randn(H, 1), weights(L.E, (2, I, H), H, 2), L.randn(I, 3)

    def call():
        h, gu, dgu, dx, dw = L.out(I), L.out(2, I), L.out(2, I), L.out(H), torch.full_like(w, -77.0)
        ep.ep_expert_glu(x, None, w, None, L.dcounts, L.psum, ep.ACTS[act], h, gu=gu)
        ep.ep_expert_glu_backward(dh, gu, x, w, L.dcounts, L.psum, ep.ACTS[act], dgu, dx, dw)
        assert all(L.untouched(t) for t in (h, gu, dgu, dx))
        return bits(h, gu, dgu, dx, dw)

    on_budgets(budget, call)
