"""The layer for few tokens and the optimiser's step as a model uses them: a training
step, its update, answers from the updated weights; then what they share: graphs,
workspaces, budgets, large calls.

Tolerances, as relative 2-norms.  An answer's h and output are rounded to bf16
once each, and with the layer's other path y too: 3 roundings of 2^-9 / sqrt(3)
on average, bounded by 2^-8 sqrt(3) < 0.007.  The update: fp16 operands, 2^-11 /
sqrt(3) of a matrix each, six in a step's product, which is at most 4 times the
step's result, and five steps: 4 * 2^-11 / sqrt(3) * sqrt(30) < 0.0062; the
difference of two weights in 32 bits adds 2^-23 |w| / |difference|."""
import math
import os
import sys

import pytest
import torch

from combine_get_dispatch_gb300 import ep

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

ANSWER, UPDATE = 0.007, 0.0062


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def data(seed, R, T_r, E, H, I):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return (rand(R, T_r, H).bfloat16(), rand(R, T_r, E), (rand(E, 2, I, H) * H ** -0.5).bfloat16(), (rand(E, H, I) * I ** -0.5).bfloat16(),
            rand(R, T_r, H).bfloat16())


def muon64(g, m, w, steps, lr, scale, momentum, decay):
    """m, w after a step with Nesterov's momentum."""
    m = momentum * m.double() + g.double()
    u = g.double() + momentum * m
    tall = u.shape[-2] > u.shape[-1]
    x = u.transpose(-1, -2) if tall else u
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + 1e-7)
    for a, b, c in steps:
        A = x @ x.transpose(-1, -2)
        x = a * x + (b * A + c * (A @ A)) @ x
    return m, (1 - lr * decay) * w.double() - lr * scale * (x.transpose(-1, -2) if tall else x)


def dense64(x, logits, k, w_in, w_out):
    p = torch.softmax(logits.double(), -1).reshape(-1, logits.shape[-1])
    idx = torch.sort(logits, dim=-1, descending=True, stable=True)[1][..., :k].reshape(-1, k)
    xf, out = x.double().reshape(-1, x.shape[-1]), torch.zeros((p.shape[0], x.shape[-1]), dtype=torch.float64, device="cuda")
    for e in range(p.shape[1]):
        t = (idx == e).any(-1).nonzero()[:, 0]
        h = torch.nn.functional.silu(xf[t] @ w_in[e, 0].double().t()) * (xf[t] @ w_in[e, 1].double().t())
        out.index_add_(0, t, p[t, e, None] * (h @ w_out[e].double().t()))
    return out.reshape(x.shape)


@pytest.mark.parametrize("R,T_r,E,k,H,I", [(2, 32, 8, 2, 512, 264), (4, 16, 16, 4, 256, 128), (1, 64, 4, 2, 264, 520)])
def test_training_step_update_and_answers(R, T_r, E, k, H, I):
    import moe_layer
    x, logits, w_in, w_out, d_out = data(H + I, R, T_r, E, H, I)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cap = R * T_r * min(k, E // R)
    states = [moe_layer.masters(w) for w in (w_in, w_out)]
    for step in range(2):
        _, saved = moe_layer.forward(x, logits, k, w_in, w_out, cap, status)
        grads = moe_layer.backward(d_out, saved, status)[2:]
        for w, g, s in zip((w_in, w_out), grads, states):
            M, N = w.shape[-2:]
            scale, before = max(1.0, M / N) ** 0.5, s["w"].clone()
            m64, w64 = muon64(g, s["m"], s["w"], moe_layer.QUINTIC, 0.02, scale, 0.95, 0.1)
            moe_layer.update(w, g, s, 0.02, status, weight_decay=0.1)
            assert rel(s["m"], m64) < 2.0 ** -23
            # (the weights that decay are known exactly: what is off is the update)
            kept = before.double() * (1 - 0.02 * 0.1)
            assert rel(s["w"].double() - kept, w64 - kept) < UPDATE + 2.0 ** -23 * float(before.norm() / (w64 - kept).norm())
            assert torch.equal(w, s["w"].bfloat16())
    want = dense64(x, logits, k, w_in, w_out)
    other, _ = moe_layer.forward(x, logits, k, w_in, w_out, cap, status)
    few = moe_layer.serve_few(x, logits, k, w_in, w_out, status)
    assert rel(few, want) < ANSWER and rel(other, want) < ANSWER
    if H % 128 == 0 and I % 128 == 0:
        q_in, q_out = moe_layer.quantise_weights(w_in), moe_layer.quantise_weights(w_out)
        wide = lambda q, s: q.view(torch.float8_e4m3fn).double() * (2.0 ** (s.double() - 127)).repeat_interleave(128, -1).repeat_interleave(128, -2)  # noqa: E731
        assert rel(moe_layer.serve_few(x, logits, k, q_in, q_out, status), dense64(x, logits, k, wide(*q_in), wide(*q_out))) < ANSWER
    assert ep.ep_read_status(status) == ep.EP_OK


def test_example_runs(capsys):
    import moe_layer
    moe_layer.main()
    assert "few (4, 8, 1024)" in capsys.readouterr().out


def test_two_graphs_share_workspaces():
    """Update and answer captured, each twice, on a stream of their own and with the same workspaces; replayed in turn
    they do what eager calls do."""
    import moe_layer
    R, T_r, E, k, H, I = 1, 8, 8, 2, 384, 256
    x, logits, w_in, w_out, _ = data(5, R, T_r, E, H, I)
    gen = torch.Generator(device="cuda").manual_seed(6)
    grads = [torch.randn(w.shape, generator=gen, device="cuda").bfloat16() for w in (w_in, w_out)]
    idx = torch.sort(logits, dim=-1, descending=True, stable=True)[1][..., :k].contiguous()
    weights = torch.softmax(torch.gather(logits, -1, idx), -1)
    few_ws = ep.alloc_moe_few_workspace(R, T_r, k, E, I)
    news = lambda: [(w.clone(), moe_layer.masters(w)) for w in (w_in, w_out)]  # noqa: E731

    def step(sets, out):
        for (w, s), g in zip(sets, grads):
            moe_layer.update(w, g, s, 0.02, None)
        ep.ep_moe_few(x, idx, weights, sets[0][0], None, sets[1][0], None, ep.EP_ACT_GELU, out, few_ws)

    eager, want = news(), []
    for _ in range(4):
        out = torch.empty_like(x)
        step(eager, out)
        want.append(out)
    sets = news()
    outs = [torch.empty_like(x) for _ in range(2)]
    torch.cuda.synchronize()
    stream, graphs = torch.cuda.Stream(), []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step(sets, out)
        graphs.append(g)
    for n in range(4):
        graphs[n % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[n % 2], want[n])
    for (w, s), (w2, s2) in zip(sets, eager):
        assert torch.equal(w, w2) and torch.equal(s["w"], s2["w"]) and torch.equal(s["m"], s2["m"])


@pytest.mark.parametrize("kind,E,H,I", [("bf16", 20, 2568, 2056), ("e4m3", 52, 2560, 2176)])
def test_large_calls(kind, E, H, I):
    """E4M3: large enough for more CTAs than run at once; with an SM budget they are not, and give the same."""
    from test_gpu_few import call, check, make
    s = make(11, 1, 32, 8, E, H, I, kind)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(s, "silu", status=status)
    check(s, "silu", out)
    for budget in (151, 40, 1):
        ep.ep_set_num_sms(budget)
        try:
            assert torch.equal(call(s, "silu", status=status), out)
        finally:
            ep.ep_set_num_sms(0)
    assert ep.ep_read_status(status) == ep.EP_OK


def test_e4m3_infinity_stays_with_its_token():
    from test_gpu_few import call, make
    s = make(12, 1, 24, 2, 4, 384, 256, "e4m3")
    clean = call(s, "silu")
    for value in (float("inf"), -float("inf"), float("nan")):
        s["x"][0, 5, 200] = value
        out = call(s, "silu")
        assert bool(out[0, 5].isnan().all())
        out[0, 5] = clean[0, 5]
        assert torch.equal(out, clean)


@pytest.mark.parametrize("shape", [(3, 1416, 520), (2, 520, 1416), (1, 2048, 840), (7, 584, 584), (2, 1100, 512)])
def test_edges_of_tiles(shape):
    """Widths whose last tile is narrow, and rows that are not whole lines, of either orientation."""
    from test_gpu_newton import QUINTIC, call, exact, gradient, off
    for dtype in (torch.bfloat16, torch.float32):
        g = gradient(sum(shape), *shape, dtype=dtype)
        steps = [QUINTIC] * 5
        assert rel(call(g, steps), exact(g, steps)) < off(steps) + 2.0 ** -8 / math.sqrt(3)


@pytest.mark.parametrize("shape,count", [((300, 296), 40), ((1000, 520), 12), ((264, 1416), 90), ((40, 136), 700)])
def test_a_matrix_comes_out_as_it_does_alone(shape, count):
    """Stacks of few and of many matrices are cut into tiles of different widths."""
    from test_gpu_newton import QUINTIC, call, gradient
    g = gradient(count, count, *shape)
    out = call(g, [QUINTIC] * 4)
    for z in (0, count // 2, count - 1):
        assert torch.equal(call(g[z:z + 1].contiguous(), [QUINTIC] * 4)[0], out[z])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("R,T_r,k,E,H,I", [(1, 1, 8, 16, 1024, 512), (1, 4, 2, 16, 256, 128), (2, 16, 2, 4, 384, 256), (1, 32, 1, 1, 512, 640), (1, 9, 4, 6, 128, 2176)])
def test_h_is_kept_for_few_tokens(kind, R, T_r, k, E, H, I):
    """Up to 32 tokens the output is off by its own rounding (2^-8 of itself), by sums in 32 bits (2^-23 a product of the
    magnitudes) and by h's: two bf16 words are off by 2^-16 of it, two E4M3 parts by 2^-9 and, where they run out of
    exponents, 2^-21 of the largest; the same 2^-21 holds for x; the activation is off by 2^-16."""
    from test_gpu_few import act64, call, make, wide
    s = make(R + T_r + H, R, T_r, k, E, H, I, kind)
    x, idx, weights = s["x"].double().reshape(-1, H), s["idx"].reshape(R * T_r, -1), s["weights"].double().reshape(R * T_r, -1)
    out, off = torch.zeros_like(x), torch.zeros_like(x)
    part, low = (2.0 ** -16, 0.0) if kind == "bf16" else (2.0 ** -9, 2.0 ** -21)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        gu, down = wide(s["w_gu"], s["gu_scales"], e), wide(s["w_down"], s["down_scales"], e)
        gate, up = x[t] @ gu[0].t(), x[t] @ gu[1].t()
        a = act64(gate, "silu")
        h = a * up
        dx = low * x[t].abs().amax(-1, keepdim=True) + H * 2.0 ** -23 * x[t].abs()
        dg, du = dx @ gu[0].abs().t(), dx @ gu[1].abs().t()
        dh = (part + 2.0 ** -16) * h.abs() + 1.13 * dg * up.abs() + a.abs() * du + 1.13 * dg * du
        if h.numel():
            dh = dh + low * h.abs().amax(-1, keepdim=True)
        w = weights[t, j].unsqueeze(1)
        out.index_add_(0, t, w * (h @ down.t()))
        off.index_add_(0, t, w.abs() * (dh @ down.abs().t() + (I + 16) * 2.0 ** -23 * (h.abs() @ down.abs().t())))
    d = (call(s, "silu").double().reshape(-1, H) - out).abs()
    bound = 1.004 * off + 2.0 ** -8 * out.abs() + 1e-30
    assert bool((d <= bound).all()), f"{float((d / bound).max())} of the bound"


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_one_expert_takes_every_token(kind):
    """More tokens an expert than are taken at a time, on either side of 32 tokens."""
    from test_gpu_few import call, check, make
    for T in (16, 17, 24, 31, 32, 33, 48, 64):
        s = make(T, 1, T, 2, 2, 256, 384, kind)
        check(s, "gelu", call(s, "gelu"))


def test_a_workspace_for_more_tokens_serves_fewer():
    from test_gpu_few import call, make
    sizes = [ep.ep_moe_few_workspace_size(1, T, 2, 8, 72) for T in range(65)]
    assert sizes == sorted(sizes)
    ws = ep.alloc_moe_few_workspace(1, 40, 2, 8, 72)
    s = make(3, 1, 32, 2, 8, 64, 72, "bf16")
    assert torch.equal(call(s, "silu", workspace=ws), call(s, "silu"))
