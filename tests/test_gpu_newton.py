"""Newton-Schulz orthogonalisation and the optimiser's step against their
definitions in 64 bits.

Tolerances, as relative 2-norms.  A matrix rounded to 11 significant bits is off
by at most 2^-11 / sqrt(3) of its norm (q).  A step's product (b A + c A^2) X takes
X three times, A twice and the polynomial once, so it is off by less than
q sqrt(6) of itself; where the singular values are near 1, as in the last steps,
it is up to 4 times the step's result (3.44 - 2.74 = 0.7).  The steps' errors are
independent and the polynomial's slope there is below 1: 4 q sqrt(6 steps) bounds
them, and the output in bf16 adds 2^-8 / sqrt(3).  Weights in 32 bits are off by
what the update is off, and two roundings of 2^-24."""
import math

import pytest
import torch

from combine_get_dispatch_gb300 import ep

pytestmark = pytest.mark.gpu

QUINTIC = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)
Q = 2.0 ** -11 / math.sqrt(3)


def off(steps):
    return 4 * Q * math.sqrt(6 * len(steps))


def gradient(seed, *shape, dtype=torch.bfloat16, spread=0.5, size=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    rows, cols = torch.exp(spread * rand(*shape[:-1], 1)), torch.exp(spread * rand(*shape[:-2], 1, shape[-1]))
    return (rand(*shape) * rows * cols * size).to(dtype)


def exact(u, steps, eps=1e-7):
    u = u.double()
    tall = u.shape[-2] > u.shape[-1]
    x = u.transpose(-1, -2) if tall else u
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + eps)
    for a, b, c in steps:
        A = x @ x.transpose(-1, -2)
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.transpose(-1, -2) if tall else x


def call(g, steps, eps=1e-7, out=None, status=None, workspace=None):
    out = torch.full(g.shape, float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    if workspace is None:
        workspace = ep.alloc_orthogonalize_workspace(g.shape)
        workspace.fill_(0xFF)   # NaN in every word of it
    ep.ep_orthogonalize(g, steps, out, workspace, eps=eps, status=status)
    return out


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


SHAPES = [(1, 1, 8), (1, 8, 8), (3, 5, 24), (2, 24, 8), (1, 64, 64), (1, 33, 40), (4, 128, 256), (2, 256, 128), (1, 255, 264), (1, 257, 512), (2, 129, 1000),
          (1, 300, 296), (3, 512, 512), (1, 1000, 64), (1, 64, 1000), (1, 2048, 1000), (2, 700, 1416), (1, 1, 4096), (1, 4099, 8), (33, 40, 48)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quintic(shape, dtype):
    steps = [QUINTIC] * 5
    g = gradient(sum(shape), *shape, dtype=dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(g, steps, status=status)
    assert rel(out, exact(g, steps)) < off(steps) + 2.0 ** -8 / math.sqrt(3)
    assert ep.ep_read_status(status) == ep.EP_OK


@pytest.mark.parametrize("shape", [(2, 130, 264), (1, 264, 136), (1, 520, 520), (5, 16, 16)])
@pytest.mark.parametrize("steps", [[CUBIC], [CUBIC] * 8, [QUINTIC], [QUINTIC, CUBIC], [CUBIC, QUINTIC, (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)],
                                   [(1.0, 0.0, 0.0)] * 2, [(0.5, 0.0, 0.25)]])
def test_polynomials(shape, steps):
    g = gradient(3 + sum(shape), *shape)
    assert rel(call(g, steps), exact(g, steps)) < off(steps) + 2.0 ** -8 / math.sqrt(3)


def test_cubic_converges_to_the_polar_factor():
    """Singular values of at least 0.3 of the largest: after 12 cubic steps all are 1."""
    g = gradient(1, 2, 96, 640, spread=0.1)
    out = call(g, [CUBIC] * 12).double()
    u, _, v = torch.linalg.svd(g.double(), full_matrices=False)
    assert rel(out, u @ v) < off([CUBIC] * 12) + 2.0 ** -8 / math.sqrt(3)


@pytest.mark.parametrize("size", [1e-9, 1e-3, 1.0, 1e4, 1e12])
def test_sizes(size):
    g = gradient(2, 2, 72, 136, size=size)
    steps = [QUINTIC] * 5
    assert rel(call(g, steps), exact(g, steps)) < off(steps) + 2.0 ** -8 / math.sqrt(3)
    assert rel(call(g.float(), steps, eps=1e-12), exact(g, steps, 1e-12)) < off(steps) + 2.0 ** -8 / math.sqrt(3)


def test_eps_counts():
    g = gradient(2, 1, 40, 72, size=1e-6)
    norm = float(g.double().norm())
    steps = [QUINTIC] * 3
    assert rel(call(g, steps, eps=3 * norm), exact(g, steps, 3 * norm)) < off(steps) + 2.0 ** -8 / math.sqrt(3)


@pytest.mark.parametrize("shape", [(4, 40, 72), (4, 300, 136)])
def test_zeros_and_non_finite(shape):
    g = gradient(4, *shape)
    steps = [QUINTIC] * 5
    want = call(g, steps)
    for bad in (float("nan"), float("inf"), -float("inf"), 3e38):
        h = g.clone()
        h[1] = 0
        h[2, -1, 3] = bad
        out = call(h, steps)
        assert torch.equal(out[0], want[0]) and torch.equal(out[3], want[3])
        assert (out[1] == 0).all() and torch.isnan(out[2]).all()
    assert (call(torch.zeros_like(g), steps) == 0).all()


def test_low_rank():
    """A gradient of 24 rows through a 200 x 520 layer: the zero directions stay small."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    g = torch.randn((200, 24), generator=gen, device="cuda") @ torch.randn((24, 520), generator=gen, device="cuda")
    g = (g * 1e-3).float().unsqueeze(0)
    steps = [QUINTIC] * 5
    assert rel(call(g, steps), exact(g, steps)) < off(steps) + 2.0 ** -8 / math.sqrt(3)


@pytest.mark.parametrize("shape", [(3, 200, 328), (2, 520, 264)])
def test_in_place_and_repeatable(shape):
    steps = [QUINTIC] * 5
    g = gradient(5, *shape)
    want = call(g, steps)
    assert torch.equal(call(g, steps), want)
    h = g.clone()
    assert torch.equal(call(h, steps, out=h), want)
    for sms in (1, 6, 77):
        ep.ep_set_num_sms(sms)
        try:
            assert torch.equal(call(g, steps), want), sms
        finally:
            ep.ep_set_num_sms(0)
    one = call(g[1:2].contiguous(), steps)   # a matrix alone is what it is in the stack
    assert torch.equal(one[0], want[1])


def test_leading_shapes_and_nothing():
    steps = [QUINTIC] * 2
    g = gradient(6, 3, 2, 40, 72)
    assert torch.equal(call(g, steps).reshape(6, 40, 72), call(g.reshape(6, 40, 72), steps))
    assert torch.equal(call(g[0, 0].contiguous(), steps), call(g, steps)[0, 0])
    before = ep.ep_launch_count()
    call(g[:0], steps)
    assert ep.ep_launch_count() == before


def test_buffers_keep_their_neighbours():
    g = gradient(7, 2, 41, 72)
    buf = torch.full((4, 41, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    size = ep.ep_orthogonalize_workspace_size(2, 41, 72)
    ws = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    call(g, [QUINTIC] * 5, out=buf[1:3], workspace=ws[:-64])
    assert (buf[0] == 7).all() and (buf[3] == 7).all() and (ws[-64:] == 0x5A).all()


def test_past_31_bits():
    """2.5 G elements: the last matrices come out as they do alone."""
    count, M, N = 300, 8, 1 << 20
    g = torch.zeros((count, M, N), dtype=torch.bfloat16, device="cuda")
    g[[0, 299]] = gradient(9, 2, M, N)
    out = call(g, [QUINTIC] * 2)
    want = call(g[[0, 299]].contiguous(), [QUINTIC] * 2)
    assert torch.equal(out[[0, 299]], want) and (out[1:299] == 0).all()


# ---- the optimiser's step

def state(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return rand(*shape) * 1e-2, rand(*shape) * 0.02


def check_update(g, m, w, got_m, got_w, got16, steps, lr, scale, mu, nesterov, decay):
    g64, m64 = g.double(), m.double()
    new_m = mu * m64 + g64
    assert bool(((got_m.double() - new_m).abs() <= 2.0 ** -23 * (mu * m64.abs() + g64.abs())).all())
    o = exact(g64 + mu * new_m if nesterov else new_m, steps)
    new_w = (1 - lr * decay) * w.double() - lr * scale * o
    # u is off by 2^-22 of the larger of its terms, the weights by the update and two roundings
    tol = abs(lr * scale) * off(steps) * float(o.norm()) + 2.0 ** -22 * float(w.double().norm() + new_w.norm())
    assert float((got_w.double() - new_w).norm()) < tol
    assert torch.equal(got16, got_w.to(torch.bfloat16))


@pytest.mark.parametrize("shape", [(1, 1, 8), (2, 40, 72), (3, 128, 256), (2, 264, 136), (1, 515, 520), (16, 64, 48), (1, 1416, 256)])
@pytest.mark.parametrize("dtype,nesterov,decay", [(torch.bfloat16, True, 0.1), (torch.float32, False, 0.0)])
def test_muon(shape, dtype, nesterov, decay):
    steps = [QUINTIC] * 5
    g = gradient(11, *shape, dtype=dtype)
    m, w = state(12, *shape)
    gm, gw, g16 = m.clone(), w.clone(), torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = ep.alloc_orthogonalize_workspace(shape)
    ws.fill_(0xFF)
    keep = g.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_muon_update(g, gm, gw, g16, steps, ws, lr=0.1, scale=1.5, momentum=0.9, nesterov=nesterov, weight_decay=decay, status=status)
    # the binding hands 32-bit numbers on
    f = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    check_update(g, m, w, gm, gw, g16, steps, f(0.1), f(1.5), f(0.9), nesterov, f(decay))
    assert torch.equal(g, keep) and ep.ep_read_status(status) == ep.EP_OK
    # without a bf16 copy, and with momentum 0
    m2, w2 = m.clone(), w.clone()
    ep.ep_muon_update(g, m2, w2, None, steps, ws, lr=0.1, scale=1.5, momentum=0.9, nesterov=nesterov, weight_decay=decay)
    assert torch.equal(m2, gm) and torch.equal(w2, gw)
    m3, w3 = m.clone(), w.clone()
    ep.ep_muon_update(g, m3, w3, g16, steps, ws, lr=0.1, scale=1.5, momentum=0.0, nesterov=nesterov, weight_decay=decay)
    assert torch.equal(m3, g.float())
    check_update(g, m, w, m3, w3, g16, steps, f(0.1), f(1.5), 0.0, nesterov, f(decay))


def test_muon_idle_and_non_finite():
    """A zero gradient moves its weights along the momentum; zeros all over leave them to the decay; a NaN stays in its matrix."""
    steps = [QUINTIC] * 5
    g = gradient(13, 4, 40, 72)
    m, w = state(14, 4, 40, 72)
    g[0] = 0
    g[1] = 0
    m[1] = 0
    g[3, 2, 2] = float("nan")
    gm, gw, g16 = m.clone(), w.clone(), torch.empty_like(g)
    ep.ep_muon_update(g, gm, gw, g16, steps, ep.alloc_orthogonalize_workspace(g.shape), lr=0.125, momentum=0.5, weight_decay=0.5)
    check_update(g[:3], m[:3], w[:3], gm[:3], gw[:3], g16[:3], steps, 0.125, 1.0, 0.5, True, 0.5)
    assert torch.equal(gw[1], w[1] * (1 - 0.0625)) and torch.isnan(gw[3]).all()


def test_muon_graph_and_streams():
    """Captured, replayed on new gradients in place; a second call on a stream and workspace of its own meanwhile."""
    steps = [QUINTIC] * 5
    shape = (4, 136, 264)
    gs = [gradient(20 + i, *shape) for i in range(3)]
    m, w = state(15, *shape)
    eager = [m.clone(), w.clone(), torch.empty(shape, dtype=torch.bfloat16, device="cuda")]
    ws = ep.alloc_orthogonalize_workspace(shape)
    for g in gs:
        ep.ep_muon_update(g, *eager, steps, ws, lr=0.01, scale=2.0)
    live, bufs = gs[0].clone(), [m.clone(), w.clone(), torch.empty(shape, dtype=torch.bfloat16, device="cuda")]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        ep.ep_muon_update(live, *bufs, steps, ws, lr=0.01, scale=2.0)
    other = [m.clone(), w.clone(), torch.empty(shape, dtype=torch.bfloat16, device="cuda")]
    ws2, second = ep.alloc_orthogonalize_workspace(shape), torch.cuda.Stream()
    torch.cuda.synchronize()
    for g in gs:
        live.copy_(g)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(second):
            ep.ep_muon_update(g, *other, steps, ws2, lr=0.01, scale=2.0)
        torch.cuda.synchronize()
    for a, b, c in zip(eager, bufs, other):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_binding_refuses():
    g = gradient(16, 2, 40, 72)
    m, w = state(17, 2, 40, 72)
    w16, ws, steps = torch.empty_like(g), ep.alloc_orthogonalize_workspace(g.shape), [QUINTIC] * 5
    good = [g, m, w, w16, steps, ws]
    for i, bad in ((0, g.half()), (0, g.cpu()), (0, g.transpose(1, 2)), (0, g[0, 0]), (1, m.bfloat16()), (1, m[:1]), (2, w.double()),
                   (3, w16.float()), (3, w16[:, :39]), (4, [(1.0, 2.0)]), (5, ws.view(torch.int32))):
        with pytest.raises(ValueError):
            ep.ep_muon_update(*good[:i], bad, *good[i + 1:], lr=0.1)
    for bad in (dict(lr=float("nan")), dict(momentum=1.0), dict(momentum=-0.1), dict(eps=0.0), dict(scale=float("inf"))):
        with pytest.raises(ep.EPError):
            ep.ep_muon_update(*good, **dict(dict(lr=0.1), **bad))
    with pytest.raises(ep.EPError):
        ep.ep_muon_update(g, m, w, w16, steps, ws[:-16], lr=0.1)
    with pytest.raises(ep.EPError):
        ep.ep_orthogonalize(g, [], w16, ws)
    with pytest.raises(ValueError):
        ep.ep_orthogonalize(g, steps, w16.float(), ws)
    h = gradient(18, 1, 8, 12)
    with pytest.raises(ep.EPError):
        ep.ep_orthogonalize(h, steps, torch.empty_like(h), ws)
