"""The whole layer for a few tokens against its definition in 64 bits.

Tolerance, element by element, from the roundings counted: a sum of K products in
32 bits is off by at most K 2^-23 of the sum of their magnitudes (2^-24 for each
of K roundings, twice that where the tensor core cuts instead of rounding); h by
2^-8 of itself (bf16), the activation's own 2^-16, and what its two sums are off,
times slopes of at most 1.13 (SiLU 1.1, GELU 1.13); the output by 2^-8 of itself,
its own sums, and what h is off through |W_down|."""
import math

import pytest
import torch

from combine_get_dispatch_gb300 import ep

pytestmark = pytest.mark.gpu

ACTS = {"relu": ep.EP_ACT_RELU, "silu": ep.EP_ACT_SILU, "gelu": ep.EP_ACT_GELU}


def make(seed, R, T_r, k, E, H, I, kind, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    s = dict(x=(rand(R, T_r, H) * std).bfloat16(), weights=torch.softmax(rand(R, T_r, k), -1))
    s["idx"] = torch.argsort(torch.rand((R, T_r, E), generator=g, device="cuda"), -1)[..., :k].contiguous()
    if kind == "bf16":
        s["w_gu"], s["w_down"] = (rand(E, 2, I, H) * H ** -0.5).bfloat16(), (rand(E, H, I) * I ** -0.5).bfloat16()
        s["gu_scales"] = s["down_scales"] = None
    else:
        e4m3 = lambda *n: (rand(*n) * 96).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        s["w_gu"], s["w_down"] = e4m3(E, 2, I, H), e4m3(E, H, I)
        b = lambda K, *n: torch.randint(0, 3, n, generator=g, device="cuda", dtype=torch.uint8) + int(120 - math.log2(K) / 2)  # noqa: E731
        s["gu_scales"], s["down_scales"] = b(H, E, 2, I // 128, H // 128), b(I, E, H // 128, I // 128)
    return s


def call(s, act, out=None, status=None, workspace=None):
    R, T_r, H = s["x"].shape
    E, _, I, _ = s["w_gu"].shape
    k = s["idx"].shape[-1]
    out = torch.full_like(s["x"], float("nan")) if out is None else out
    ws = ep.alloc_moe_few_workspace(R, T_r, k, E, I) if workspace is None else workspace
    if workspace is None:
        ws.fill_(0xFF)   # NaN in every word of it
    ep.ep_moe_few(s["x"], s["idx"], s["weights"], s["w_gu"], s["gu_scales"], s["w_down"], s["down_scales"], ACTS[act], out, ws, status)
    return out


def wide(w, scales, e):
    if scales is None:
        return w[e].double()
    sc = (2.0 ** (scales[e].double() - 127)).repeat_interleave(128, -2).repeat_interleave(128, -1)
    return w[e].view(torch.float8_e4m3fn).double() * sc


def act64(z, name):
    if name == "silu":
        return z * torch.sigmoid(z)
    return z * torch.special.ndtr(z) if name == "gelu" else z.clamp(min=0)


def reference(s, act):
    """The output in 64 bits and the bound of its error."""
    R, T_r, H = s["x"].shape
    E, _, I, _ = s["w_gu"].shape
    x, idx, weights = s["x"].double().reshape(-1, H), s["idx"].reshape(R * T_r, -1), s["weights"].double().reshape(R * T_r, -1)
    out, off = torch.zeros_like(x), torch.zeros_like(x)
    for e in sorted(set(idx.flatten().tolist())):
        if not 0 <= e < E:
            continue
        t, j = (idx == e).nonzero(as_tuple=True)
        gu, down = wide(s["w_gu"], s["gu_scales"], e), wide(s["w_down"], s["down_scales"], e)
        gate, up = x[t] @ gu[0].t(), x[t] @ gu[1].t()
        a = act64(gate, act)
        h = a * up
        eps = H * 2.0 ** -23
        dg, du = eps * (x[t].abs() @ gu[0].abs().t()), eps * (x[t].abs() @ gu[1].abs().t())
        dh = 2.0 ** -8 * h.abs() + 2.0 ** -16 * (a * up).abs() + 1.13 * dg * up.abs() + a.abs() * du + 1.13 * dg * du
        w = weights[t, j].unsqueeze(1)
        out.index_add_(0, t, w * (h @ down.t()))
        off.index_add_(0, t, w.abs() * (dh @ down.abs().t() + (I + 16) * 2.0 ** -23 * (h.abs() @ down.abs().t())))
    return out.reshape(s["x"].shape), (1.004 * off + 2.0 ** -8 * out.abs() + 1e-30).reshape(s["x"].shape)


def check(s, act, out):
    ref, off = reference(s, act)
    d = (out.double() - ref).abs()
    assert bool((d <= off).all()), f"{float((d / off).max())} of the bound"


SHAPES = [  # R, T_r, k, E, H, I
    (1, 1, 1, 1, 8, 8), (1, 1, 2, 4, 64, 24), (1, 4, 2, 16, 256, 128), (2, 3, 3, 8, 264, 136), (4, 16, 2, 16, 256, 128), (1, 64, 2, 4, 520, 72),
    (1, 1, 8, 8, 4096, 1416), (1, 7, 16, 64, 1000, 760), (8, 8, 8, 256, 512, 96), (1, 33, 1, 1, 1032, 40), (64, 1, 16, 1024, 72, 16),
    (1, 64, 16, 16, 136, 264), (1, 9, 4, 12, 2056, 8), (1, 5, 3, 6, 8, 2056), (1, 17, 8, 9, 7168, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_bf16(shape, act):
    s = make(sum(shape), *shape, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(s, act, call(s, act, status=status))
    assert ep.ep_read_status(status) == ep.EP_OK


@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 128, 128), (1, 1, 8, 16, 1024, 512), (1, 4, 2, 16, 256, 128), (1, 64, 2, 4, 384, 640), (2, 16, 6, 64, 896, 256),
                                   (1, 13, 16, 32, 2176, 128), (1, 40, 1, 1, 128, 1152), (1, 1, 4, 8, 7168, 2048)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_e4m3(shape, act):
    s = make(sum(shape), *shape, "e4m3")
    check(s, act, call(s, act))


def test_e4m3_every_code_and_scale():
    """Weights of every finite code (subnormals, both zeros) and scales over 200 binades."""
    s = make(5, 1, 2, 1, 1, 256, 256, "e4m3")
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8, device="cuda")
    s["w_gu"] = codes[torch.arange(2 * 256 * 256, device="cuda") % len(codes)].reshape(1, 2, 256, 256).contiguous()
    s["w_down"] = codes[(torch.arange(256 * 256, device="cuda") * 7) % len(codes)].reshape(1, 256, 256).contiguous()
    for lo in (27, 77, 117, 137):
        s["gu_scales"] = torch.tensor([lo, lo + 1, lo + 3, lo, lo + 2, lo, lo + 1, lo], dtype=torch.uint8, device="cuda").reshape(1, 2, 2, 2)
        s["down_scales"] = torch.tensor([254 - lo, 253 - lo, 252 - lo, 254 - lo], dtype=torch.uint8, device="cuda").reshape(1, 2, 2)
        if 2 * lo + 8 < 254:   # h is tiny where the scales are: keep the output in range
            s["down_scales"] = (s["down_scales"].int() - (127 - lo)).clamp(1, 250).to(torch.uint8)
        out = call(s, "relu")
        ref, off = reference(s, "relu")
        big = ref.abs() < 1e37
        tiny = 1e-37 * 256 * 448 * 8   # what 32 bits lose below their smallest normal number
        d = (out.double() - ref).abs()
        assert bool((d <= off + tiny)[big].all()), lo


def test_e4m3_nan_code_and_nan_scale():
    s = make(6, 1, 3, 2, 4, 256, 256, "e4m3")
    s["idx"] = torch.tensor([[[0, 1], [2, 3], [0, 2]]], device="cuda")
    s["w_down"][1, 5, 77] = 0x7F
    s["w_down"][1, 9, 78] = 0xFF
    out = call(s, "silu")
    nan = torch.isnan(out)
    assert nan[0, 0].nonzero().flatten().tolist() == [5, 9] and not nan[0, 1:].any()
    s["w_down"][1, 5, 77] = s["w_down"][1, 9, 78] = 0
    s["gu_scales"][3, 1, 1, 0] = 255
    out = call(s, "silu")
    assert torch.isnan(out[0, 1]).all() and not torch.isnan(out[0, [0, 2]]).any()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_unused_places(kind):
    """Unused slots, padded tokens and experts nobody chose may hold anything."""
    s = make(7, 2, 6, 3, 8, 256, 128, kind)
    s["idx"][0, 1] = -1
    s["idx"][1, 5] = -1
    s["idx"][0, 0, 1] = -1
    s["idx"][1, 2, [0, 2]] = -1
    s["idx"][s["idx"] == 6] = 2   # experts named twice by a token, 6 by none
    s["x"][0, 1] = float("nan")
    s["x"][1, 5] = float("inf")
    s["weights"][s["idx"] < 0] = float("nan")
    s["w_gu"][6] = 0x7F if kind == "e4m3" else float("nan")
    s["w_down"][6] = 0x7F if kind == "e4m3" else float("nan")
    out = call(s, "silu")
    assert (out[0, 1] == 0).all() and (out[1, 5] == 0).all()
    s["x"][0, 1] = s["x"][1, 5] = 0
    s["weights"][s["idx"] < 0] = 0
    check(s, "silu", out)
    s["idx"].fill_(-1)
    assert (call(s, "silu") == 0).all()


def test_invalid_ids_count_as_unused():
    s = make(8, 1, 5, 4, 8, 128, 64, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["idx"][0, 0, 0] = 8
    s["idx"][0, 2, 3] = -2
    s["idx"][0, 4] = torch.tensor([1 << 40, -(1 << 62), 3, (1 << 32) + 1], device="cuda")
    out = call(s, "silu", status=status)
    assert ep.ep_read_status(status) == ep.EP_ERR_INVALID_ARG
    check(s, "silu", out)


@pytest.mark.parametrize("T,k", [(64, 16), (64, 1), (9, 16), (33, 2)])
def test_all_on_one_expert(T, k):
    """Every slot names expert 2: up to 1024 rows of one expert."""
    s = make(9, 1, T, k, 4, 136, 72, "bf16") if k <= 4 else make(9, 1, T, k, 16, 136, 72, "bf16")
    s["idx"].fill_(2)
    check(s, "gelu", call(s, "gelu"))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_neither_batch_nor_budget_changes_a_token(kind):
    s = make(10, 1, 24, 4, 12, 896, 384, kind)
    out = call(s, "silu")
    for sms in (1, 7, 100):
        ep.ep_set_num_sms(sms)
        try:
            assert torch.equal(call(s, "silu"), out), sms
        finally:
            ep.ep_set_num_sms(0)
    for t in (0, 11, 23):
        one = dict(s, **{n: s[n][:, t:t + 1].contiguous() for n in ("x", "idx", "weights")})
        assert torch.equal(call(one, "silu")[0, 0], out[0, t])
    assert torch.equal(call(s, "silu"), out)


def test_in_place_and_infinities():
    s = make(11, 1, 6, 2, 4, 200, 88, "bf16")
    want = call(s, "silu")
    x = s["x"].clone()
    assert torch.equal(call(dict(s, x=x), "silu", out=x), want)
    s["x"][0, 3, 7] = float("inf")
    out = call(s, "silu")
    assert not torch.isfinite(out[0, 3]).any()
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(out[0, keep], want[0, keep])


def test_rows_behind_out_stay():
    s = make(12, 1, 3, 2, 4, 264, 40, "bf16")
    buf = torch.full((5, 264), 7.0, dtype=torch.bfloat16, device="cuda")
    call(s, "silu", out=buf[1:4].unsqueeze(0))
    assert (buf[0] == 7).all() and (buf[4] == 7).all()
    ws = torch.full((ep.ep_moe_few_workspace_size(1, 3, 2, 4, 40) + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    call(s, "silu", workspace=ws[:-64])
    assert (ws[-64:] == 0x5A).all()


def test_graph_and_streams():
    """Captured and replayed with other inputs in place; two calls on two streams with a workspace each."""
    s = make(13, 1, 8, 4, 16, 512, 256, "bf16")
    other = make(14, 1, 8, 4, 16, 512, 256, "bf16")
    want, want2 = call(s, "silu"), call(other, "silu")
    ws, out = ep.alloc_moe_few_workspace(1, 8, 4, 16, 256), torch.empty_like(s["x"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    live = {n: v.clone() if v is not None else None for n, v in s.items()}
    with torch.cuda.stream(side):
        call(live, "silu", out=out, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(live, "silu", out=out, workspace=ws)
            call(live, "silu", out=out, workspace=ws)   # behind itself, on the same workspace
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for n in ("x", "idx", "weights", "w_gu", "w_down"):
        live[n].copy_(other[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [ep.alloc_moe_few_workspace(1, 8, 4, 16, 256) for _ in range(2)]
    outs = [torch.empty_like(out) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (st, v) in enumerate(zip(streams, (s, other))):
            with torch.cuda.stream(st):
                call(v, "silu", out=outs[i], workspace=spaces[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want2)


def test_weights_past_31_bits():
    """An expert whose weights start behind 2^31 elements (and bytes)."""
    E, H, I = 200, 4096, 1416
    s = make(15, 1, 2, 2, 2, H, I, "bf16")
    w_gu = torch.zeros((E, 2, I, H), dtype=torch.bfloat16, device="cuda")
    w_down = torch.zeros((E, H, I), dtype=torch.bfloat16, device="cuda")
    w_gu[[3, 198]], w_down[[3, 198]] = s["w_gu"], s["w_down"]
    want = call(s, "silu")
    s["idx"] = torch.where(s["idx"] == 0, 3, 198)
    assert torch.equal(call(dict(s, w_gu=w_gu, w_down=w_down), "silu"), want)


def test_empty_batch():
    s = make(16, 1, 1, 2, 4, 64, 32, "bf16")
    e = dict(s, **{n: s[n][:, :0].contiguous() for n in ("x", "idx", "weights")})
    before = ep.ep_launch_count()
    assert call(e, "silu").shape == (1, 0, 64)
    assert ep.ep_launch_count() == before


def test_two_launches():
    s = make(17, 1, 4, 2, 16, 256, 128, "bf16")
    before = ep.ep_launch_count()
    call(s, "silu")
    assert ep.ep_launch_count() == before + 2


def test_binding_refuses():
    s = make(18, 1, 4, 2, 4, 128, 128, "bf16")
    ws = ep.alloc_moe_few_workspace(1, 4, 2, 4, 128)
    out = torch.empty_like(s["x"])
    args = [s["x"], s["idx"], s["weights"], s["w_gu"], None, s["w_down"], None, ep.EP_ACT_SILU, out, ws]
    scales = torch.zeros((4, 2, 1, 1), dtype=torch.uint8, device="cuda")
    for i, bad in ((0, s["x"].float()), (0, s["x"].cpu()), (0, s["x"].transpose(0, 1)), (1, s["idx"].int()), (1, s["idx"][:, :3]),
                   (2, s["weights"].double()), (3, s["w_gu"][:, :1]), (3, s["w_gu"].transpose(2, 3)), (4, scales), (5, s["w_down"][:3]),
                   (6, scales[:, 0]), (8, out.float()), (9, ws[:0].int())):
        with pytest.raises(ValueError):
            ep.ep_moe_few(*args[:i], bad, *args[i + 1:])
    with pytest.raises(ep.EPError):
        ep.ep_moe_few(*args[:9], ws[:-16])
    with pytest.raises(ep.EPError):
        ep.ep_moe_few(*args[:7], ep.EP_ACT_NONE, *args[8:])
