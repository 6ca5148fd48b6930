"""Operators of a mixture-of-experts layer around dispatch and combine, as measured work.

Three operators, each with its gradient:

* gate    -- a router's top-k: logits [R, T_r, E] -> topk_idx, topk_weights (what dispatch and combine read);
* glu     -- the experts' gated projection h = act(x Wg^T) * (x Wu^T) over the receive layouts that dispatch fills,
             bf16, or E4M3 with ue8m0 scales for serving;
* linear  -- a product with bias, activation and residual in its epilogue, y = act(x W^T + b) + r, over the same
             layouts (the experts' down projection; with one expert an ordinary dense layer).

A receive layout holds expert e's rows as one segment: psum[r][l] .. + counts[e] of rank r's cap_rows rows (normal
layout), or the first counts[e] of the expert's own cap_rows rows (packed layout). Rows that belong to no segment are
never read and never written; here they hold NaN on the way in and zeros on the way out.
"""
import math

import numpy as np
import torch

own = False

LISTED = [
    # the decode batch of 16 ranks x 128 tokens, routed: the smallest call of a serving step, where latency counts
    {"name": "gate decode", "op": "gate", "R": 16, "T": 2048, "E": 256, "k": 8, "type": "fp32", "score": "softmax_topk"},
    # routing of a large training or prefill batch (8 ranks x 16384 tokens), probabilities over all experts
    {"name": "gate large", "op": "gate", "R": 8, "T": 131072, "E": 256, "k": 8, "type": "fp32", "score": "softmax"},
    # the router's gradient for 8 ranks x 4096 tokens
    {"name": "gate backward", "op": "gate_backward", "R": 8, "T": 32768, "E": 256, "k": 8, "type": "fp32", "score": "softmax"},
    # a tiny layer (4 ranks x 16 tokens, top-2 of 16 experts): eight rows an expert, bound by latency
    {"name": "glu tiny", "op": "glu", "layout": "normal", "type": "bf16", "R": 4, "E": 16, "T": 64, "k": 2, "zipf": 0.0,
     "align": 1, "H": 256, "I": 128, "act": "silu", "save": False},
    # decode on E4M3 rows in the packed layout, 64 rows an expert on average: bound by reading the weights
    {"name": "glu decode e4m3", "op": "glu", "layout": "packed", "type": "e4m3", "R": 4, "E": 64, "T": 512, "k": 8,
     "zipf": 0.0, "align": 1, "H": 7168, "I": 2048, "act": "silu", "save": False},
    # a training step's forward over 8192 tokens and 32 experts, which keeps gate and up for the backward
    {"name": "glu train", "op": "glu", "layout": "normal", "type": "bf16", "R": 2, "E": 32, "T": 8192, "k": 8,
     "zipf": 0.0, "align": 1, "H": 7168, "I": 2048, "act": "silu", "save": True},
    # its backward: gradients of the rows and of both weights
    {"name": "glu backward", "op": "glu_backward", "layout": "normal", "type": "bf16", "R": 2, "E": 32, "T": 8192, "k": 8,
     "zipf": 0.0, "align": 1, "H": 7168, "I": 2048, "act": "silu"},
    # the same with skewed routing: hot experts, near-empty ones, an intermediate size that no tile divides
    {"name": "glu backward skewed", "op": "glu_backward", "layout": "normal", "type": "bf16", "R": 8, "E": 32, "T": 2048,
     "k": 6, "zipf": 1.2, "align": 128, "H": 4096, "I": 1416, "act": "silu"},
    # decode's down projection on E4M3 rows
    {"name": "linear decode e4m3", "op": "linear", "layout": "packed", "type": "e4m3", "R": 4, "E": 64, "T": 512, "k": 8,
     "zipf": 0.0, "align": 1, "K": 2048, "N": 7168, "act": "none", "bias": False, "residual": False, "save": False},
    # a dense layer over 8192 tokens with all of its epilogue, as a training step's forward
    {"name": "linear dense", "op": "linear", "layout": "normal", "type": "bf16", "R": 1, "E": 1, "T": 8192, "k": 1,
     "zipf": 0.0, "align": 1, "K": 4096, "N": 7168, "act": "gelu", "bias": True, "residual": True, "save": True},
    # the down projection's backward in the same training step as the gated one
    {"name": "linear backward", "op": "linear_backward", "layout": "normal", "type": "bf16", "R": 2, "E": 32, "T": 8192,
     "k": 8, "zipf": 0.0, "align": 1, "K": 2048, "N": 7168, "act": "none", "bias": False},
    # a small dense layer's backward through bias and activation, 777 tokens
    {"name": "linear backward dense", "op": "linear_backward", "layout": "normal", "type": "bf16", "R": 1, "E": 1,
     "T": 777, "k": 1, "zipf": 0.0, "align": 1, "K": 1000, "N": 2048, "act": "silu", "bias": True},
]

# what a drawn case may cost at most: the largest listed ones' products, weights, and rows times width
MOST_FLOPS, MOST_WEIGHTS, MOST_ROWS = 2 * 65536 * 7168 * 4096, 32 * 4096 * 7168, 65536


def listed():
    return [dict(c) for c in LISTED]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["gate", "gate_backward", "glu", "glu_backward", "linear", "linear_backward"])
    while True:
        R = rng.choice([1, 2, 4, 8, 16])
        E = R * _log(rng, 1, 64)
        T = R * _log(rng, 1, 65536 // R)
        k = rng.randint(1, min(E, 16))
        if op.startswith("gate"):
            E = rng.randint(max(k, R), 64) * R if rng.random() < 0.5 else E
            if E <= 1024 and T * E <= 131072 * 256 and T % 1024:
                return {"op": op, "R": R, "T": T, "E": E, "k": k, "type": rng.choice(["fp32", "bf16"]),
                        "score": rng.choice(["softmax", "softmax_topk"])}
            continue
        kind = "e4m3" if not op.endswith("backward") and rng.random() < 0.4 else "bf16"
        unit = 128 if kind == "e4m3" else 8
        wide, narrow = unit * max(1, _log(rng, 64, 7168) // unit), unit * max(1, _log(rng, 64, 4096) // unit)
        packed = rng.random() < 0.4 and T <= 4096
        if T % 1024 == 0 or wide % 1024 == 0 or narrow % 512 == 0:
            continue  # the listed cases have the round sizes
        c = {"op": op, "layout": "packed" if packed else "normal", "type": kind, "R": R, "E": E, "T": T, "k": k,
             "zipf": rng.choice([0.0, 0.0, 1.2]) if T * k <= 16384 else 0.0, "align": 1 if packed else rng.choice([1, 4, 128])}
        if op.startswith("glu"):
            c.update(H=wide, I=narrow, act=rng.choice(["silu", "gelu", "relu"]))
            N = 2 * narrow
        else:
            c.update(K=narrow, N=wide, act=rng.choice(["none", "none", "relu", "silu", "gelu"]), bias=rng.random() < 0.5)
            N = narrow
        if op == "linear":
            c["residual"] = rng.random() < 0.5
        if not op.endswith("backward"):
            c["save"] = rng.random() < 0.3 and kind == "bf16" and (op == "glu" or c["act"] != "none")
        if T * k * 2 * wide * N <= MOST_FLOPS and E * wide * N <= MOST_WEIGHTS and T * k <= MOST_ROWS and (not packed or E * T * (wide + N) <= 1 << 30):
            return c


# ---- inputs ----

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _routing(case, seed):
    """(counts [E] and starts [E] as numpy, rows a rank or an expert holds): tokens drawn over experts, uniform or Zipf."""
    rng = np.random.default_rng([seed, 101])
    R, E, T, k = (case[n] for n in "RETk")
    p = np.arange(1, E + 1, dtype=np.float64) ** -case["zipf"]
    counts = rng.multinomial(T * k, p / p.sum())
    if case["layout"] == "packed":
        counts = np.minimum(counts, T)  # a token reaches an expert once
        return counts, np.arange(E, dtype=np.int64) * T, T
    aligned = -(-counts // case["align"]) * case["align"]
    psum = np.zeros((R, E // R + 1), dtype=np.int64)
    psum[:, 1:] = np.cumsum(aligned.reshape(R, -1), axis=1)
    # the receive buffer is sized before the routing is known: the busiest rank's expected rows and a wide margin
    busy = T * k * float((p / p.sum()).reshape(R, -1).sum(1).max())
    cap = max(int(busy + 8 * math.sqrt(busy) + 16) + (E // R) * (case["align"] - 1), int(psum[:, -1].max()))
    return counts, (psum[:, :-1] + np.arange(R)[:, None] * cap).reshape(-1), cap


def _normal(g, shape, std, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=g.device, dtype=dtype).mul_(std)


def _e4m3(g, shape, std):
    """E4M3 bytes of normal values, as a quantiser with power-of-two scales leaves them (largest of a block near 448 * 2^-1)."""
    return _normal(g, shape, 96.0 * std).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed * 7919 + 13)
    s = {"case": case}
    if case["op"].startswith("gate"):
        return _prepare_gate(s, case, seed, g)
    dev = g.device
    R, E = case["R"], case["E"]
    counts, starts, cap = _routing(case, seed)
    glu = case["op"].startswith("glu")
    K, N = (case["H"], 2 * case["I"]) if glu else (case["K"], case["N"])
    rows = (E if case["layout"] == "packed" else R) * cap
    lead = (R, E // R, cap) if case["layout"] == "packed" else (R, cap)
    s["counts"] = torch.from_numpy(counts.astype(np.int32)).reshape(R, E // R).to(dev)
    s["psum"] = None
    if case["layout"] == "normal":
        psum = np.zeros((R, E // R + 1), dtype=np.int64)
        psum[:, :-1] = starts.reshape(R, -1) - np.arange(R)[:, None] * cap
        psum[:, -1] = psum[:, -2] + -(-counts.reshape(R, -1)[:, -1] // case["align"]) * case["align"]
        s["psum"] = torch.from_numpy(psum).to(dev)
    s["most"] = max(1, int(counts.max()))  # the plain form's padded length
    s["starts"] = torch.from_numpy(starts).to(dev)
    at = torch.arange(rows, device=dev)
    seg = torch.searchsorted(s["starts"], at, right=True) - 1
    free = (at >= s["starts"][seg] + s["counts"].reshape(-1)[seg]).unsqueeze(1)  # rows of no segment

    def rows_of(width, std):
        return _normal(g, (rows, width), std).masked_fill_(free, float("nan")).reshape(*lead, width)

    wshape = (E, 2, case["I"], K) if glu else (E, N, K)
    if case["type"] == "e4m3":
        s["x"] = _e4m3(g, (rows, K), 1.0).masked_fill_(free, 0x7F).reshape(*lead, K)
        s["x_scales"] = torch.randint(118, 122, (*lead[:-1], K // 128, cap), generator=g, device=dev, dtype=torch.uint8)
        s["w"] = _e4m3(g, wshape, 1.0)
        s["w_scales"] = torch.randint(113, 116, (*wshape[:-2], wshape[-2] // 128, K // 128), generator=g, device=dev, dtype=torch.uint8)
    else:
        s["x"] = rows_of(K, 1.0)
        s["x_scales"] = s["w_scales"] = None
        s["w"] = _normal(g, wshape, K ** -0.5)
    s["bias"] = _normal(g, (E, N), 0.5) if case.get("bias") else None
    s["residual"] = rows_of(N, 1.0) if case.get("residual") else None
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device=dev)  # noqa: E731
    if case["op"] == "glu":
        s["h"] = zeros(*lead, case["I"])
        s["gu"] = zeros(*lead, 2, case["I"]) if case["save"] else None
    elif case["op"] == "glu_backward":
        s["dh"] = rows_of(case["I"], 1.0)
        s["gu"] = rows_of(N, 1.0).reshape(*lead, 2, case["I"])
        s["dgu"], s["dx"], s["dw"] = zeros(*lead, 2, case["I"]), zeros(*lead, K), zeros(*wshape)
    elif case["op"] == "linear":
        s["y"] = zeros(*lead, N)
        s["pre"] = zeros(*lead, N) if case["save"] else None
    else:
        s["dy"] = rows_of(N, 1.0)
        s["pre"] = rows_of(N, 1.0) if case["act"] != "none" else None
        s["dpre"] = zeros(*lead, N) if case["act"] != "none" else None
        s["dx"], s["dw"] = zeros(*lead, K), zeros(*wshape)
        s["dbias"] = zeros(E, N) if case["bias"] else None
    return s


def _prepare_gate(s, case, seed, g):
    R, T, E, k = (case[n] for n in "RTEk")
    dtype = torch.float32 if case["type"] == "fp32" else torch.bfloat16
    logits = _normal(g, (R, T // R, E), 1.5, torch.float32)
    # experts switched off for a token hold -inf, as do all of a padding token's
    off = torch.rand((R, T // R, E), generator=g, device=g.device) < 0.02
    off |= torch.rand((R, T // R, 1), generator=g, device=g.device) < 0.01
    s["logits"] = logits.masked_fill_(off, -math.inf).to(dtype)
    if case["op"] == "gate_backward":
        s["topk_idx"] = _gate(s["logits"], k, case["score"])[0]
        s["grad"] = _normal(g, (R, T // R, k), 1.0, torch.float32)
        s["grad_logits"] = torch.empty_like(s["logits"])
    else:
        s["topk_idx"] = torch.empty((R, T // R, k), dtype=torch.int64, device=g.device)
        s["topk_weights"] = torch.empty((R, T // R, k), dtype=torch.float32, device=g.device)
    return s


# ---- the operators in their plain form ----

def _gate(logits, k, score):
    """Top-k of the logits, ties to the lower expert; an expert at -inf is never taken (index -1, weight 0)."""
    l = logits.float()
    top, idx = torch.sort(l, dim=-1, descending=True, stable=True)
    top, idx = top[..., :k], idx[..., :k]
    none = top == -math.inf
    most = top[..., :1].masked_fill(none[..., :1], 0.0)
    below = torch.exp((l if score == "softmax" else top) - most).sum(-1, keepdim=True)
    w = torch.exp(top - most) / below.masked_fill(none[..., :1], 1.0)
    return idx.masked_fill(none, -1), w.masked_fill(none, 0.0)


def _gate_backward(logits, idx, grad, score):
    l = logits.float()
    none = idx < 0
    at = idx.clamp(min=0)
    grad = grad.masked_fill(none, 0.0)
    chosen = torch.gather(l, -1, at).masked_fill(none, -math.inf)
    whole = l if score == "softmax" else chosen
    most = whole.amax(-1, keepdim=True)
    most = most.masked_fill(most == -math.inf, 0.0)
    total = torch.exp(whole - most).sum(-1, keepdim=True)
    total = total.masked_fill(total == 0, 1.0)
    w = torch.exp(chosen - most) / total
    inner = (w * grad).sum(-1, keepdim=True)
    if score == "softmax":
        d = -torch.exp(l - most) / total * inner
        d = d.scatter_add(-1, at, w * grad)
    else:
        d = torch.zeros_like(l).scatter_add(-1, at, w * (grad - inner))
    return d.to(logits.dtype)


def _act(z, name):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return torch.relu(z) if name == "relu" else z


def _act_slope(z, name):
    if name == "silu":
        q = torch.sigmoid(z)
        return q * (1 + z * (1 - q))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (0.5 / math.pi) ** 0.5
    return (z > 0).to(z.dtype)


def _segments(s):
    """Row numbers [E, most] of the padded segments, and which of them are rows of the expert."""
    j = torch.arange(s["most"], device=s["counts"].device)
    valid = j < s["counts"].reshape(-1, 1)
    return torch.where(valid, s["starts"].unsqueeze(1) + j, 0), valid


def _take(t, seg):
    """Rows [rows, width] -> [E, most, width] in 32 bits, zeros where the segment has ended."""
    return t[seg[0]].float().masked_fill_(~seg[1].unsqueeze(-1), 0.0)


def _put(v, seg, shape):
    """[E, most, width] -> rows of a zeroed bf16 tensor of `shape`."""
    rows, width = math.prod(shape[:-1]), shape[-1]
    out = torch.zeros((rows + 1, width), dtype=torch.bfloat16, device=v.device)
    out[torch.where(seg[1], seg[0], rows)] = v.to(torch.bfloat16)
    return out[:rows].reshape(shape)


def _scale(b):
    return torch.exp2(b.float() - 127)


def _x(s):
    """The rows in 32 bits, [rows, K], scales applied."""
    x = s["x"]
    if x.dtype != torch.uint8:
        return x.reshape(-1, x.shape[-1])
    q = x.view(torch.float8_e4m3fn).float()
    sc = _scale(s["x_scales"]).transpose(-1, -2).unsqueeze(-1)
    return (q.reshape(*q.shape[:-1], -1, 128) * sc).reshape(-1, x.shape[-1])


def _w(s):
    w = s["w"]
    if w.dtype != torch.uint8:
        return w.float()
    q = w.view(torch.float8_e4m3fn).float()
    blocks = q.reshape(*q.shape[:-2], q.shape[-2] // 128, 128, q.shape[-1] // 128, 128)
    return (blocks * _scale(s["w_scales"])[..., :, None, :, None]).reshape(q.shape)


def _plain(s):
    case = s["case"]
    if case["op"] == "gate":
        idx, w = _gate(s["logits"], case["k"], case["score"])
        return {"topk_idx": idx, "topk_weights": w}
    if case["op"] == "gate_backward":
        return {"grad_logits": _gate_backward(s["logits"], s["topk_idx"], s["grad"], case["score"])}
    seg = _segments(s)
    x, w = _take(_x(s), seg), _w(s)
    lead = s["x"].shape[:-1]
    if case["op"] == "glu":
        gate, up = x @ w[:, 0].transpose(1, 2), x @ w[:, 1].transpose(1, 2)
        out = {"h": _put(_act(gate, case["act"]) * up, seg, (*lead, case["I"]))}
        if case["save"]:
            out["gu"] = _put(torch.cat([gate, up], -1), seg, (*lead, 2 * case["I"])).reshape(*lead, 2, case["I"])
        return out
    if case["op"] == "linear":
        z = x @ w.transpose(1, 2)
        z = z + s["bias"].float().unsqueeze(1) if case["bias"] else z
        y = _act(z, case["act"])
        y = y + _take(s["residual"].reshape(-1, case["N"]), seg) if case["residual"] else y
        out = {"y": _put(y, seg, (*lead, case["N"]))}
        if case["save"]:
            out["pre"] = _put(z, seg, (*lead, case["N"]))
        return out
    if case["op"] == "glu_backward":
        dh = _take(s["dh"].reshape(-1, case["I"]), seg)
        gate, up = _take(s["gu"].reshape(-1, 2 * case["I"]), seg).chunk(2, -1)
        d = torch.cat([dh * up * _act_slope(gate, case["act"]), dh * _act(gate, case["act"])], -1)
        w = w.reshape(w.shape[0], -1, w.shape[-1])
    else:
        d = _take(s["dy"].reshape(-1, case["N"]), seg)
        if case["act"] != "none":
            d = d * _act_slope(_take(s["pre"].reshape(-1, case["N"]), seg), case["act"])
    out = {"dx": _put(d @ w, seg, s["x"].shape), "dw": (d.transpose(1, 2) @ x).to(torch.bfloat16).reshape(s["w"].shape)}
    if case.get("bias"):
        out["dbias"] = d.sum(1).to(torch.bfloat16)
    return out


# ---- the framework's calls ----

def _own(s):
    from combine_get_dispatch_gb300 import ep

    case = s["case"]
    if case["op"] == "gate":
        ep.ep_gate_topk(s["logits"], ep.GATE_SCORES[case["score"]], s["topk_idx"], s["topk_weights"])
        return {"topk_idx": s["topk_idx"], "topk_weights": s["topk_weights"]}
    if case["op"] == "gate_backward":
        ep.ep_gate_topk_backward(s["logits"], ep.GATE_SCORES[case["score"]], s["topk_idx"], s["grad"], s["grad_logits"])
        return {"grad_logits": s["grad_logits"]}
    act = ep.ACTS[case["act"]]
    if case["op"] == "glu":
        ep.ep_expert_glu(s["x"], s["x_scales"], s["w"], s["w_scales"], s["counts"], s["psum"], act, s["h"], gu=s["gu"])
        return {n: s[n] for n in ("h", "gu") if s[n] is not None}
    if case["op"] == "linear":
        ep.ep_expert_linear(s["x"], s["x_scales"], s["w"], s["w_scales"], s["bias"], s["residual"], s["counts"], s["psum"], act,
                            s["y"], pre=s["pre"])
        return {n: s[n] for n in ("y", "pre") if s[n] is not None}
    if case["op"] == "glu_backward":
        ep.ep_expert_glu_backward(s["dh"], s["gu"], s["x"], s["w"], s["counts"], s["psum"], act, s["dgu"], s["dx"], s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    ep.ep_expert_linear_backward(s["dy"], s["pre"], s["x"], s["w"], s["counts"], s["psum"], act, s["dpre"], s["dx"], s["dw"],
                                 dbias=s["dbias"])
    return {n: s[n] for n in ("dx", "dw", "dbias") if s[n] is not None}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----

def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"].startswith("gate"):
        wide = 4 if case["type"] == "fp32" else 2
        if case["op"] == "gate":
            return {"bytes": T * (E * wide + k * 12), "flops": 0}
        return {"bytes": T * (2 * E * wide + k * 12), "flops": 0}
    rows = T * k
    glu = case["op"].startswith("glu")
    K, N = (case["H"], 2 * case["I"]) if glu else (case["K"], case["N"])
    p = np.arange(1, E + 1, dtype=np.float64) ** -case["zipf"]
    used = float(np.sum(1 - (1 - p / p.sum()) ** rows))  # experts that get a row, on average
    one = 1 if case["type"] == "e4m3" else 2
    flops = 2 * rows * K * N
    if case["op"].endswith("backward"):
        read = 2 * rows * (N * (1 if case["act"] == "none" else 2) - (case["I"] if glu else 0) + K) + 2 * used * N * K
        return {"bytes": int(read + 2 * (rows * K + E * N * K)), "flops": 2 * flops}
    out = case["I"] if glu else N
    byte = rows * K * one + used * N * K * one + 2 * rows * out * (2 if case.get("residual") else 1)
    return {"bytes": int(byte + (2 * rows * N if case["save"] else 0)), "flops": flops}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("gate"):
        return _exact_gate(case, s)
    counts, starts, _ = _routing(case, seed)
    if case["T"] * case["k"] * 4e-12 * case.get("H", case.get("K")) * case.get("I", case.get("N")) > 20:
        return None
    rows = {n: s[n].reshape(-1, math.prod(s[n].shape[-2:]) if n == "gu" else s[n].shape[-1])
            for n in ("x", "dh", "dy", "gu", "pre", "residual") if s.get(n) is not None}
    names = {"glu": ["h"] + ["gu"] * bool(case.get("save")), "linear": ["y"] + ["pre"] * bool(case.get("save")),
             "glu_backward": ["dx", "dw"], "linear_backward": ["dx", "dw"] + ["dbias"] * bool(case.get("bias"))}[case["op"]]
    out = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=s["x"].device) for n in names}
    flat = {n: v.reshape(len(rows["x"]), -1) for n, v in out.items() if n not in ("dw", "dbias")}
    for e in range(case["E"]):
        a, b = int(starts[e]), int(starts[e] + counts[e])
        if a == b:
            continue
        w = s["w"][e].reshape(-1, s["w"].shape[-1])
        x = rows["x"][a:b]
        if case["type"] == "e4m3":
            per = math.prod(s["x_scales"].shape[:-2])
            cap = len(rows["x"]) // per
            sc = s["x_scales"].reshape(per, -1, cap)[a // cap][:, a % cap: a % cap + b - a].t()
            x = x.view(torch.float8_e4m3fn).double() * 2.0 ** (sc.double() - 127).repeat_interleave(128, 1)
            ws = s["w_scales"][e].reshape(-1, s["w_scales"].shape[-1]).double()
            w = w.view(torch.float8_e4m3fn).double() * (2.0 ** (ws - 127)).repeat_interleave(128, 0).repeat_interleave(128, 1)
        x, w = x.double(), w.double()
        if case["op"] == "glu":
            z = x @ w.t()
            gate, up = z[:, :case["I"]], z[:, case["I"]:]
            flat["h"][a:b] = _exact_act(gate, case["act"])[0] * up
            if case["save"]:
                flat["gu"][a:b] = z
            continue
        if case["op"] == "linear":
            z = x @ w.t() + (s["bias"][e].double() if case["bias"] else 0.0)
            flat["y"][a:b] = _exact_act(z, case["act"])[0] + (rows["residual"][a:b].double() if case["residual"] else 0.0)
            if case["save"]:
                flat["pre"][a:b] = z
            continue
        if case["op"] == "glu_backward":
            dh, gu = rows["dh"][a:b].double(), rows["gu"][a:b].double()
            value, slope = _exact_act(gu[:, :case["I"]], case["act"])
            d = torch.cat((dh * gu[:, case["I"]:] * slope, dh * value), 1)
        else:
            d = rows["dy"][a:b].double()
            d = d * _exact_act(rows["pre"][a:b].double(), case["act"])[1] if case["act"] != "none" else d
        flat["dx"][a:b] = d @ w
        out["dw"][e] = (d.t() @ x).reshape(out["dw"][e].shape)
        if case.get("bias"):
            out["dbias"][e] = d.sum(0)
    return out


def _exact_act(z, name):
    """The activation and its slope."""
    if name == "silu":
        e = torch.exp(-z)
        return z / (1 + e), 1 / (1 + e) + z * e / (1 + e) ** 2
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "relu":
        return z.clamp(min=0), torch.where(z > 0, 1.0, 0.0).double()
    return z, torch.ones_like(z)


def _exact_gate(case, s):
    l = s["logits"].double().cpu().numpy().reshape(-1, case["E"])
    k = case["k"]
    with np.errstate(invalid="ignore"):
        top = l.max(1, keepdims=True)
        e = np.exp(l - np.where(np.isinf(top), 0.0, top))
    if case["op"] == "gate":
        idx = np.argsort(-l, axis=1, kind="stable")[:, :k]
    else:
        idx = s["topk_idx"].cpu().numpy().reshape(-1, k)
    at = np.maximum(idx, 0)
    dead = (np.take_along_axis(l, at, 1) == -np.inf) | (idx < 0)
    part = np.where(dead, 0.0, np.take_along_axis(e, at, 1))
    total = (e if case["score"] == "softmax" else part).sum(1, keepdims=True)
    w = part / np.where(total == 0, 1.0, total)
    shape = s["logits"].shape[:2]
    if case["op"] == "gate":
        return {"topk_idx": np.where(dead, -1, idx).reshape(*shape, k), "topk_weights": w.reshape(*shape, k)}
    g = np.where(dead, 0.0, s["grad"].double().cpu().numpy().reshape(-1, k))
    inner = (w * g).sum(1, keepdims=True)
    d = -(e / np.where(total == 0, 1.0, total)) * inner if case["score"] == "softmax" else np.zeros_like(l)
    rows = np.arange(len(l))[:, None]
    np.add.at(d, (rows, at), np.where(dead, 0.0, w * (g if case["score"] == "softmax" else g - inner)))
    return {"grad_logits": d.reshape(s["logits"].shape)}
