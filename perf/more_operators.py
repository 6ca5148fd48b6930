"""Operators on the experts' whole weight stacks, as measured work.

Three operators, for the two ends of a mixture-of-experts layer's life:

* few    -- the whole layer for a few tokens, from routed tokens to combined output without a dispatch between:
            out[t] = sum_j weight[t, j] W_down[e] (act(W_gate[e] x[t]) * (W_up[e] x[t])), e = idx[t, j];
            weights in bf16, or in E4M3 with one ue8m0 scale per 128 x 128 block, tokens in bf16;
* ortho  -- the orthogonalised form of each matrix of a stack, by Newton-Schulz products:
            X = G / (|G| + eps), then (a, b, c) a step: X <- a X + (b A + c A^2) X, A = X X^T
            (of the transposed matrix where it has more rows than columns);
* muon   -- the optimiser's step on a stack of weights from the gradient that the experts' backward leaves:
            m <- mu m + g, u = g + mu m (Nesterov) or m, w <- (1 - lr decay) w - lr scale ortho(u),
            momentum and weights in 32 bits, with the bf16 copy that the products read.

Stacks are what the expert calls read and write: [E, 2, I, H] for gate and up, [E, H, I] for the down projection, one
matrix an expert (and half).
"""
import math

import numpy as np
import torch

own = False

# (a, b, c) of every step: the quintic that lifts small singular values most, and the cubic that converges
POLYNOMIALS = {"quintic": (3.4445, -4.7750, 2.0315), "cubic": (1.5, -0.5, 0.0)}
EPS = 1e-7

LISTED = [
    # the tiny layer (top-2 of 16 experts) with four tokens: the smallest call, where latency counts
    {"name": "few tiny", "op": "few", "type": "bf16", "T": 4, "k": 2, "E": 16, "H": 256, "I": 128, "act": "silu", "zipf": 0.0, "pad": 0},
    # one token through a large layer, E4M3 weights: a single user's decode step, bound by reading eight experts
    {"name": "few one token e4m3", "op": "few", "type": "e4m3", "T": 1, "k": 8, "E": 128, "H": 7168, "I": 2048, "act": "silu", "zipf": 0.0, "pad": 0},
    # one token, bf16 weights, widths that no tile divides
    {"name": "few one token", "op": "few", "type": "bf16", "T": 1, "k": 6, "E": 32, "H": 4096, "I": 1416, "act": "silu", "zipf": 0.0, "pad": 0},
    # a decode batch of 32 users on E4M3 weights: most experts reached, by two tokens each
    {"name": "few batch e4m3", "op": "few", "type": "e4m3", "T": 32, "k": 8, "E": 128, "H": 7168, "I": 2048, "act": "silu", "zipf": 0.0, "pad": 0},
    # skewed routing of a padded batch: hot experts with many tokens, the last rows of the batch unused
    {"name": "few batch skewed", "op": "few", "type": "bf16", "T": 21, "k": 6, "E": 32, "H": 4096, "I": 1416, "act": "gelu", "zipf": 1.2, "pad": 3},
    # drafted tokens of several users, few experts: sixteen tokens an expert, the most that the layer takes at once
    {"name": "few drafted", "op": "few", "type": "bf16", "T": 64, "k": 2, "E": 8, "H": 4096, "I": 2048, "act": "silu", "zipf": 0.0, "pad": 0},
    # one dense layer's gradient (1000 -> 2048), more rows than columns: bound by the chain of small products
    {"name": "ortho dense", "op": "ortho", "type": "bf16", "count": 1, "M": 2048, "N": 1000, "poly": "quintic", "steps": 5, "idle": 0},
    # gate and up gradients of eight experts, one of which saw no token; widths that no tile divides
    {"name": "ortho gate up", "op": "ortho", "type": "bf16", "count": 16, "M": 1416, "N": 4096, "poly": "quintic", "steps": 5, "idle": 2},
    # down projections of four large experts, by the convergent cubic
    {"name": "ortho down cubic", "op": "ortho", "type": "bf16", "count": 4, "M": 7168, "N": 2048, "poly": "cubic", "steps": 6, "idle": 0},
    # the tiny layer's gate and up (16 experts), gradients accumulated in 32 bits: launch after launch of one tile a matrix
    {"name": "muon tiny", "op": "muon", "type": "fp32", "count": 32, "M": 128, "N": 256, "poly": "quintic", "steps": 5, "idle": 1, "nesterov": True, "lr": 1e-4, "decay": 0.1},
    # a training step's gate and up of four experts, gradients as the experts' backward leaves them
    {"name": "muon gate up", "op": "muon", "type": "bf16", "count": 8, "M": 2048, "N": 4096, "poly": "quintic", "steps": 5, "idle": 0, "nesterov": True, "lr": 1e-4, "decay": 0.1},
    # down projections of eight narrow experts, plain momentum
    {"name": "muon down", "op": "muon", "type": "bf16", "count": 8, "M": 4096, "N": 1416, "poly": "quintic", "steps": 5, "idle": 0, "nesterov": False, "lr": 5e-5, "decay": 0.0},
]

# what a drawn case may cost at most: the largest listed ones' weights held, weights read, products and elements
MOST_HELD, MOST_READ, MOST_FLOPS, MOST_ELEMENTS = 128 * 3 * 7168 * 2048, 111 * 3 * 7168 * 2048, 5 * 8 * (4 * 2048 ** 2 * 4096 + 2 * 2048 ** 3), 16 * 1416 * 4096


def listed():
    return [dict(c) for c in LISTED]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["few", "few", "ortho", "muon"])
    while True:
        if op == "few":
            kind = rng.choice(["bf16", "e4m3"])
            unit = 128 if kind == "e4m3" else 8
            E = _log(rng, 1, 256)
            c = {"op": op, "type": kind, "T": _log(rng, 1, 64), "k": rng.randint(1, min(E, 10)), "E": E, "H": unit * max(1, _log(rng, 64, 7168) // unit),
                 "I": unit * max(1, _log(rng, 64, 4096) // unit), "act": rng.choice(["silu", "silu", "gelu", "relu"]), "zipf": rng.choice([0.0, 0.0, 1.2])}
            c["pad"] = rng.randint(0, c["T"] // 4)
            each = 3 * c["H"] * c["I"] * (1 if kind == "e4m3" else 2)
            if c["E"] * each <= MOST_HELD and min(c["E"], c["T"] * c["k"]) * each <= MOST_READ and c["H"] % 1024 and c["I"] % 512:
                return c
            continue
        poly = rng.choice(["quintic", "quintic", "cubic"])
        c = {"op": op, "type": rng.choice(["bf16", "bf16", "fp32"]), "count": _log(rng, 1, 64), "M": _log(rng, 16, 8192), "N": 8 * _log(rng, 2, 1024),
             "poly": poly, "steps": 5 if poly == "quintic" else rng.randint(3, 8)}
        c["idle"] = rng.randint(0, 2) if c["count"] > 4 else 0
        if op == "muon":
            c.update(nesterov=rng.random() < 0.5, lr=rng.choice([2e-5, 5e-5, 1e-4]), decay=rng.choice([0.0, 0.1]))
        S, L = min(c["M"], c["N"]), max(c["M"], c["N"])
        if c["steps"] * c["count"] * (4 * S * S * L + 2 * S ** 3) <= MOST_FLOPS and c["count"] * S * L <= MOST_ELEMENTS and c["M"] % 1024 and c["N"] % 1024:
            return c


# ---- inputs ----

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, shape, std, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=g.device, dtype=dtype).mul_(std)


def _e4m3(g, shape):
    """E4M3 bytes of normal values, as a quantiser with power-of-two scales leaves them (largest of a block near 448 / 2)."""
    return _normal(g, shape, 96.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed * 7919 + 13)
    return _prepare_few(case, seed, g) if case["op"] == "few" else _prepare_stack(case, g)


def _routing(case, seed):
    """[T, k] experts, distinct within a token, drawn uniformly or by Zipf; -1 in the padded rows at the end."""
    rng = np.random.default_rng([seed, 103])
    T, k, E = case["T"], case["k"], case["E"]
    p = np.arange(1, E + 1, dtype=np.float64) ** -case["zipf"]
    # the k largest of log p + Gumbel noise: k draws without repetition
    idx = np.argsort(-(np.log(p) + rng.gumbel(size=(T, E))), axis=1)[:, :k].astype(np.int64)
    idx[T - case["pad"]:] = -1
    return idx


def _prepare_few(case, seed, g):
    dev = g.device
    T, k, E, H, I = (case[n] for n in ("T", "k", "E", "H", "I"))
    idx = _routing(case, seed)
    s = {"case": case, "x": _normal(g, (1, T, H), 1.0), "topk_idx": torch.from_numpy(idx).reshape(1, T, k).to(dev)}
    s["topk_weights"] = torch.softmax(_normal(g, (1, T, k), 1.0, torch.float32), -1)
    s["x"][:, T - case["pad"]:] = float("nan")  # what a padded batch's unused rows hold is nobody's business
    if case["type"] == "e4m3":
        s["w_gu"], s["w_down"] = _e4m3(g, (E, 2, I, H)), _e4m3(g, (E, H, I))
        # values near H^-0.5 and I^-0.5, as the bf16 weights: 96 * 2^(scale - 127)
        low = lambda width: int(round(math.log2(width ** -0.5 / 96.0))) + 127  # noqa: E731
        s["w_gu_scales"] = torch.randint(low(H), low(H) + 2, (E, 2, I // 128, H // 128), generator=g, device=dev, dtype=torch.uint8)
        s["w_down_scales"] = torch.randint(low(I), low(I) + 2, (E, H // 128, I // 128), generator=g, device=dev, dtype=torch.uint8)
    else:
        s["w_gu"], s["w_down"] = _normal(g, (E, 2, I, H), H ** -0.5), _normal(g, (E, H, I), I ** -0.5)
        s["w_gu_scales"] = s["w_down_scales"] = None
    s["out"] = torch.empty((1, T, H), dtype=torch.bfloat16, device=dev)
    # the plain form's table: the experts that got a token, and each one's slots, padded with slot T k
    used, counts = np.unique(idx[idx >= 0], return_counts=True)
    slots = np.full((len(used), max(1, counts.max(initial=0))), T * k, dtype=np.int64)
    flat = idx.reshape(-1)
    order = np.argsort(flat, kind="stable")
    order = order[flat[order] >= 0]
    column = np.arange(len(order)) - np.repeat(np.cumsum(counts) - counts, counts)
    slots[np.searchsorted(used, flat[order]), column] = order
    s["used"], s["slots"] = torch.from_numpy(used).to(dev), torch.from_numpy(slots).to(dev)
    if own:
        from combine_get_dispatch_gb300 import ep

        s["workspace"] = ep.alloc_moe_few_workspace(1, T, k, E, I, device=dev)
    return s


def _prepare_stack(case, g):
    dev = g.device
    shape = (case["count"], case["M"], case["N"])
    # a gradient's rows and columns differ in size by a few times: outputs and inputs that are more or less active
    rows = torch.exp(_normal(g, (case["count"], case["M"], 1), 0.5, torch.float32))
    columns = torch.exp(_normal(g, (case["count"], 1, case["N"]), 0.5, torch.float32))
    grad = _normal(g, shape, 1e-3, torch.float32).mul_(rows).mul_(columns)
    if case["idle"]:
        grad[-case["idle"]:] = 0  # an expert without rows: the backward leaves zeros
    s = {"case": case, "g": grad if case["type"] == "fp32" else grad.to(torch.bfloat16)}
    if case["op"] == "ortho":
        s["out"] = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    else:
        s["m"] = _normal(g, shape, 1e-2, torch.float32).mul_(rows).mul_(columns)  # twenty steps' worth
        s["w"] = _normal(g, shape, 0.02, torch.float32)
        s["w16"] = s["w"].to(torch.bfloat16)
    if own:
        from combine_get_dispatch_gb300 import ep

        s["workspace"] = ep.alloc_orthogonalize_workspace(shape, device=dev)
    return s


MU = 0.95


def _scale_of(case):
    """Of the orthogonalised update, so that its entries are about 0.2."""
    return 0.2 * math.sqrt(max(case["M"], case["N"]))


# ---- the operators in their plain form ----

def _act(z, name):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return torch.relu(z)


def _dequantised(w, scales):
    """The used experts' weights in 32 bits."""
    if scales is None:
        return w.float()
    q = w.view(torch.float8_e4m3fn).float()
    blocks = q.reshape(*q.shape[:-2], q.shape[-2] // 128, 128, q.shape[-1] // 128, 128)
    return (blocks * torch.exp2(scales.float() - 127)[..., :, None, :, None]).reshape(q.shape)


def _few(s):
    case, used, slots = s["case"], s["used"], s["slots"]
    T, k, H = case["T"], case["k"], case["H"]
    taken = lambda t: None if t is None else t[used]  # noqa: E731
    x = s["x"].reshape(T, H).float()[(slots // k).clamp(max=T - 1)]
    z = x @ _dequantised(taken(s["w_gu"]), taken(s["w_gu_scales"])).reshape(len(used), -1, H).transpose(1, 2)
    gate, up = z.chunk(2, -1)
    y = (_act(gate, case["act"]) * up) @ _dequantised(taken(s["w_down"]), taken(s["w_down_scales"])).transpose(1, 2)
    each = torch.zeros((T * k + 1, H), dtype=torch.float32, device=x.device)
    each[slots.reshape(-1)] = y.reshape(-1, H)
    weights = s["topk_weights"].masked_fill(s["topk_idx"] < 0, 0.0)
    out = (each[:T * k].reshape(1, T, k, H).masked_fill_((s["topk_idx"] < 0).unsqueeze(-1), 0.0) * weights.unsqueeze(-1)).sum(2)
    return {"out": out.to(torch.bfloat16)}


def _orthogonalised(u, case):
    x = u.float()
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + EPS)
    tall = case["M"] > case["N"]
    x = x.transpose(1, 2) if tall else x
    a, b, c = POLYNOMIALS[case["poly"]]
    for _ in range(case["steps"]):
        A = x @ x.transpose(1, 2)
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.transpose(1, 2) if tall else x


def _muon(s):
    case = s["case"]
    g = s["g"].float()
    m = MU * s["m"] + g
    o = _orthogonalised(g + MU * m if case["nesterov"] else m, case)
    w = (1 - case["lr"] * case["decay"]) * s["w"] - case["lr"] * _scale_of(case) * o
    return {"m": s["m"].copy_(m), "w": s["w"].copy_(w), "w16": s["w16"].copy_(w)}


def _plain(s):
    if s["case"]["op"] == "few":
        return _few(s)
    if s["case"]["op"] == "ortho":
        return {"out": _orthogonalised(s["g"], s["case"]).to(torch.bfloat16)}
    return _muon(s)


# ---- the framework's calls ----

def _own(s):
    from combine_get_dispatch_gb300 import ep

    case = s["case"]
    if case["op"] == "few":
        ep.ep_moe_few(s["x"], s["topk_idx"], s["topk_weights"], s["w_gu"], s["w_gu_scales"], s["w_down"], s["w_down_scales"], ep.ACTS[case["act"]],
                      s["out"], s["workspace"])
        return {"out": s["out"]}
    steps = [POLYNOMIALS[case["poly"]]] * case["steps"]
    if case["op"] == "ortho":
        ep.ep_orthogonalize(s["g"], steps, s["out"], s["workspace"], eps=EPS)
        return {"out": s["out"]}
    ep.ep_muon_update(s["g"], s["m"], s["w"], s["w16"], steps, s["workspace"], lr=case["lr"], scale=_scale_of(case), momentum=MU,
                      nesterov=case["nesterov"], weight_decay=case["decay"], eps=EPS)
    return {"m": s["m"], "w": s["w"], "w16": s["w16"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----

def work(case):
    if case["op"] == "few":
        T, k, E, H, I = (case[n] for n in ("T", "k", "E", "H", "I"))
        tokens = T - case["pad"]
        p = np.arange(1, E + 1, dtype=np.float64) ** -case["zipf"]
        p /= p.sum()
        # experts reached on average: a token takes expert e with probability about 1 - (1 - p)^n, n so that k are taken
        low, high = 0.0, 1e6
        for _ in range(100):
            n = 0.5 * (low + high)
            low, high = (n, high) if np.sum(1 - (1 - p) ** n) < k else (low, n)
        used = float(np.sum(1 - (1 - p) ** (n * tokens)))
        each = 3 * H * I * (2 if case["type"] == "bf16" else 1) + (3 * (H // 128) * (I // 128) if case["type"] == "e4m3" else 0)
        return {"bytes": int(used * each) + T * (4 * H + 12 * k), "flops": 2 * tokens * k * 3 * H * I}
    S, L = min(case["M"], case["N"]), max(case["M"], case["N"])
    # X X^T and A^2 are symmetric: half of each is the work
    flops = case["count"] * case["steps"] * (S * S * L + 2 * S * S * L + (S ** 3 if POLYNOMIALS[case["poly"]][2] else 0))
    one = 4 if case["type"] == "fp32" else 2
    return {"bytes": case["count"] * S * L * (one + (2 if case["op"] == "ortho" else 18)), "flops": flops}


# ---- the definitions in 64 bits ----

def _exact_act(z, name):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z * torch.special.ndtr(z) if name == "gelu" else z.clamp(min=0)


def _exact_weights(w, scales):
    """One expert's matrix in 64 bits."""
    if scales is None:
        return w.double()
    blocks = (2.0 ** (scales.double() - 127)).repeat_interleave(128, -2).repeat_interleave(128, -1)
    return w.view(torch.float8_e4m3fn).double() * blocks


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "few":
        T, H = case["T"], case["H"]
        out = torch.zeros((T, H), dtype=torch.float64, device=s["x"].device)
        idx, weights, x = s["topk_idx"].reshape(T, -1).cpu(), s["topk_weights"].reshape(T, -1).double(), s["x"].reshape(T, H).double()
        scales = lambda name, e: None if s[name] is None else s[name][e]  # noqa: E731
        for e in sorted(set(idx.reshape(-1).tolist()) - {-1}):
            t, j = (v.to(x.device) for v in torch.nonzero(idx == e, as_tuple=True))
            gu, down = _exact_weights(s["w_gu"][e], scales("w_gu_scales", e)), _exact_weights(s["w_down"][e], scales("w_down_scales", e))
            h = _exact_act(x[t] @ gu[0].t(), case["act"]) * (x[t] @ gu[1].t())
            out.index_add_(0, t, weights[t, j].unsqueeze(1) * (h @ down.t()))
        return {"out": out.reshape(1, T, H)}
    S, L = min(case["M"], case["N"]), max(case["M"], case["N"])
    if case["count"] * case["steps"] * (4 * S * S * L + 2 * S ** 3) * 1.2e-12 > 20:
        return None
    a, b, c = POLYNOMIALS[case["poly"]]
    u = s["g"].double()
    if case["op"] == "muon":
        m = MU * s["m"].double() + u
        u = u + MU * m if case["nesterov"] else m
    x = torch.empty_like(u)
    for i in range(case["count"]):
        # by the singular values' own side: the smaller Gram matrix P, X_n = X_0 q_n with q_n a polynomial of P
        v = u[i] if case["M"] > case["N"] else u[i].t()
        v = v / (torch.linalg.vector_norm(v) + EPS)
        gram, one = v.t() @ v, torch.eye(v.shape[1], dtype=torch.float64, device=v.device)
        q = one
        for _ in range(case["steps"]):
            square = q @ gram @ q  # X_n^T X_n, all polynomials of P
            q = q @ (a * one + b * square + c * (square @ square))
        x[i] = v @ q if case["M"] > case["N"] else (v @ q).t()
    if case["op"] == "ortho":
        return {"out": x}
    w = (1 - case["lr"] * case["decay"]) * s["w"].double() - case["lr"] * _scale_of(case) * x
    return {"m": m, "w": w, "w16": w}
