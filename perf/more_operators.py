"""The operators of a mixture-of-experts block as a user calls them, beside their
plain forms: the root-mean-square norm in front of it with the residual's addition
(bf16, or int8 with a scale a row), the routing of tokens to experts, tokens sorted
by expert and back, and the experts' products, each forward and with gradients.

``own`` selects the side: False computes the plain form (elementary torch
operations in 32 bits, rounded once at the end), True calls the library.
"""
import math

import torch

own = False

EPS = 1e-6

# ---------------------------------------------------------------- the cases ---


def listed():
    return [
        # One decoding token: the sublayer's output joins the residual stream, which
        # is normalised for the next one.  Latency counts.
        {"name": "norm token", "op": "norm", "T": 1, "D": 4096, "residual": True, "out": "bf16",
         "grad": False},
        # A prompt in front of an int8 product: odd count of tokens.
        {"name": "norm int8 prompt", "op": "norm", "T": 4097, "D": 5120, "residual": True,
         "out": "i8", "grad": False},
        # A training step's norm, both directions.
        {"name": "norm train", "op": "norm", "T": 8192, "D": 4096, "residual": True,
         "out": "bf16", "grad": True},
        # A batch of decoding tokens chooses its experts.
        {"name": "route tokens", "op": "route", "T": 24, "E": 64, "k": 8, "normalise": True,
         "masked": False, "grad": False},
        # A training step's routing, weights from the softmax over all experts, some of
        # which are closed to a token (-inf).
        {"name": "route train", "op": "route", "T": 16384, "E": 128, "k": 8, "normalise": False,
         "masked": True, "grad": True},
        # A batch of decoding tokens sorted by expert and back.
        {"name": "dispatch tokens", "op": "dispatch", "T": 24, "E": 64, "k": 8, "D": 2048,
         "grad": False},
        # A training step's, both directions.
        {"name": "dispatch train", "op": "dispatch", "T": 8192, "E": 64, "k": 4, "D": 4096,
         "grad": True},
        # The experts' output projection for a batch of decoding tokens.
        {"name": "experts linear tokens", "op": "linear", "T": 24, "E": 64, "k": 8, "N": 2048,
         "K": 1024, "grad": False},
        # A training step of it: ragged groups of a few hundred rows.
        {"name": "experts linear train", "op": "linear", "T": 4096, "E": 32, "k": 4, "N": 4096,
         "K": 2048, "grad": True},
        # One decoding token through the two projections of its eight experts.
        {"name": "experts gated token", "op": "gated", "T": 1, "E": 64, "k": 8, "F": 1024,
         "K": 2048, "act": "silu", "grad": False, "saved": False},
        # A prompt through few wide experts.
        {"name": "experts gated prompt", "op": "gated", "T": 4096, "E": 8, "k": 2, "F": 8192,
         "K": 4096, "act": "silu", "grad": False, "saved": False},
        # A training step of many narrow experts, pre-activations kept.
        {"name": "experts gated train", "op": "gated", "T": 4096, "E": 64, "k": 8, "F": 1024,
         "K": 2048, "act": "silu", "grad": True, "saved": True},
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]; two in three are multiples of 8 where that fits."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 16 and rng.random() < 0.67:
        v = v // 8 * 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "route", "dispatch", "linear", "gated", "linear", "gated"])
    grad = rng.random() < 0.5
    if op == "norm":
        out = "bf16" if grad or rng.random() < 0.6 else "i8"
        return {"op": op, "T": _size(rng, 1, 8192), "D": _size(rng, 64, 8192),
                "residual": rng.random() < 0.7, "out": out, "grad": grad}
    if op == "route":
        E = _size(rng, 4, 256)
        return {"op": op, "T": _size(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E)),
                "normalise": rng.random() < 0.5, "masked": rng.random() < 0.3, "grad": grad}
    if op == "dispatch":
        E = _size(rng, 4, 256)
        return {"op": op, "T": _size(rng, 1, 8192), "E": E, "k": rng.randint(1, min(4, E)),
                "D": _size(rng, 64, 4096), "grad": grad}
    while True:  # as much work and memory as the largest listed case at most
        T, E = _size(rng, 1, 4096), _size(rng, 4, 128)
        k = rng.randint(1, min(8, E))
        N, K = _size(rng, 128, 4096), _size(rng, 128, 4096)
        m = 2 if op == "gated" else 1
        if m * E * N * K <= 1 << 28 and m * T * k * N * K <= 1 << 37:
            break
    case = {"op": op, "T": T, "E": E, "k": k, "K": K, "grad": grad}
    if op == "linear":
        case["N"] = N
    else:
        case.update({"F": N, "act": rng.choice(["gelu", "gelu_tanh", "silu"]),
                     "saved": grad and rng.random() < 0.5})
    return case


def work(case):
    """Bytes: every input read once, every output written once (what the forward
    direction hands to the backward one is neither read nor written again).  The
    experts' weights: of as many experts as there can be with rows.  Operations: the
    matrix products without any recomputation; elsewhere the few an element takes."""
    T, grad, op = case["T"], case["grad"], case["op"]
    if op == "norm":
        n = T * case["D"]
        b = 2 * n * (2 if case["residual"] else 1) + 2 * case["D"]  # X, R, gain
        b += 2 * n + (2 * n if case["out"] == "bf16" else n + 4 * T)  # S; Y or Q and scales
        if grad:
            b += 3 * 2 * n + 2 * case["D"]  # dY and dS; dX and dgain
        return {"bytes": b, "flops": n * (14 if grad else 5)}
    k, E = case["k"], case["E"]
    if op == "route":
        b = 4 * T * E + 8 * T * k + ((4 * T * k + 4 * T * E) if grad else 0)
        return {"bytes": b, "flops": T * E * (k + 4)}
    R = T * k
    if op == "dispatch":
        D = case["D"]
        b = 4 * R + 4 * (E + 1) + 4 * R  # experts; offsets and rows
        b += 2 * T * D + 2 * R * D  # X; Xs
        b += 2 * R * D + 4 * R + 2 * T * D + 2 * T * D  # Ys, weights, residual; Y
        if grad:
            b += 2 * T * D + 2 * R * D + 4 * R  # dY; dYs, dweights
            b += 2 * R * D + 2 * T * D  # dXs; dX
        return {"bytes": b, "flops": 2 * R * D * (4 if grad else 1)}
    N, K, live = case["N"] if op == "linear" else case["F"], case["K"], min(E, R)
    m = 1 if op == "linear" else 2
    b = 2 * (R * K + R * N) + 2 * m * live * K * N + 4 * (E + 1)
    f = 2 * m * R * K * N
    if grad:
        b += 2 * (R * N + R * K) + 2 * m * E * K * N
        f *= 3
    return {"bytes": b, "flops": f}


# --------------------------------------------------------------- the inputs ---


def _normal(g, shape, std):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _choose(g, T, E, k):
    """k different experts for each of T tokens, some experts more popular than
    others (up to some three times the mean), as a router's are: T x k int32."""
    pop = 0.5 * torch.randn((1, E), generator=g, device="cuda")
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-6, 1.0 - 1e-6)
    return (pop - torch.log(-torch.log(u))).topk(k, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    """Activations of unit scale, weights of 1/sqrt(fan-in), gradients as they come
    back scaled by a mean over tokens."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    T = case["T"]
    if case["op"] == "norm":
        D = case["D"]
        s["X"] = _normal(g, (T, D), 0.5)
        # a residual stream whose tokens differ in scale
        scale = torch.exp(0.7 * torch.randn((T, 1), generator=g, device="cuda"))
        s["R"] = (torch.randn((T, D), generator=g, device="cuda") * scale).to(torch.bfloat16) \
            if case["residual"] else None
        s["gain"] = (1.0 + 0.1 * torch.randn((D,), generator=g, device="cuda")).to(torch.bfloat16)
        s["dY"] = _normal(g, (T, D), 1.0 / T) if case["grad"] else None
        s["dS"] = _normal(g, (T, D), 1.0 / T) if case["grad"] else None
        return s
    E, k = case["E"], case["k"]
    if case["op"] == "route":
        z = 1.5 * torch.randn((T, E), generator=g, device="cuda")
        if case["masked"]:  # one expert in eight closed to a token, all of them to a padded one
            z[torch.rand((T, E), generator=g, device="cuda") < 0.125] = -math.inf
            z[torch.rand((T,), generator=g, device="cuda") < 0.03] = -math.inf
        s["logits"] = z
        s["dweights"] = torch.randn((T, k), generator=g, device="cuda") / T if case["grad"] else None
        return s
    experts = _choose(g, T, E, k)
    R = T * k
    if case["op"] == "dispatch":
        D = case["D"]
        s["experts"] = experts
        s["X"] = _normal(g, (T, D), 1.0)
        s["Ys"] = _normal(g, (R, D), 1.0)  # what the experts made of the sorted rows
        s["residual"] = _normal(g, (T, D), 1.0)
        s["weights"] = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1)
        s["dY"] = _normal(g, (T, D), 1.0 / T) if case["grad"] else None
        s["dXs"] = _normal(g, (R, D), 1.0 / T) if case["grad"] else None
        return s
    counts = torch.bincount(experts.reshape(-1), minlength=E)
    offsets = torch.zeros((E + 1,), dtype=torch.int64, device="cuda")
    offsets[1:] = counts.cumsum(0)
    s["R"] = R
    s["offsets"] = offsets.to(torch.int32)
    # for the plain form: each row's expert and place in its group, the largest group
    s["row_expert"] = torch.repeat_interleave(torch.arange(E, device="cuda"), counts)
    s["row_place"] = torch.arange(R, device="cuda") - offsets[:-1][s["row_expert"]]
    s["largest"] = int(counts.max())
    K = case["K"]
    s["X"] = _normal(g, (R, K), 1.0)
    if case["op"] == "linear":
        s["W"] = _normal(g, (E, K, case["N"]), K ** -0.5)
        s["dY"] = _normal(g, (R, case["N"]), 1.0 / T) if case["grad"] else None
    else:
        s["Wg"] = _normal(g, (E, K, case["F"]), K ** -0.5)
        s["Wu"] = _normal(g, (E, K, case["F"]), K ** -0.5)
        s["dH"] = _normal(g, (R, case["F"]), 1.0 / T) if case["grad"] else None
    return s


# ----------------------------------------------------------- the plain forms ---


def _plain_norm(s):
    bf = torch.bfloat16
    stream = s["X"] if s["R"] is None else (s["X"].float() + s["R"].float()).to(bf)
    x, gain = stream.float(), s["gain"].float()
    rstd = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    n = x * rstd
    y = n * gain
    out = {"S": stream}
    if s["out"] == "i8":
        scale = y.abs().amax(1, keepdim=True) / 127.0
        q = torch.round(y / scale)
        out["scale"] = scale.squeeze(1)
        out["Y"] = (q * scale).to(bf)
    else:
        out["Y"] = y.to(bf)
    if s["grad"]:
        dy = s["dY"].float()
        a = dy * gain
        dx = rstd * (a - n * (a * n).mean(1, keepdim=True)) + s["dS"].float()
        out["dX"] = dx.to(bf)
        out["dgain"] = (dy.double() * n.double()).sum(0).to(bf)
    return out


def _plain_route(s):
    z, k = s["logits"], s["k"]
    top, index = torch.sort(z, dim=1, descending=True, stable=True)
    top, index = top[:, :k], index[:, :k]
    there = top > -math.inf
    most = torch.where(there[:, :1], top[:, :1], 0.0)
    e = torch.exp(top - most)
    over = e if s["normalise"] else torch.exp(z - most)
    total = over.sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0)
    w = e / total
    out = {"experts": torch.where(there, index, -1).to(torch.int32), "weights": w}
    if s["grad"]:
        dw = torch.where(there, s["dweights"], 0.0)
        dot = (w * dw).sum(1, keepdim=True)
        dz = torch.zeros_like(z) if s["normalise"] else -over / total * dot
        chosen = w * (dw - dot) if s["normalise"] else w * dw
        out["dlogits"] = dz.scatter_add(1, index, chosen)
    return out


def _plain_dispatch(s):
    bf, T, k, E = torch.bfloat16, s["T"], s["k"], s["E"]
    flat = s["experts"].reshape(-1)
    order = torch.argsort(flat, stable=True)
    rows = torch.empty_like(order)
    rows[order] = torch.arange(T * k, device=order.device)
    ends = (flat.unsqueeze(0) < torch.arange(E + 1, device=flat.device).unsqueeze(1)).sum(1)
    rows = rows.reshape(T, k)
    w = s["weights"]
    y = (s["Ys"][rows].float() * w.unsqueeze(2)).sum(1) + s["residual"].float()
    out = {"offsets": ends.to(torch.int32), "rows": rows.to(torch.int32),
           "Xs": s["X"][order // k], "Y": y.to(bf)}
    if s["grad"]:
        dy = s["dY"].float().unsqueeze(1)
        dys = torch.empty(s["Ys"].shape, dtype=torch.float32, device=flat.device)
        dys[rows.reshape(-1)] = (w.unsqueeze(2) * dy).reshape(T * k, -1)
        out["dYs"] = dys.to(bf)
        out["dweights"] = (s["Ys"][rows].double() * dy.double()).sum(2).float()
        out["dX"] = s["dXs"][rows].float().sum(1).to(bf)
    return out


def _pad(s, x):
    """Rows of R x n laid out as E x (largest group) x n, zeros behind each group."""
    p = torch.zeros((s["E"], s["largest"], x.shape[1]), dtype=x.dtype, device=x.device)
    p[s["row_expert"], s["row_place"]] = x
    return p


def _each(s, x, w):
    """Row r of x times the matrix of its expert."""
    if s["R"] < s["E"]:  # few rows: their own experts' matrices only
        return torch.bmm(x.unsqueeze(1), w[s["row_expert"]].float()).squeeze(1)
    return torch.bmm(_pad(s, x), w.float())[s["row_expert"], s["row_place"]]


def _outer(s, x, y):
    """For each expert, x^T y over its rows."""
    return torch.bmm(_pad(s, x).transpose(1, 2), _pad(s, y))


def _plain_linear(s):
    bf = torch.bfloat16
    x = s["X"].float()
    out = {"Y": _each(s, x, s["W"]).to(bf)}
    if s["grad"]:
        dy = s["dY"].float()
        out["dX"] = _each(s, dy, s["W"].transpose(1, 2)).to(bf)
        out["dW"] = _outer(s, x, dy).to(bf)
    return out


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _dact(z, act):
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)


def _plain_gated(s):
    bf = torch.bfloat16
    x = s["X"].float()
    g, u = _each(s, x, s["Wg"]), _each(s, x, s["Wu"])
    a = _act(g, s["act"])
    out = {"H": (a * u).to(bf)}
    if s["grad"]:
        dh = s["dH"].float()
        dg, du = dh * u * _dact(g, s["act"]), dh * a
        out["dX"] = (_each(s, dg, s["Wg"].transpose(1, 2))
                     + _each(s, du, s["Wu"].transpose(1, 2))).to(bf)
        out["dWg"] = _outer(s, x, dg).to(bf)
        out["dWu"] = _outer(s, x, du).to(bf)
    return out


# ------------------------------------------------------- the library's calls ---


def _own_norm(s):
    import software_pipelined_tiled_loop_gb300 as pg
    T, D, X, R, gain = s["T"], s["D"], s["X"], s["R"], s["gain"]
    S = torch.empty_like(X) if R is not None else X
    keep = S if R is not None else None
    out = {"S": S}
    if s["out"] == "i8":
        Q = torch.empty((T, D), dtype=torch.int8, device=X.device)
        scale = torch.empty((T,), dtype=torch.float32, device=X.device)
        pg.rmsnorm_i8(T, D, X, R, gain, EPS, keep, Q, scale)
        out["scale"] = scale
        out["Y"] = torch.mul(Q, scale.unsqueeze(1), out=torch.empty_like(X))
        return out
    Y = torch.empty_like(X)
    pg.rmsnorm_bf16(T, D, X, R, gain, EPS, keep, Y)
    out["Y"] = Y
    if s["grad"]:
        dX, dgain = torch.empty_like(X), torch.empty_like(gain)
        pg.rmsnorm_bf16_backward(T, D, S, gain, EPS, s["dY"], s["dS"], dX, dgain)
        out.update({"dX": dX, "dgain": dgain})
    return out


def _own_route(s):
    import software_pipelined_tiled_loop_gb300 as pg
    T, E, k, z = s["T"], s["E"], s["k"], s["logits"]
    experts = torch.empty((T, k), dtype=torch.int32, device=z.device)
    weights = torch.empty((T, k), dtype=torch.float32, device=z.device)
    pg.route_topk(T, E, k, z, s["normalise"], experts, weights)
    out = {"experts": experts, "weights": weights}
    if s["grad"]:
        dz = torch.empty_like(z)
        pg.route_topk_backward(T, E, k, z, s["normalise"], experts, s["dweights"], dz)
        out["dlogits"] = dz
    return out


def _own_dispatch(s):
    import software_pipelined_tiled_loop_gb300 as pg
    T, E, k, D, X, Ys, w = s["T"], s["E"], s["k"], s["D"], s["X"], s["Ys"], s["weights"]
    offsets = torch.empty((E + 1,), dtype=torch.int32, device=X.device)
    rows = torch.empty((T, k), dtype=torch.int32, device=X.device)
    Xs, Y = torch.empty_like(Ys), torch.empty_like(X)
    pg.expert_sort(T, E, k, s["experts"], offsets, rows)
    pg.expert_gather_bf16(T, k, D, X, rows, Xs)
    pg.expert_combine_bf16(T, k, D, Ys, rows, w, s["residual"], Y)
    out = {"offsets": offsets, "rows": rows, "Xs": Xs, "Y": Y}
    if s["grad"]:
        dYs, dw, dX = torch.empty_like(Ys), torch.empty_like(w), torch.empty_like(X)
        pg.expert_combine_bf16_backward(T, k, D, Ys, rows, w, s["dY"], dYs, dw)
        pg.expert_combine_bf16(T, k, D, s["dXs"], rows, None, None, dX)  # the gather's gradient
        out.update({"dYs": dYs, "dweights": dw, "dX": dX})
    return out


def _own_linear(s):
    import software_pipelined_tiled_loop_gb300 as pg
    R, N, K, E, X, W, offsets = s["R"], s["N"], s["K"], s["E"], s["X"], s["W"], s["offsets"]
    Y = X.new_empty((R, N))
    pg.experts_linear_bf16(R, N, K, E, offsets, X, W, Y)
    out = {"Y": Y}
    if s["grad"]:
        dX, dW = torch.empty_like(X), torch.empty_like(W)
        pg.experts_linear_bf16_backward(R, N, K, E, offsets, X, W, s["dY"], dX, dW)
        out.update({"dX": dX, "dW": dW})
    return out


def _own_gated(s):
    import software_pipelined_tiled_loop_gb300 as pg
    R, F, K, E, X, act = s["R"], s["F"], s["K"], s["E"], s["X"], s["act"]
    Wg, Wu, offsets = s["Wg"], s["Wu"], s["offsets"]
    H = X.new_empty((R, F))
    Z = torch.empty((2, R, F), dtype=torch.float32, device=X.device) if s["saved"] else None
    pg.experts_gated_bf16(R, F, K, E, offsets, X, Wg, Wu, act, H, preact=Z)
    out = {"H": H}
    if s["grad"]:
        dX, dWg, dWu = torch.empty_like(X), torch.empty_like(Wg), torch.empty_like(Wu)
        pg.experts_gated_bf16_backward(R, F, K, E, offsets, X, Wg, Wu, act, s["dH"], dX, dWg, dWu,
                                       preact=Z)
        out.update({"dX": dX, "dWg": dWg, "dWu": dWu})
    return out


def run(state):
    if own:
        return {"norm": _own_norm, "route": _own_route, "dispatch": _own_dispatch,
                "linear": _own_linear, "gated": _own_gated}[state["op"]](state)
    return {"norm": _plain_norm, "route": _plain_route, "dispatch": _plain_dispatch,
            "linear": _plain_linear, "gated": _plain_gated}[state["op"]](state)


# ------------------------------------------------- the definition in 64 bits ---


def exact(case, seed):
    """From torch's own double-precision functions and their automatic gradients,
    group by group."""
    s = prepare(case, seed)
    f = torch.nn.functional
    grad = case["grad"]

    def leaf(t):
        return t.double().requires_grad_(grad)

    if case["op"] == "norm":
        total = s["X"].double() if s["R"] is None else s["X"].double() + s["R"].double()
        # the residual stream is a bf16 tensor, and it is what is normalised
        x = total.to(torch.bfloat16).double().requires_grad_(grad)
        gain = leaf(s["gain"])
        y = f.rms_norm(x, (case["D"],), gain, EPS)
        out = {"S": x.detach()}
        if case["out"] == "i8":
            step = y.norm(math.inf, dim=1, keepdim=True) / 127
            out.update({"scale": step.squeeze(1), "Y": torch.round(y / step) * step})
        else:
            out["Y"] = y.detach()
        if grad:
            dx, dgain = torch.autograd.grad(y, (x, gain), s["dY"].double())
            out.update({"dX": dx + s["dS"].double(), "dgain": dgain})
        return out
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        z = leaf(s["logits"])
        open_ = torch.isfinite(z)
        # rows without an open expert choose none; others softmax over what is open
        some = open_.any(1, keepdim=True)
        p = torch.softmax(torch.where(some, z, 0.0), 1) * some
        left, picks = z.detach().clone(), []
        for _ in range(k):
            # the lowest of the largest ones left
            place = torch.arange(E, device=z.device).expand(T, E)
            at = torch.where(left == left.amax(1, keepdim=True), place, E).amin(1, keepdim=True)
            ok = left.gather(1, at) > -math.inf
            picks.append(torch.where(ok, at, -1))
            left.scatter_(1, at, -math.inf)
        index = torch.cat(picks, 1)
        got = p.gather(1, index.clamp(min=0)) * (index >= 0)
        if case["normalise"]:
            whole = got.sum(1, keepdim=True)
            got = got / torch.where(whole > 0, whole, 1.0)
        out = {"experts": index.to(torch.int32), "weights": got.detach()}
        if grad:
            out["dlogits"] = torch.autograd.grad(got, z, s["dweights"].double())[0]
        return out
    if case["op"] == "dispatch":
        flat = s["experts"].reshape(-1).long()
        key = flat * (T * k) + torch.arange(T * k, device=flat.device)  # expert, then slot
        sorted_key, order = torch.sort(key)
        rows = torch.searchsorted(sorted_key, key)
        counts = torch.bincount(flat, minlength=E)
        offsets = f.pad(counts.cumsum(0), (1, 0))
        Ys, w = leaf(s["Ys"]), leaf(s["weights"])
        y = torch.einsum("tk,tkd->td", w, Ys[rows.reshape(T, k)])
        out = {"offsets": offsets.to(torch.int32), "rows": rows.reshape(T, k).to(torch.int32),
               "Xs": s["X"].double()[order // k], "Y": (y + s["residual"].double()).detach()}
        if grad:
            dys, dw = torch.autograd.grad(y, (Ys, w), s["dY"].double())
            dx = torch.zeros_like(s["X"], dtype=torch.float64)
            dx.index_add_(0, order // k, s["dXs"].double())
            out.update({"dYs": dys, "dweights": dw, "dX": dx})
        return out
    acts = {"silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda z: f.gelu(z, approximate="tanh")}
    names = ["W"] if case["op"] == "linear" else ["Wg", "Wu"]
    ends = s["offsets"].tolist()
    outs, dxs, dws = [], [], [[] for _ in names]
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        x, ws = leaf(s["X"][a:b]), [leaf(s[n][e]) for n in names]
        if case["op"] == "linear":
            y, up = torch.mm(x, ws[0]), s["dY"]
        else:
            y, up = acts[case["act"]](torch.mm(x, ws[0])) * torch.mm(x, ws[1]), s["dH"]
        outs.append(y.detach())
        if grad:
            d = torch.autograd.grad(y, [x, *ws], up[a:b].double())
            dxs.append(d[0])
            for held, v in zip(dws, d[1:]):
                held.append(v.float())
    out = {"Y" if case["op"] == "linear" else "H": torch.cat(outs)}
    if grad:
        out["dX"] = torch.cat(dxs)
        out.update({"d" + n: torch.stack(v) for n, v in zip(names, dws)})
    return out
