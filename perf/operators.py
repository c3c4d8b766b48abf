"""The transformer operators of pipegemm as a user calls them, beside their
plain forms: a linear layer with its epilogue, a gated feed-forward block and
softmax cross entropy over a vocabulary, each forward and with gradients.

``own`` selects the side: False computes the plain form (elementary torch
operations in 32 bits, rounded once at the end), True calls the library.
"""
import math

import torch

own = False

# ---------------------------------------------------------------- the cases ---


def listed():
    return [
        # One decoding token through an attention output projection: bias and
        # the residual stream added in the same call.  Latency counts.
        {"name": "linear token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "act": "none",
         "bias": True, "residual": True, "grad": False, "saved": False},
        # A batch of decoding tokens through the first feed-forward layer.
        {"name": "linear 24 tokens", "op": "linear", "M": 24, "N": 16384, "K": 2048,
         "act": "gelu_tanh", "bias": True, "residual": False, "grad": False, "saved": False},
        # The ragged shape of the GEMM benchmark: no extent a multiple of 8.
        {"name": "linear ragged", "op": "linear", "M": 4095, "N": 4097, "K": 4100, "act": "gelu",
         "bias": True, "residual": True, "grad": False, "saved": False},
        # A long prompt, or the largest forward batch.
        {"name": "linear prompt", "op": "linear", "M": 8192, "N": 8192, "K": 8192, "act": "none",
         "bias": False, "residual": True, "grad": False, "saved": False},
        # A training step of a feed-forward layer, pre-activations kept.
        {"name": "linear train", "op": "linear", "M": 4096, "N": 4096, "K": 2048,
         "act": "gelu_tanh", "bias": True, "residual": False, "grad": True, "saved": True},
        # One decoding token through a gated block's two projections.
        {"name": "gated token", "op": "gated", "M": 1, "F": 8192, "K": 4096, "act": "silu",
         "grad": False, "saved": False},
        # A prompt through the same block, wide.
        {"name": "gated prompt", "op": "gated", "M": 4096, "F": 16384, "K": 4096, "act": "silu",
         "grad": False, "saved": False},
        # A small training step of odd sizes that keeps nothing for its backward pass.
        {"name": "gated train odd", "op": "gated", "M": 777, "F": 1365, "K": 520,
         "act": "gelu_tanh", "grad": True, "saved": False},
        # A large training step, pre-activations kept.
        {"name": "gated train", "op": "gated", "M": 8192, "F": 8192, "K": 4096, "act": "silu",
         "grad": True, "saved": True},
        # Scoring a text with a small model: losses only, an odd vocabulary.
        {"name": "xent score", "op": "xent", "T": 512, "V": 50257, "D": 1024, "grad": False},
        # A fine-tuning step: ragged token count and vocabulary.
        {"name": "xent train ragged", "op": "xent", "T": 1001, "V": 32003, "D": 2048,
         "grad": True},
        # A pre-training step with a large vocabulary.
        {"name": "xent train", "op": "xent", "T": 4096, "V": 131072, "D": 4096, "grad": True},
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]; two in three are multiples of 8 where that fits."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 16 and rng.random() < 0.67:
        v = v // 8 * 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["linear", "gated", "xent"])
    grad = rng.random() < 0.5
    if op == "xent":
        return {"op": op, "T": _size(rng, 1, 4096), "V": _size(rng, 1000, 131072),
                "D": _size(rng, 128, 4096), "grad": grad}
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"] if op == "linear"
                     else ["relu", "gelu", "gelu_tanh", "silu"])
    case = {"op": op, "M": _size(rng, 1, 8192), "K": _size(rng, 128, 8192 if op == "linear" else 4096),
            "act": act, "grad": grad, "saved": grad and rng.random() < 0.5}
    if op == "linear":
        case.update({"N": _size(rng, 128, 8192), "bias": rng.random() < 0.6,
                     "residual": not grad and rng.random() < 0.5})
    else:
        case["F"] = _size(rng, 128, 8192)
    return case


def work(case):
    """Bytes: every input read once, every output written once (what `saved`
    keeps between the two directions is neither).  Operations: the matrix
    products without any recomputation."""
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        b = 2 * (M * K + K * N + M * N) + 2 * N * case["bias"] + 2 * M * N * case["residual"]
        f = 2 * M * N * K
        if case["grad"]:
            b += 2 * (M * N + M * K + K * N) + 2 * N * case["bias"]
            f *= 3
    elif case["op"] == "gated":
        M, F, K = case["M"], case["F"], case["K"]
        b, f = 2 * (M * K + 2 * K * F + M * F), 4 * M * K * F
        if case["grad"]:
            b += 2 * (M * F + M * K + 2 * K * F)
            f *= 3
    else:
        T, V, D = case["T"], case["V"], case["D"]
        b, f = 2 * (T * D + V * D) + 8 * T + 8 * T, 2 * T * V * D
        if case["grad"]:
            b += 2 * (T * D + V * D) + 4 * T
            f *= 3
    return {"bytes": b, "flops": f}


# --------------------------------------------------------------- the inputs ---


def _normal(g, shape, std):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def prepare(case, seed):
    """Activations of unit scale (as after a norm), weights of 1/sqrt(fan-in),
    gradients as they come back scaled by a mean over tokens; token ids with
    the skew of a text, a few of them padding (-100)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["X"] = _normal(g, (M, K), 1.0)
        s["W"] = _normal(g, (K, N), K ** -0.5)
        s["b"] = _normal(g, (N,), 0.1) if case["bias"] else None
        s["R"] = _normal(g, (M, N), 1.0) if case["residual"] else None
        s["dY"] = _normal(g, (M, N), 1.0 / M) if case["grad"] else None
    elif case["op"] == "gated":
        M, F, K = case["M"], case["F"], case["K"]
        s["X"] = _normal(g, (M, K), 1.0)
        s["Wg"] = _normal(g, (K, F), K ** -0.5)
        s["Wu"] = _normal(g, (K, F), K ** -0.5)
        s["dH"] = _normal(g, (M, F), 1.0 / M) if case["grad"] else None
    else:
        T, V, D = case["T"], case["V"], case["D"]
        s["X"] = _normal(g, (T, D), 1.0)
        s["W"] = _normal(g, (V, D), 2.0 * D ** -0.5)  # logits of standard deviation 2
        u = torch.rand((T,), generator=g, device="cuda", dtype=torch.float64)
        y = (torch.pow(float(V), u) - 1.0).to(torch.int64).clamp_(0, V - 1)
        pad = torch.rand((T,), generator=g, device="cuda") < 0.06
        s["y"] = torch.where(pad, torch.full_like(y, -100), y)
        # the gradient of a mean over the tokens that count
        s["dl"] = torch.full((T,), 1.0 / T, device="cuda") if case["grad"] else None
    return s


# ----------------------------------------------------------- the plain forms ---


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _dact(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)


def _plain_linear(s):
    bf = torch.bfloat16
    X, W = s["X"].float(), s["W"].float()
    z = X @ W
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["R"] is not None:
        y = y + s["R"].float()
    out = {"Y": y.to(bf)}
    if s["grad"]:
        dz = s["dY"].float() * _dact(z, s["act"])
        out["dX"] = (dz @ W.t()).to(bf)
        out["dW"] = (X.t() @ dz).to(bf)
        if s["b"] is not None:
            out["db"] = dz.sum(0).to(bf)
    return out


def _plain_gated(s):
    bf = torch.bfloat16
    X, Wg, Wu = s["X"].float(), s["Wg"].float(), s["Wu"].float()
    g, u = X @ Wg, X @ Wu
    a = _act(g, s["act"])
    out = {"H": (a * u).to(bf)}
    if s["grad"]:
        dh = s["dH"].float()
        dg, du = dh * u * _dact(g, s["act"]), dh * a
        out["dX"] = (dg @ Wg.t() + du @ Wu.t()).to(bf)
        out["dWg"] = (X.t() @ dg).to(bf)
        out["dWu"] = (X.t() @ du).to(bf)
    return out


def _plain_xent(s):
    bf = torch.bfloat16
    X, W, y = s["X"].float(), s["W"].float(), s["y"]
    logits = X @ W.t()
    m = logits.amax(1, keepdim=True)
    e = torch.exp(logits - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    valid = y >= 0
    at = y.clamp(min=0).unsqueeze(1)
    out = {"loss": torch.where(valid, (lse - logits.gather(1, at)).squeeze(1), 0.0),
           "lse": lse.squeeze(1)}
    if s["grad"]:
        p = e / total
        p.scatter_add_(1, at, torch.full_like(total, -1.0))
        p *= torch.where(valid, s["dl"], 0.0).unsqueeze(1)
        out["dX"] = (p @ W).to(bf)
        out["dW"] = (p.t() @ X).to(bf)
    return out


# ------------------------------------------------------- the library's calls ---


def _own_linear(s):
    import software_pipelined_tiled_loop_gb300 as pg
    M, N, K, X, W, b, act = s["M"], s["N"], s["K"], s["X"], s["W"], s["b"], s["act"]
    Y = X.new_empty((M, N))
    Z = torch.empty((M, N), dtype=torch.float32, device=X.device) if s["saved"] else None
    pg.linear_bf16(M, N, K, X, W, b, act, s["R"], Y, preact=Z)
    out = {"Y": Y}
    if s["grad"]:
        dX, dW = torch.empty_like(X), torch.empty_like(W)
        db = torch.empty_like(b) if b is not None else None
        pg.linear_bf16_backward(M, N, K, X, W, b, act, s["dY"], dX, dW, db, preact=Z)
        out.update({"dX": dX, "dW": dW})
        if db is not None:
            out["db"] = db
    return out


def _own_gated(s):
    import software_pipelined_tiled_loop_gb300 as pg
    M, F, K, X, Wg, Wu, act = s["M"], s["F"], s["K"], s["X"], s["Wg"], s["Wu"], s["act"]
    H = X.new_empty((M, F))
    Z = torch.empty((2, M, F), dtype=torch.float32, device=X.device) if s["saved"] else None
    pg.gated_bf16(M, F, K, X, Wg, Wu, act, H, preact=Z)
    out = {"H": H}
    if s["grad"]:
        dX, dWg, dWu = torch.empty_like(X), torch.empty_like(Wg), torch.empty_like(Wu)
        pg.gated_bf16_backward(M, F, K, X, Wg, Wu, act, s["dH"], dX, dWg, dWu, preact=Z)
        out.update({"dX": dX, "dWg": dWg, "dWu": dWu})
    return out


def _own_xent(s):
    import software_pipelined_tiled_loop_gb300 as pg
    T, V, D, X, W, y = s["T"], s["V"], s["D"], s["X"], s["W"], s["y"]
    loss = torch.empty((T,), dtype=torch.float32, device=X.device)
    lse = torch.empty_like(loss)
    out = {"loss": loss, "lse": lse}
    if s["grad"]:
        dX, dW = torch.empty_like(X), torch.empty_like(W)
        pg.xent_bf16_grad(T, V, D, X, W, y, s["dl"], loss, lse, dX, dW)
        out.update({"dX": dX, "dW": dW})
    else:
        pg.xent_bf16(T, V, D, X, W, y, loss, lse)
    return out


def run(state):
    if own:
        return {"linear": _own_linear, "gated": _own_gated, "xent": _own_xent}[state["op"]](state)
    return {"linear": _plain_linear, "gated": _plain_gated, "xent": _plain_xent}[state["op"]](state)


# ------------------------------------------------- the definition in 64 bits ---


def exact(case, seed):
    """From torch's own double-precision functions and their automatic
    gradients.  None where the products would take over about 20 seconds."""
    if work(case)["flops"] > 2e13:
        return None
    s = prepare(case, seed)
    f = torch.nn.functional
    acts = {"none": lambda z: z, "relu": f.relu, "silu": f.silu, "gelu": f.gelu,
            "gelu_tanh": lambda z: f.gelu(z, approximate="tanh")}

    def leaf(t):
        return None if t is None else t.double().requires_grad_(case["grad"])

    def grads(of, with_, **named):
        if not case["grad"]:
            return {}
        got = torch.autograd.grad(of, list(named.values()), with_)
        return dict(zip(named, got))

    X = leaf(s["X"])
    if case["op"] == "linear":
        W, b = leaf(s["W"]), leaf(s["b"])
        y = torch.addmm(b, X, W) if b is not None else torch.mm(X, W)
        y = acts[case["act"]](y)
        out = {"Y": (y if s["R"] is None else y + s["R"].double()).detach()}
        named = {"dX": X, "dW": W}
        if b is not None:
            named["db"] = b
        out.update(grads(y, s["dY"].double() if case["grad"] else None, **named))
        return out
    if case["op"] == "gated":
        Wg, Wu = leaf(s["Wg"]), leaf(s["Wu"])
        h = acts[case["act"]](torch.mm(X, Wg)) * torch.mm(X, Wu)
        out = {"H": h.detach()}
        out.update(grads(h, s["dH"].double() if case["grad"] else None, dX=X, dWg=Wg, dWu=Wu))
        return out
    W = leaf(s["W"])
    logits = f.linear(X, W)
    loss = f.cross_entropy(logits, s["y"], ignore_index=-100, reduction="none")
    out = {"loss": loss.detach(), "lse": torch.logsumexp(logits, 1).detach()}
    out.update(grads(loss, s["dl"].double() if case["grad"] else None, dX=X, dW=W))
    return out
