"""The operators' definitions in 64 bits, with the error a right kernel may
have, element by element.

Every bound is built from what the kernels are documented to do, before any of
them ran:
  * products accumulate in fp32: at most one rounding (by truncation) of every
    16-product step, so |error| <= STEP(K) * sum |a b|, STEP(K) =
    (K / 16 + 4) * 2^-23, of which two are for a bias or residual added after;
  * activations: their slopes are at most 1.13 (gelu, silu), and the fast
    exponential and divide are good to 2^-18 of the value (the argument of the
    exponential carries 2^-24 of its size, at most about 2^6);
  * an operand rounded to bf16 (8 significant bits) is off by 2^-8 of itself at
    most, an output likewise
    (2^-133 absolutely, below the normal range).
A gradient operand's error goes through the next product as sum |error b|.
"""
from __future__ import annotations

import math

import torch

SLOPE, FAST, HALF = 1.13, 2.0 ** -18, 2.0 ** -8
TINY = 2.0 ** -133


def step(K: int) -> float:
    return (K / 16 + 4) * 2.0 ** -23


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z)


def act_grad(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return (0.5 * torch.erfc(-z / math.sqrt(2))
                + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def _bf16_out(y, err):
    """Bound of a bf16 output of value y computed to within err."""
    return err + HALF * (y.abs() + err) + TINY


def linear(X, W, b, name, R):
    """(Y, bound, Z, bound of Z)."""
    X, W = X.double(), W.double()
    z = X @ W
    size = X.abs() @ W.abs()
    if b is not None:
        z = z + b.double()
        size = size + b.double().abs()
    ez = step(X.shape[1]) * size
    y = act(z, name)
    ey = ez * (SLOPE if name != "none" else 1) + (FAST * (y.abs() + z.abs()) if name != "none" else 0)
    if R is not None:
        y = y + R.double()
        ey = ey + 2.0 ** -23 * y.abs()
    return y, _bf16_out(y, ey), z, ez


def _products(X, Ws, dzs, edzs):
    """dX = sum dz W^T and dW = X^T dz with their bounds, for dz off by edz."""
    M, N = dzs[0].shape
    dX = sum(d @ w.t() for d, w in zip(dzs, Ws))
    eX = sum(e @ w.abs().t() + step(len(Ws) * N) * (d.abs() @ w.abs().t())
             for d, e, w in zip(dzs, edzs, Ws))
    out = {"dX": (dX, _bf16_out(dX, eX))}
    for i, (d, e) in enumerate(zip(dzs, edzs)):
        dW = X.t() @ d
        eW = X.abs().t() @ e + step(M) * (X.abs().t() @ d.abs())
        out[f"dW{i}"] = (dW, _bf16_out(dW, eW))
    return out


def linear_backward(X, W, b, name, dY):
    _, _, z, ez = linear(X, W, b, "none", None)
    X, W, dY = X.double(), W.double(), dY.double()
    dz = dY * act_grad(z, name)
    # curvature of the activations is at most 1.2; relu: exact but for the
    # sign of a Z within its own error of zero
    edz = dY.abs() * (1.2 * ez + FAST * (1 + z.abs())) if name != "none" else torch.zeros_like(dz)
    if name == "relu":
        edz = dY.abs() * (z.abs() <= ez)
    rounded = edz + HALF * (dz.abs() + edz) + TINY
    if name == "none":
        rounded = edz  # dY itself is the operand
    out = _products(X, [W], [dz], [rounded])
    db = dz.sum(0)
    edb = rounded.sum(0) + dz.shape[0] * 2.0 ** -23 * dz.abs().sum(0)
    out["db"] = (db, _bf16_out(db, edb))
    return out


def gated(X, Wg, Wu, name):
    """(H, bound, G, U, bounds)."""
    X, Wg, Wu = X.double(), Wg.double(), Wu.double()
    g, u = X @ Wg, X @ Wu
    eg, eu = (step(X.shape[1]) * (X.abs() @ w.abs()) for w in (Wg, Wu))
    a = act(g, name)
    ea = SLOPE * eg + FAST * (a.abs() + g.abs())
    h = a * u
    eh = ea * u.abs() + eu * (a.abs() + ea) + 2.0 ** -23 * h.abs()
    return h, _bf16_out(h, eh), g, u, eg, eu, a, ea


def gated_backward(X, Wg, Wu, name, dH):
    _, _, g, u, eg, eu, a, ea = gated(X, Wg, Wu, name)
    X, Wg, Wu, dH = X.double(), Wg.double(), Wu.double(), dH.double()
    d = act_grad(g, name)
    ed = 1.2 * eg + FAST * (1 + g.abs())
    if name == "relu":
        ed = (g.abs() <= eg).double()
    if name == "none":
        ed = torch.zeros_like(d)
    dg, du = dH * u * d, dH * a
    edg = dH.abs() * (u.abs() * ed + eu * (d.abs() + ed)) + 2.0 ** -22 * dg.abs()
    edu = dH.abs() * ea + 2.0 ** -23 * du.abs()
    edg, edu = (e + HALF * (v.abs() + e) + TINY for e, v in ((edg, dg), (edu, du)))
    return _products(X, [Wg, Wu], [dg, du], [edg, edu])


def xent(X, W, y, dl=None):
    """loss, lse and (with dl) dX, dW, each with its bound.  The exponentials may
    have been kept as fp16 relative to a column block's largest: 2^-11 of
    themselves, or half an fp16 subnormal step of the row's largest."""
    X, W = X.double(), W.double()
    T, D = X.shape
    V = W.shape[0]
    logits = X @ W.t()
    # the sum of exponentials: each logit's error, the fast exponential's, and
    # V fp32 additions of positive numbers in at most V / 32 + 32 chained steps
    el = step(D) * (X.abs() @ W.abs().t())
    spread = logits.amax(1) - logits.amin(1)
    elog = el.amax(1) + 2.0 ** -22 * (1 + spread) + (V / 32 + 64) * 2.0 ** -24
    lse = torch.logsumexp(logits, 1)
    elog = elog + 2.0 ** -22 * lse.abs()
    valid = (y >= 0) & (y < V)
    at = torch.where(valid, y, 0).unsqueeze(1)
    ly, ely = logits.gather(1, at).squeeze(1), el.gather(1, at).squeeze(1)
    zero = torch.zeros_like(lse)
    loss = torch.where(valid, lse - ly, zero)
    out = {"lse": (lse, elog),
           "loss": (loss, torch.where(valid, elog + ely + 2.0 ** -23 * loss.abs(), zero))}
    if dl is None:
        return out
    w = torch.where(valid, dl.double(), zero).unsqueeze(1)
    p = torch.exp(logits - lse.unsqueeze(1))
    ep = p * (torch.expm1(el + elog.unsqueeze(1)) + 2.0 ** -20 + 2.0 ** -22 * logits.abs())
    ep = ep + 2.0 ** -11 * p + 2.0 ** -25 * p.amax(1, keepdim=True)
    p = p.scatter_add(1, at, -torch.ones_like(at, dtype=torch.float64))
    d, e = p * w, ep * w.abs()
    e = e + HALF * (d.abs() + e) + TINY
    dX, dW = d @ W, d.t() @ X
    eX = e @ W.abs() + step(V) * (d.abs() @ W.abs())
    eW = e.t() @ X.abs() + step(T) * (d.abs().t() @ X.abs())
    out["dX"] = (dX, _bf16_out(dX, eX))
    out["dW"] = (dW, _bf16_out(dW, eW))
    return out


def check(got, ref, bound, what=""):
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    over = (got - ref).abs() - bound
    if over.numel() and over.max() > 0:
        i = int(over.argmax())
        raise AssertionError(f"{what}: {int((over > 0).sum())} of {over.numel()} entries beyond "
                             f"the bound; worst at {i}: {got.flatten()[i]:g} for "
                             f"{ref.flatten()[i]:g}, bound {bound.flatten()[i]:g}")
