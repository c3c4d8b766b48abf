"""Definitions in 64 bits of the operators of a mixture-of-experts block, with the error a
right kernel may have, element by element.

The bounds are built from what the kernels are documented to do, before any of them ran:
  * fp32 sums of n terms in a tree over chains of c: (c + log2 n) roundings of 2^-24 of
    the sum of magnitudes;
  * the norm: chains of at most 40 squares a thread, ten steps of a tree, mean, eps, root
    and divide: rstd is within 2^-19 of itself (the root halves the sum's error);
  * exp: 2 units in the last place (2^-22), its argument off by 2^-24 of its size;
  * a bf16 output is off by 2^-8 of itself (2^-133 below the normal range).
The experts' products are the dense operators' on each group of rows.
"""
from __future__ import annotations

import math

import torch

import operator_reference as ref

RSTD = 2.0 ** -19
EPS24 = 2.0 ** -24


def bf16_out(y, err):
    return err + ref.HALF * (y.abs() + err) + ref.TINY


def norm(S, gain, eps):
    """(y, error of the unrounded y, n, rstd) for the stored S."""
    s = S.double()
    g = torch.ones(s.shape[1], dtype=torch.float64, device=s.device) if gain is None \
        else gain.double()
    rstd = 1 / torch.sqrt(s.square().mean(1, keepdim=True) + eps)
    n = s * rstd
    y = n * g
    return y, y.abs() * (RSTD + 4 * EPS24), n, rstd


def norm_backward(S, gain, eps, dY, dS):
    """{"dX": (value, bound), "dgain": (value, bound)}."""
    T, D = S.shape
    _, _, n, rstd = norm(S, gain, eps)
    dy = dY.double()
    a = dy if gain is None else dy * gain.double()
    m = (a * n).mean(1, keepdim=True)
    dx = rstd * (a - n * m)
    # a and n m each carry rstd's error and that of the sum behind m
    size = rstd * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True))
    err = size * (4 * RSTD)
    if dS is not None:
        dx = dx + dS.double()
        err = err + 2 * EPS24 * dx.abs()
    dg = (dy * n).sum(0)
    eg = (dy * n).abs().sum(0) * (2 * RSTD + (T + 16) * EPS24)
    return {"dX": (dx, bf16_out(dx, err)), "dgain": (dg, bf16_out(dg, eg))}


def route(z, k, normalise):
    """(experts, weights, bound of the weights): -1 and 0 where nothing is open."""
    z = z.double()
    T, E = z.shape
    order = torch.argsort(-z, dim=1, stable=True)[:, :k]
    top = z.gather(1, order)
    open_ = top > -math.inf
    experts = torch.where(open_, order, -1).int()
    most = torch.where(open_[:, :1], top[:, :1], 0.0)
    e = torch.where(open_, torch.exp(top - most), 0.0)
    total = e.sum(1, keepdim=True) if normalise else torch.exp(z - most).sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0)
    w = e / total
    finite = torch.where(z > -math.inf, z, most)
    spread = (most - finite).amax(1, keepdim=True)
    rel = (spread + E / 32 + 24) * 2.0 ** -22
    return experts, w, w * rel + 2.0 ** -140, rel


def route_backward(z, k, normalise, experts, dw):
    _, _, _, rel = route(z, k, normalise)
    zd = z.double()
    ok = (experts >= 0) & (experts < z.shape[1])
    at = torch.where(ok, experts, 0).long()
    top = torch.where(ok, zd.gather(1, at), -math.inf)
    p_all = torch.softmax(torch.where((zd > -math.inf).any(1, keepdim=True), zd, 0.0), 1)
    if normalise:
        some = ok.any(1, keepdim=True)
        w = torch.where(some, torch.softmax(torch.where(some, top, 0.0), 1), 0.0)
    else:
        w = torch.where(ok, p_all.gather(1, at), 0.0)
    d = torch.where(ok, dw.double(), 0.0)
    dot, size = (w * d).sum(1, keepdim=True), (w * d).abs().sum(1, keepdim=True)
    own = w * (d - dot) if normalise else w * d
    own_size = w * (d.abs() + size) if normalise else w * d.abs()
    base = torch.zeros_like(zd) if normalise else -p_all * dot
    base_size = torch.zeros_like(zd) if normalise else p_all * size
    if not normalise:  # rows without an open expert have no gradient
        none = ~(zd > -math.inf).any(1, keepdim=True)
        base, base_size = (torch.where(none, 0.0, v) for v in (base, base_size))
    dz = base.scatter_add(1, at, torch.where(ok, own, 0.0))
    size = base_size.scatter_add(1, at, torch.where(ok, own_size, 0.0))
    return dz, size * (2 * rel + k * EPS24) + 2.0 ** -140


def sort(experts, E):
    flat = experts.reshape(-1).long().cpu()
    rows = torch.full_like(flat, -1)
    offsets = [0]
    for e in range(E):
        at = (flat == e).nonzero().squeeze(1)
        rows[at] = offsets[-1] + torch.arange(at.numel())
        offsets.append(offsets[-1] + at.numel())
    return torch.tensor(offsets, dtype=torch.int32), rows.reshape(experts.shape).int()


def combine(Ys, rows, weights, residual):
    T, k = rows.shape
    ok = rows >= 0
    y = Ys.double()[rows.clamp(min=0).long()] * ok.unsqueeze(2)
    y = torch.where(ok.unsqueeze(2), y, 0.0)
    if weights is not None:
        y = y * weights.double().unsqueeze(2)
    total, size = y.sum(1), y.abs().sum(1)
    if residual is not None:
        total, size = total + residual.double(), size + residual.double().abs()
    return total, bf16_out(total, (k + 2) * EPS24 * size)


def combine_backward(Ys, rows, weights, dY):
    """(dYs rows in slot order, bound, dweights, bound); zero where a slot does not count."""
    ok = (rows >= 0).unsqueeze(2)
    y = torch.where(ok, Ys.double()[rows.clamp(min=0).long()], 0.0)
    dy = dY.double().unsqueeze(1)
    w = torch.ones(rows.shape, dtype=torch.float64, device=Ys.device) if weights is None \
        else weights.double()
    d = torch.where(ok, w.unsqueeze(2) * dy, 0.0)
    dw = (dy * y).sum(2)
    return d, bf16_out(d, EPS24 * d.abs()), dw, \
        (dy * y).abs().sum(2) * (dY.shape[1] / 32 + 16) * EPS24 + 2.0 ** -140


def groups(offsets):
    o = offsets.tolist()
    return [(e, a, b) for e, (a, b) in enumerate(zip(o[:-1], o[1:]))]


def over_groups(offsets, f):
    """f(expert, first row, last row) -> {name: (value, bound)} for each group; rows' results
    joined in order ("Y", "H", "dX", ...) and weights' stacked ("dW0", "dW1")."""
    parts = {}
    for e, a, b in groups(offsets):
        for name, pair in f(e, a, b).items():
            parts.setdefault(name, []).append(pair)
    join = {}
    for name, pairs in parts.items():
        put = torch.stack if name.startswith("dW") else torch.cat
        join[name] = tuple(put([p[i] for p in pairs]) for i in range(2))
    return join


def experts_linear(offsets, X, W):
    def one(e, a, b):
        y, bound, _, _ = ref.linear(X[a:b], W[e], None, "none", None)
        return {"Y": (y, bound)}
    return over_groups(offsets, one)


def experts_linear_backward(offsets, X, W, dY):
    def one(e, a, b):
        out = ref.linear_backward(X[a:b], W[e], None, "none", dY[a:b])
        return {k: out[k] for k in ("dX", "dW0")}
    return over_groups(offsets, one)


def experts_gated(offsets, X, Wg, Wu, act):
    def one(e, a, b):
        h, bound, g, u, eg, eu, _, _ = ref.gated(X[a:b], Wg[e], Wu[e], act)
        return {"H": (h, bound), "G": (g, eg), "U": (u, eu)}
    return over_groups(offsets, one)


def experts_gated_backward(offsets, X, Wg, Wu, act, dH):
    return over_groups(offsets, lambda e, a, b: ref.gated_backward(X[a:b], Wg[e], Wu[e], act,
                                                                   dH[a:b]))
