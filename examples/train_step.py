"""A one-block language model trained and sampled with the library's operators.

The block is the dense part of a transformer layer over a bag of the last few
tokens (no attention), so that every learned product runs through the library:

    h0 = mean of the context's embeddings            (torch: a gather)
    h1 = silu(h0 Wa + ba) + h0                       linear_bf16
    g  = silu(h1 Wg) * (h1 Wu)                       gated_bf16
    h2 = g Wd + h1                                   linear_bf16
    loss = cross entropy of h2 E^T                   xent_bf16_grad (E: the embeddings)

With --experts E the gated block is a mixture of E of them behind a norm, of which each
token takes two:

    n  = h1 gain / rms(h1)                           rmsnorm_bf16
    experts, w = the two largest of softmax(n Wr)    gemm_bf16, route_topk
    n's rows sorted by expert                        expert_sort, expert_gather_bf16
    y  = (silu(n Wg[e]) * (n Wu[e])) Wd[e]           experts_gated_bf16, experts_linear_bf16
    h2 = h1 + sum over a token's two of w y          expert_combine_bf16

Training uses the backward entry points and SGD (clipped to a gradient norm of 1) on fp32
master weights;
sampling runs the same forward calls one token at a time.  The text is a
periodic sequence of random tokens, which the block learns by heart.

    python examples/train_step.py [--steps N] [--experts E]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import software_pipelined_tiled_loop_gb300 as pg  # noqa: E402

BF16 = torch.bfloat16


class Block:
    def __init__(self, vocab=1000, width=256, hidden=512, context=4, seed=0):
        self.V, self.D, self.F, self.C = vocab, width, hidden, context
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, std):
            return torch.randn(shape, generator=g, device="cuda") * std

        self.master = {
            "E": weight(vocab, width, std=0.2),
            "Wa": weight(width, width, std=width ** -0.5),
            "ba": torch.zeros(width, device="cuda"),
            "Wg": weight(width, hidden, std=width ** -0.5),
            "Wu": weight(width, hidden, std=width ** -0.5),
            "Wd": weight(hidden, width, std=hidden ** -0.5),
        }
        self.refresh()

    def refresh(self):
        self.p = {k: v.to(BF16) for k, v in self.master.items()}

    def body(self, ids, keep):
        """h2 of contexts ids (T x C), and what the backward pass needs."""
        T, D, F, p = ids.shape[0], self.D, self.F, self.p
        h0 = p["E"][ids].float().mean(1).to(BF16)
        h1, g, h2 = (h0.new_empty((T, n)) for n in (D, F, D))
        z = torch.empty((T, D), device="cuda") if keep else None
        gu = torch.empty((2, T, F), device="cuda") if keep else None
        pg.linear_bf16(T, D, D, h0, p["Wa"], p["ba"], "silu", h0, h1, preact=z)
        pg.gated_bf16(T, F, D, h1, p["Wg"], p["Wu"], "silu", g, preact=gu)
        pg.linear_bf16(T, D, F, g, p["Wd"], None, "none", h1, h2)
        return h0, h1, g, h2, z, gu

    def gradients(self, ids, target):
        """The losses, how many targets count, and every weight's gradient of their mean."""
        T, D, F, p = ids.shape[0], self.D, self.F, self.p
        h0, h1, g, h2, z, gu = self.body(ids, keep=True)
        loss, valid, dh2, dE = self.loss_gradient(h2, target)

        dg, dWd = torch.empty_like(g), torch.empty_like(p["Wd"])
        pg.linear_bf16_backward(T, D, F, g, p["Wd"], None, "none", dh2, dg, dWd, None)
        dh1, dWg, dWu = torch.empty_like(h1), torch.empty_like(p["Wg"]), torch.empty_like(p["Wu"])
        pg.gated_bf16_backward(T, F, D, h1, p["Wg"], p["Wu"], "silu", dg, dh1, dWg, dWu, preact=gu)
        dh1 += dh2  # the residual of h2
        return loss, valid, {"Wg": dWg, "Wu": dWu, "Wd": dWd,
                             **self.front_gradients(ids, h0, z, dh1, dE)}

    def loss_gradient(self, h2, target):
        T, D, V, p = h2.shape[0], self.D, self.V, self.p
        valid = (target >= 0).sum()
        dloss = torch.ones(T, device="cuda") / valid
        loss = torch.empty(T, device="cuda")
        dh2, dE = torch.empty_like(h2), torch.empty_like(p["E"])
        pg.xent_bf16_grad(T, V, D, h2, p["E"], target, dloss, loss, None, dh2, dE)
        return loss, valid, dh2, dE

    def front_gradients(self, ids, h0, z, dh1, dE):
        """Of what makes h1: the first layer and, added to dE, the embeddings."""
        T, D, p = ids.shape[0], self.D, self.p
        dh0, dWa, dba = torch.empty_like(h0), torch.empty_like(p["Wa"]), torch.empty_like(p["ba"])
        pg.linear_bf16_backward(T, D, D, h0, p["Wa"], p["ba"], "silu", dh1, dh0, dWa, dba,
                                preact=z)
        dh0 += dh1  # the residual of h1
        grads = {"E": dE.float(), "Wa": dWa, "ba": dba}
        share = (dh0.float() / self.C).repeat_interleave(self.C, 0)
        grads["E"].index_add_(0, ids.reshape(-1), share)
        return grads

    def step(self, ids, target, lr):
        """One SGD step; the mean loss over the targets that count."""
        loss, valid, grads = self.gradients(ids, target)
        norm = torch.sqrt(sum(v.float().square().sum() for v in grads.values()))
        scale = lr / norm.clamp(min=1.0)
        for k, v in grads.items():
            self.master[k] -= scale * v.float()
        self.refresh()
        return (loss.sum() / valid).item()

    def next_token(self, ids):
        """Greedy next token of one context: each call streams the weights once."""
        h2 = self.body(ids.view(1, -1), keep=False)[3]
        logits = torch.empty((1, self.V), device="cuda", dtype=BF16)
        pg.linear_bf16(1, self.V, self.D, h2, self.p["E"].t().contiguous(), None, "none", None,
                       logits)
        return int(logits.argmax())


class SparseBlock(Block):
    """The block with `experts` gated blocks of hidden / 2, of which a token takes two."""
    K, EPS = 2, 1e-6

    def __init__(self, vocab=1000, width=256, hidden=512, context=4, experts=8, seed=0):
        super().__init__(vocab, width, hidden, context, seed)
        self.F, self.X = hidden // 2, experts
        g = torch.Generator(device="cuda").manual_seed(seed + 1)

        def weight(*shape, std):
            return torch.randn(shape, generator=g, device="cuda") * std

        E, D, F = experts, width, self.F
        self.master.update({
            "gain": torch.ones(D, device="cuda"),
            "Wr": weight(D, E, std=D ** -0.5),
            "Wg": weight(E, D, F, std=D ** -0.5), "Wu": weight(E, D, F, std=D ** -0.5),
            "Wd": weight(E, F, D, std=F ** -0.5),
        })
        self.refresh()

    def body(self, ids, keep):
        T, D, F, E, K, p = ids.shape[0], self.D, self.F, self.X, self.K, self.p

        def new(*shape, dtype=BF16):
            return torch.empty(shape, dtype=dtype, device="cuda")

        f32, i32 = torch.float32, torch.int32
        h0 = p["E"][ids].float().mean(1).to(BF16)
        h1, n, h2 = new(T, D), new(T, D), new(T, D)
        z = new(T, D, dtype=f32) if keep else None
        pg.linear_bf16(T, D, D, h0, p["Wa"], p["ba"], "silu", h0, h1, preact=z)
        pg.rmsnorm_bf16(T, D, h1, None, p["gain"], self.EPS, None, n)
        logits, w = new(T, E, dtype=f32), new(T, K, dtype=f32)
        experts, rows, offsets = new(T, K, dtype=i32), new(T, K, dtype=i32), new(E + 1, dtype=i32)
        pg.gemm_bf16(T, E, D, 1.0, n, p["Wr"], 0.0, logits)
        pg.route_topk(T, E, K, logits, False, experts, w)
        pg.expert_sort(T, E, K, experts, offsets, rows)
        ns, g, y = new(T * K, D), new(T * K, F), new(T * K, D)
        gu = new(2, T * K, F, dtype=f32) if keep else None
        pg.expert_gather_bf16(T, K, D, n, rows, ns)
        pg.experts_gated_bf16(T * K, F, D, E, offsets, ns, p["Wg"], p["Wu"], "silu", g, preact=gu)
        pg.experts_linear_bf16(T * K, D, F, E, offsets, g, p["Wd"], y)
        pg.expert_combine_bf16(T, K, D, y, rows, w, h1, h2)
        return h0, h1, (n, logits, experts, w, rows, offsets, ns, g, y), h2, z, gu

    def gradients(self, ids, target):
        T, D, F, E, K, p = ids.shape[0], self.D, self.F, self.X, self.K, self.p
        h0, h1, (n, logits, experts, w, rows, offsets, ns, g, y), h2, z, gu = self.body(ids, True)
        loss, valid, dh2, dE = self.loss_gradient(h2, target)
        like = torch.empty_like
        dy, dw, dg, dns = like(y), like(w), like(g), like(ns)
        dWd, dWg, dWu = like(p["Wd"]), like(p["Wg"]), like(p["Wu"])
        pg.expert_combine_bf16_backward(T, K, D, y, rows, w, dh2, dy, dw)
        pg.experts_linear_bf16_backward(T * K, D, F, E, offsets, g, p["Wd"], dy, dg, dWd)
        pg.experts_gated_bf16_backward(T * K, F, D, E, offsets, ns, p["Wg"], p["Wu"], "silu", dg,
                                       dns, dWg, dWu, preact=gu)
        dlogits, dn = like(logits), like(n)
        pg.route_topk_backward(T, E, K, logits, False, experts, dw, dlogits)
        dWr, dr = like(p["Wr"]), dlogits.to(BF16)
        pg.linear_bf16_backward(T, E, D, n, p["Wr"], None, "none", dr, dn, dWr, None)
        # the gather's gradient, beside the router's
        pg.expert_combine_bf16(T, K, D, dns, rows, None, dn, dn)
        dh1, dgain = like(h1), like(p["gain"])
        pg.rmsnorm_bf16_backward(T, D, h1, p["gain"], self.EPS, dn, dh2, dh1, dgain)
        return loss, valid, {"gain": dgain, "Wr": dWr, "Wg": dWg, "Wu": dWu, "Wd": dWd,
                             **self.front_gradients(ids, h0, z, dh1, dE)}


def main(steps=200, lr=0.5, quiet=False, experts=0):
    g = torch.Generator(device="cuda").manual_seed(1)
    model = SparseBlock(experts=experts) if experts else Block()
    period = torch.randint(0, model.V, (97,), generator=g, device="cuda")
    text = period.repeat(6)
    ids = text.unfold(0, model.C, 1)[:-1].contiguous()
    target = text[model.C:].clone()
    target[::50] = -100  # padding: counts for nothing
    losses = []
    for i in range(steps):
        losses.append(model.step(ids, target, lr))
        if not quiet and (i % 20 == 0 or i == steps - 1):
            print(f"step {i:3d}  loss {losses[-1]:.4f}")
    ctx = period[:model.C].clone()
    got = []
    for _ in range(20):
        t = model.next_token(ctx)
        got.append(t)
        ctx = torch.cat([ctx[1:], torch.tensor([t], device="cuda")])
    right = sum(int(a == b) for a, b in zip(got, period[model.C:model.C + 20].tolist()))
    assert pg.pgemm_get_device_status() == 0
    if not quiet:
        print(f"{right} of 20 sampled tokens continue the text")
    return losses, right


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--experts", type=int, default=0, help="of a mixture (0: one gated block)")
    a = ap.parse_args()
    main(a.steps, experts=a.experts)
