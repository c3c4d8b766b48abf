"""A one-block language model trained and sampled with the library's operators.

The block is the dense part of a transformer layer over a bag of the last few
tokens (no attention), so that every learned product runs through the library:

    h0 = mean of the context's embeddings            (torch: a gather)
    h1 = silu(h0 Wa + ba) + h0                       linear_bf16
    g  = silu(h1 Wg) * (h1 Wu)                       gated_bf16
    h2 = g Wd + h1                                   linear_bf16
    loss = cross entropy of h2 E^T                   xent_bf16_grad (E: the embeddings)

Training uses the backward entry points and SGD (clipped to a gradient norm of 1) on fp32
master weights;
sampling runs the same forward calls one token at a time.  The text is a
periodic sequence of random tokens, which the block learns by heart.

    python examples/train_step.py [--steps N]
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

    def step(self, ids, target, lr):
        """One SGD step; the mean loss over the targets that count."""
        T, D, F, V, p = ids.shape[0], self.D, self.F, self.V, self.p
        h0, h1, g, h2, z, gu = self.body(ids, keep=True)
        valid = (target >= 0).sum()
        dloss = torch.ones(T, device="cuda") / valid
        loss = torch.empty(T, device="cuda")
        dh2, dE = torch.empty_like(h2), torch.empty_like(p["E"])
        pg.xent_bf16_grad(T, V, D, h2, p["E"], target, dloss, loss, None, dh2, dE)

        dg, dWd = torch.empty_like(g), torch.empty_like(p["Wd"])
        pg.linear_bf16_backward(T, D, F, g, p["Wd"], None, "none", dh2, dg, dWd, None)
        dh1, dWg, dWu = torch.empty_like(h1), torch.empty_like(p["Wg"]), torch.empty_like(p["Wu"])
        pg.gated_bf16_backward(T, F, D, h1, p["Wg"], p["Wu"], "silu", dg, dh1, dWg, dWu, preact=gu)
        dh1 += dh2  # the residual of h2
        dh0, dWa, dba = torch.empty_like(h0), torch.empty_like(p["Wa"]), torch.empty_like(p["ba"])
        pg.linear_bf16_backward(T, D, D, h0, p["Wa"], p["ba"], "silu", dh1, dh0, dWa, dba,
                                preact=z)
        dh0 += dh1  # the residual of h1
        grads = {"E": dE.float(), "Wa": dWa, "ba": dba, "Wg": dWg, "Wu": dWu, "Wd": dWd}
        share = (dh0.float() / self.C).repeat_interleave(self.C, 0)
        grads["E"].index_add_(0, ids.reshape(-1), share)
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


def main(steps=200, lr=0.5, quiet=False):
    g = torch.Generator(device="cuda").manual_seed(1)
    model = Block()
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
    a = ap.parse_args()
    main(a.steps)
