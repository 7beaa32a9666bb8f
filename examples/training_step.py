"""One training step of a small model around the optimizer, on one GPU.

    python examples/training_step.py [--steps 20]

A one-layer language model with a tied embedding and a gated feed-forward
layer, trained with the clipped policy loss. The step runs the library's
operators together: embedding lookup, activations held in 8 bits between
forward and backward, the policy loss with its gradient, weight gradients from
the 8-bit activations, the embedding's gradient added onto the output head's,
and the fused Muon update of the two weight matrices. The plain matrix
products in between are torch's.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from newton_schulz_quintic_gb300 import api  # noqa: E402


class Model:
    """table (vocab x dim, tied with the output head), w_gu (2 ffn x dim: gate
    above up) and w_down (dim x ffn), all bf16, and the optimizer's momenta."""

    def __init__(self, vocab=1000, dim=256, ffn=512, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(rows, cols, std):
            return (torch.randn((rows, cols), device=device, generator=g) * std).to(torch.bfloat16)

        self.table = normal(vocab, dim, dim ** -0.5)
        self.w_gu = normal(2 * ffn, dim, dim ** -0.5)
        self.w_down = normal(dim, ffn, ffn ** -0.5)
        self.scale = math.sqrt(dim)
        self.momenta = [torch.zeros_like(self.w_gu), torch.zeros_like(self.w_down)]

    def forward(self, ids):
        """Logits, and what the backward pass needs: 8-bit activations and y."""
        x = api.embed_lookup(self.table, ids, scale=self.scale)
        ck_x = api.checkpoint_store(x)
        gu = x @ self.w_gu.t()
        ffn = gu.shape[1] // 2
        h, ck_gate, ck_up = api.gated_forward(gu[:, :ffn], gu[:, ffn:])
        ck_h = api.checkpoint_store(h)
        y = x + h @ self.w_down.t()
        return y @ self.table.t() / self.scale, (ids, ck_x, ck_gate, ck_up, ck_h, y)

    def backward(self, dlogits, kept):
        """Gradients of table (fp32), w_gu and w_down."""
        ids, ck_x, ck_gate, ck_up, ck_h, y = kept
        dlogits = dlogits / self.scale
        dtable = (dlogits.t() @ y).float()                      # as the output head
        dy = dlogits @ self.table
        dw_down = api.checkpoint_wgrad(dy, ck_h)[0]
        dgu, _ = api.gated_backward(dy @ self.w_down, ck_gate, ck_up, recompute=False)
        dw_gu = api.checkpoint_wgrad(dgu, ck_x)[0]
        dx = dy + dgu @ self.w_gu
        api.embed_grad(dx, ids, grad=dtable, scale=self.scale, accumulate=True)  # as the embedding
        return dtable, dw_gu, dw_down

    def step(self, ids, targets, advantages, weights, old_logp=None, ref_logp=None, lr=0.02, table_lr=0.1, **loss):
        """One policy-gradient step; returns the loss's result."""
        logits, kept = self.forward(ids)
        out = api.policy_loss(logits, targets, advantages, weights, old_logp=old_logp, ref_logp=ref_logp, **loss)
        dtable, dw_gu, dw_down = self.backward(out.dlogits, kept)
        grads = [dw_gu, dw_down]
        api.muon_update_batched(grads, self.momenta, grads, mu=0.95)  # the update over the gradient
        self.w_gu.sub_(grads[0], alpha=lr)
        self.w_down.sub_(grads[1], alpha=lr)
        self.table.sub_((dtable * table_lr).to(self.table.dtype))
        return out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=2048)
    args = ap.parse_args()
    model = Model()
    g = torch.Generator(device="cuda").manual_seed(1)
    n, vocab = args.tokens, model.table.shape[0]
    ids = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    targets = (ids * 7 + 1) % vocab
    targets[: n // 4] = -100                                    # prompt tokens: no loss
    weights = (targets >= 0).float() / (targets >= 0).sum()
    advantages = torch.ones(n, device="cuda")
    first, _ = model.forward(ids)
    reference = api.token_logprobs(first, targets)
    for k in range(args.steps):
        out = model.step(ids, targets, advantages, weights, ref_logp=reference, kl_coef=0.01)
        if k % 5 == 0 or k == args.steps - 1:
            live = targets >= 0
            print(f"step {k:3d}  loss {float(out.loss):8.4f}  mean logp {float(out.logp[live].mean()):8.4f}  "
                  f"mean kl {float(out.kl[live].mean()):8.4f}")


if __name__ == "__main__":
    main()
