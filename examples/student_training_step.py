"""Training steps of a small student: gated experts, a head, and a loss on its logits
whose gradient goes all the way back to the Muon and AdamW steps.

    python examples/student_training_step.py [--loss distill|policy --vocab 131072 --tokens 2048]

``distill``: towards a teacher's top logits of each token.  ``policy``: sampled tokens
with their advantages, the log probabilities of the policy that sampled them and of a
reference; prompt tokens are masked.  Hidden states stand in for the layers below.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from moe_training_step import GatedExpertLayer, ns  # noqa: E402


class Student:
    def __init__(self, handle, hidden, intermediate, experts, top_k, vocab, seed=0, device="cuda"):
        self.h = handle
        self.layer = GatedExpertLayer(handle, hidden, intermediate, experts, top_k, seed, device)
        g = torch.Generator(device).manual_seed(seed + 2)
        self.head = torch.randn(vocab, hidden, generator=g, device=device) * 0.02
        self.head_grad = torch.zeros_like(self.head)
        self.head_state = [torch.zeros_like(self.head) for _ in range(2)]
        self.steps = 0

    def logits(self, x, mask=None):
        y, saved = self.layer.forward(x, mask)
        hidden = x + y
        return hidden @ self.head.bfloat16().t(), (hidden, saved)

    def backward(self, grad_logits, saved):
        """From the logits' gradient to that of x; weights' gradients are left in place."""
        hidden, saved = saved
        torch.matmul(grad_logits.float().t(), hidden.float(), out=self.head_grad)
        g = grad_logits @ self.head.bfloat16()
        return g + self.layer.backward(g, saved)

    def step(self, lr):
        self.steps += 1
        self.layer.step(lr=lr)
        ns.muon_adamw_step(self.h, [self.head], [self.head_grad], [self.head_state[0]], [self.head_state[1]], lr * 0.1, 0.9, 0.95, 1e-8,
                           0.0, self.steps)

    def distill(self, x, teacher, ids, mask=None, temperature=2.0):
        """(loss of each token, gradient of x) of the mean over the tokens that count."""
        z, saved = self.logits(x, mask)
        loss, lse = (torch.empty(x.shape[0], device=x.device) for _ in range(2))
        weight = _weights(x.shape[0], mask, x.device)
        # The gradient takes the logits' place.
        ns.muon_distill_loss(self.h, z, teacher, ids, loss, lse, temperature=temperature, scale=temperature ** 2, mask=mask,
                             grad_loss=weight, grad_logits=z)
        return loss, self.backward(z, saved)

    def log_probs(self, x, actions, mask=None, temperature=1.0):
        """Of the actions, at the temperature that they were sampled with (and ``policy`` trains at)."""
        z, _ = self.logits(x, mask)
        loss, logp, lse = (torch.empty(x.shape[0], device=x.device) for _ in range(3))
        ns.muon_policy_loss(self.h, z, actions, torch.zeros_like(loss), loss, logp, lse, mask=mask,
                            temperature=temperature)
        return logp

    def policy(self, x, actions, advantages, old_logp, ref_logp, mask=None, temperature=1.0, **options):
        """As distill; ``old_logp`` and ``ref_logp`` are log_probs of the same temperature."""
        z, saved = self.logits(x, mask)
        loss, logp, lse = (torch.empty(x.shape[0], device=x.device) for _ in range(3))
        weight = _weights(x.shape[0], mask, x.device)
        ns.muon_policy_loss(self.h, z, actions, advantages, loss, logp, lse, old_logp=old_logp, ref_logp=ref_logp, mask=mask,
                            temperature=temperature, grad_loss=weight, grad_logits=z, **options)
        return loss, self.backward(z, saved)


def _weights(tokens, mask, device):
    """Of the mean over the tokens that count."""
    n = torch.full((), float(tokens), device=device) if mask is None else mask.float().sum().clamp(min=1.0)
    return (torch.ones(tokens, device=device) if mask is None else mask.float()) / n


def main():
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--loss", choices=["distill", "policy"], default="distill")
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--intermediate", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--vocab", type=int, default=131072)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    g = torch.Generator("cuda").manual_seed(1)
    with ns.Handle() as handle:
        student = Student(handle.value, a.hidden, a.intermediate, a.experts, a.top_k, a.vocab)
        x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
        if a.loss == "distill":
            ids = torch.randint(0, a.vocab, (a.tokens, 32), generator=g, device="cuda", dtype=torch.int32)
            teacher = torch.randn(a.tokens, 32, generator=g, device="cuda") * 2
            mask = None
            run = lambda: student.distill(x, teacher, ids)  # noqa: E731
        else:
            actions = torch.randint(0, a.vocab, (a.tokens,), generator=g, device="cuda", dtype=torch.int32)
            advantages = torch.randn(a.tokens, generator=g, device="cuda")
            mask = (torch.arange(a.tokens, device="cuda") >= a.tokens // 4).to(torch.uint8)
            old = student.log_probs(x, actions, mask)
            run = lambda: student.policy(x, actions, advantages, old, old, mask, kl_coef=0.05)  # noqa: E731
        weight = _weights(a.tokens, mask, "cuda")
        for i in range(a.steps):
            loss, _ = run()
            student.step(0.02)
            print(f"step {i}: loss {float((loss * weight).sum()):.5f}")
        ns.muon_last_device_error(handle.value)


if __name__ == "__main__":
    main()
