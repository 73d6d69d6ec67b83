"""One training step of a mixture-of-experts layer: routing, FP8 products
forwards and backwards, and the Muon step on the FP32 weights.

    python examples/moe_training_step.py [--hidden 4096 --intermediate 1536 --experts 512 --tokens 8192]

The layer is y = sum over a token's experts e of w_e down_e relu(up_e x)^2, with
a router x -> logits of the experts.  Its weights are FP32; every step quantises
them once in both orientations, and the gradients arrive as FP32
[experts][rows][cols], which muon_step takes as they are.  ``forward`` alone is
the serving path.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_03_gb300 as ns  # noqa: E402

F8 = torch.float8_e4m3fn


def _blocks(n: int) -> int:
    return -(-n // 128)


class Quantized:
    """FP8 copies of weights [experts, n, k] and of their transposes."""

    def __init__(self, w):
        e, n, k = w.shape
        dev = w.device
        self.q = torch.empty(e, n, k, dtype=F8, device=dev)
        self.s = torch.empty(e, _blocks(n), _blocks(k), dtype=torch.uint8, device=dev)
        self.qt = torch.empty(e, k, n, dtype=F8, device=dev)
        self.st = torch.empty(e, _blocks(k), _blocks(n), dtype=torch.uint8, device=dev)

    def update(self, h, w):
        ns.muon_fp8_quantize_blocks(h, w, self.q, self.s, self.qt, self.st)


class ExpertLayer:
    def __init__(self, handle, hidden, intermediate, experts, top_k, seed=0, device="cuda"):
        g = torch.Generator(device).manual_seed(seed)

        def weight(*shape):
            return torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5

        self.h, self.top_k, self.experts = handle, top_k, experts
        self.up = weight(experts, intermediate, hidden)
        self.down = weight(experts, hidden, intermediate)
        self.router = weight(1, experts, hidden)
        self.weights = [self.up, self.down, self.router]
        self.momentum = [torch.zeros_like(w) for w in self.weights]
        self.grads = [torch.zeros_like(w) for w in self.weights]
        self.q_up, self.q_down = Quantized(self.up), Quantized(self.down)
        self.bias = torch.zeros(experts, device=device)
        self.quantize()

    def quantize(self):
        self.q_up.update(self.h, self.up)
        self.q_down.update(self.h, self.down)

    # ---------------------------------------------------------------- pieces
    def _rows(self, x, pos=None, rows=None, offsets=None):
        """x in FP8 rows (sent to the rows pos[t] of the tokens' experts; or
        the experts' rows themselves)."""
        r, d = x.shape[0] if rows is None else rows, x.shape[1]
        q = torch.empty(r, d, dtype=F8, device=x.device)
        s = torch.empty(r, _blocks(d), dtype=torch.uint8, device=x.device)
        ns.muon_fp8_quantize_rows(self.h, x, q, s, pos=pos, offsets=offsets)
        return q, s

    def _cols(self, x, offsets, rows, slots=None):
        """x in FP8 columns of each expert's rows, for a weight gradient."""
        cap, d = ns.muon_fp8_cols_capacity(rows, self.experts), x.shape[1]
        q = torch.empty(d, cap, dtype=F8, device=x.device)
        s = torch.empty(cap // 128, d, dtype=torch.uint8, device=x.device)
        ns.muon_fp8_quantize_cols(self.h, x, offsets, q, s, slots=slots, top_k=self.top_k)
        return q, s

    def _product(self, x, w, scales, offsets):
        y = torch.empty(x[0].shape[0], w.shape[1], dtype=torch.bfloat16, device=w.device)
        ns.muon_fp8_grouped_matmul(self.h, x[0], x[1], w, scales, offsets, y)
        return y

    # ---------------------------------------------------------------- passes
    def forward(self, x, mask=None):
        """x [tokens, hidden] BF16 -> (y [tokens, hidden] BF16, what backward needs).
        Tokens whose mask is 0 (padding) go to no expert: y is 0 there."""
        t, k, dev = x.shape[0], self.top_k, x.device
        logits = x.float() @ self.router[0].t()
        ids = torch.empty(t, k, dtype=torch.int32, device=dev)
        w = torch.empty(t, k, device=dev)
        ns.muon_moe_route(self.h, logits, ids, w, bias=self.bias, mask=mask)
        offsets = torch.empty(self.experts + 1, dtype=torch.int32, device=dev)
        slots = torch.empty(t * k, dtype=torch.int32, device=dev)
        pos = torch.empty(t, k, dtype=torch.int32, device=dev)
        ns.muon_moe_plan(self.h, ids, offsets, slots, pos)
        hidden = self._product(self._rows(x, pos, t * k), self.q_up.q, self.q_up.s, offsets)
        act = torch.relu(hidden).square()
        y = self._product(self._rows(act, offsets=offsets), self.q_down.q, self.q_down.s, offsets)
        out = torch.empty_like(x)
        ns.muon_moe_combine(self.h, y, pos, w, out)
        return out, (x, logits, ids, w, offsets, slots, pos, hidden, act, y)

    def backward(self, grad, saved):
        """Gradient of x; the weights' gradients are left in self.grads."""
        x, logits, ids, w, offsets, slots, pos, hidden, act, y = saved
        rows = y.shape[0]
        g_y, g_w = torch.empty_like(y), torch.empty_like(w)
        ns.muon_moe_combine_backward(self.h, grad, y, pos, w, g_y, g_w)
        g_act = self._product(self._rows(g_y, offsets=offsets), self.q_down.qt, self.q_down.st, offsets)
        g_hidden = g_act * (2 * torch.relu(hidden))
        g_rows = self._product(self._rows(g_hidden, offsets=offsets), self.q_up.qt, self.q_up.st, offsets)
        g_x = torch.empty_like(x)
        ns.muon_moe_combine(self.h, g_rows, pos, None, g_x)
        cols = self._cols(g_y, offsets, rows) + self._cols(act, offsets, rows)
        ns.muon_fp8_grouped_wgrad(self.h, *cols, offsets, self.grads[1])
        cols = self._cols(g_hidden, offsets, rows) + self._cols(x, offsets, rows, slots)
        ns.muon_fp8_grouped_wgrad(self.h, *cols, offsets, self.grads[0])
        g_logits = torch.empty_like(logits)
        ns.muon_moe_route_backward(self.h, logits, ids, g_w, g_logits)
        torch.matmul(g_logits.t(), x.float(), out=self.grads[2][0])
        return (g_x.float() + g_logits @ self.router[0]).to(x.dtype)

    def step(self, lr=0.02, wd=0.0, mu=0.9):
        groups = [(w.shape[1], w.shape[2], w.shape[0]) for w in self.weights]
        ns.muon_step(self.h, groups, self.momentum, self.grads, self.weights, lr, wd, mu)
        self.quantize()


def train(layer, x, target, steps, lr):
    """Mean squared error to `target` before each step and after the last."""
    losses = []
    for i in range(steps + 1):
        y, saved = layer.forward(x)
        diff = y.float() - target.float()
        losses.append(float(diff.square().mean()))
        if i < steps:
            layer.backward((diff * (2.0 / diff.numel()) * diff.shape[0]).to(x.dtype), saved)
            layer.step(lr=lr)
    ns.muon_last_device_error(layer.h)
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--intermediate", type=int, default=1536)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=7)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    with ns.Handle() as handle:
        layer = ExpertLayer(handle.value, a.hidden, a.intermediate, a.experts, a.top_k)
        g = torch.Generator("cuda").manual_seed(1)
        x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
        target = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16() * 0.1
        for i, loss in enumerate(train(layer, x, target, a.steps, 0.02)):
            print(f"step {i}: loss {loss:.5f}")
        one, _ = layer.forward(x[:1])      # serving: the same path with one token
        print("one token:", tuple(one.shape))


if __name__ == "__main__":
    main()
