"""The operators together: a mixture-of-experts layer's training step, against
the layer in 64 bits without quantisation."""

import importlib.util
import os

import numpy as np
import pytest

from tests import moe_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_training_step", os.path.join(ROOT, "examples", "moe_training_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


def exact(layer, x, grad, ids):
    """Output, gradient of x and of the three weights, with this choice of experts."""
    x, grad = x.double().cpu().numpy(), grad.double().cpu().numpy()
    up, down, router = (w.double().cpu().numpy() for w in layer.weights)
    router = router[0]
    logits = x @ router.T
    w = ref.weights_of(logits, ids, softmax=False, renorm=True, scale=1.0)
    out, gx = np.zeros_like(x), np.zeros_like(x)
    g_up, g_down, g_w = np.zeros_like(up), np.zeros_like(down), np.zeros_like(w)
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            hid = np.maximum(up[e] @ x[t], 0)
            y = down[e] @ hid**2
            out[t] += w[t, j] * y
            g_w[t, j] = grad[t] @ y
            g_act = down[e].T @ (w[t, j] * grad[t])
            g_hid = g_act * 2 * hid
            g_down[e] += np.outer(w[t, j] * grad[t], hid**2)
            g_up[e] += np.outer(g_hid, x[t])
            gx[t] += up[e].T @ g_hid
    g_logits = ref.route_backward(logits, ids, g_w, softmax=False, renorm=True, scale=1.0)
    return out, gx + g_logits @ router, g_up, g_down, g_logits.T @ x


def test_layer_against_64_bits(example):
    ns = example.ns
    with ns.Handle() as h:
        layer = example.ExpertLayer(h.value, hidden=272, intermediate=144, experts=8, top_k=3, seed=3)
        g = torch.Generator("cuda").manual_seed(5)
        x = torch.randn(65, 272, generator=g, device="cuda").bfloat16()
        grad = torch.randn(65, 272, generator=g, device="cuda").bfloat16()
        y, saved = layer.forward(x)
        gx = layer.backward(grad, saved)
        ns.muon_last_device_error(h.value)
        want = exact(layer, x, grad, saved[2].cpu().numpy())
        got = [v.double().cpu().numpy() for v in (y, gx, layer.grads[0], layer.grads[1], layer.grads[2][0])]
    # e4m3 keeps three bits of fraction: an operand is off by 2.6% (root mean
    # square).  The output sees four of them, the first two doubled by the
    # square, 8% together; the gradients two or four more.
    for name, a, b, tol in zip(("y", "grad x", "grad up", "grad down", "grad router"), got, want, (0.12, 0.16, 0.16, 0.12, 0.16)):
        assert rel(a, b) <= tol, (name, rel(a, b))


def test_training_lowers_the_loss(example):
    ns = example.ns
    with ns.Handle() as h:
        layer = example.ExpertLayer(h.value, hidden=256, intermediate=128, experts=16, top_k=4, seed=1)
        g = torch.Generator("cuda").manual_seed(2)
        x = torch.randn(300, 256, generator=g, device="cuda").bfloat16()
        target = 0.1 * torch.randn(300, 256, generator=g, device="cuda").bfloat16()
        losses = example.train(layer, x, target, 8, lr=0.02)
    assert losses[-1] < 0.5 * losses[0], losses


def test_one_token_and_many_agree(example):
    """The serving call: a token's output does not depend on the tokens beside it."""
    ns = example.ns
    with ns.Handle() as h:
        layer = example.ExpertLayer(h.value, hidden=256, intermediate=384, experts=32, top_k=7, seed=4)
        x = torch.randn(70, 256, device="cuda").bfloat16()
        many, _ = layer.forward(x)
        for t in (0, 33, 69):
            one, _ = layer.forward(x[t:t + 1].contiguous())
            # The router's FP32 product may add up in another order.
            assert rel(one[0].double().cpu().numpy(), many[t].double().cpu().numpy()) <= 2.0**-8
