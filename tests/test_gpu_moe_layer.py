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


def test_padding_tokens_change_nothing(example):
    """Masked tokens get zeros, leave every gradient as it was, and the rows
    that no expert has may hold anything."""
    ns = example.ns
    with ns.Handle() as h:
        layer = example.ExpertLayer(h.value, hidden=256, intermediate=128, experts=16, top_k=4, seed=6)
        x = torch.randn(50, 256, device="cuda").bfloat16()
        grad = torch.randn(50, 256, device="cuda").bfloat16()
        y, saved = layer.forward(x)
        gx = layer.backward(grad, saved)
        want = [g.clone() for g in layer.grads]
        # The same tokens with 14 padding tokens behind them; freed memory full of NaN.
        px = torch.cat([x, torch.full((14, 256), float("nan"), device="cuda", dtype=torch.bfloat16)])
        px[50:] = 1.0
        pg = torch.cat([grad, torch.zeros(14, 256, device="cuda", dtype=torch.bfloat16)])
        junk = [torch.full((64 * 4 * 256,), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(12)]
        del junk
        mask = (torch.arange(64, device="cuda") < 50).to(torch.uint8)
        py, psaved = layer.forward(px, mask)
        pgx = layer.backward(pg, psaved)
        ns.muon_last_device_error(h.value)
        assert torch.equal(py[50:], torch.zeros_like(py[50:]))
        assert torch.equal(py[:50], y) and torch.equal(pgx[:50], gx)
        assert torch.equal(layer.grads[0], want[0]) and torch.equal(layer.grads[1], want[1])


def test_in_a_graph(example):
    """The serving path captured and replayed on new input gives what eager calls give."""
    ns = example.ns
    with ns.Handle() as h:
        layer = example.ExpertLayer(h.value, hidden=256, intermediate=128, experts=16, top_k=4, seed=7)
        x = torch.randn(2000, 256, device="cuda").bfloat16()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            layer.forward(x)                 # grows the workspace, warms the router's product
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            y, _ = layer.forward(x)
        for seed in (1, 2):
            x.copy_(torch.randn(2000, 256, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").bfloat16())
            graph.replay()
            torch.cuda.synchronize()
            want, _ = layer.forward(x)
            # The router's FP32 product may run another kernel under capture.
            assert rel(y.double().cpu().numpy(), want.double().cpu().numpy()) <= 2.0**-7
        ns.muon_last_device_error(h.value)


def test_launches_are_counted(example):
    ns = example.ns
    with ns.Handle() as h:
        layer = example.ExpertLayer(h.value, hidden=64, intermediate=32, experts=4, top_k=2)
        x = torch.randn(9, 64, device="cuda").bfloat16()
        ns.muon_reset_kernel_stats(h.value)
        ns.muon_set_kernel_timing(h.value, True)
        y, saved = layer.forward(x)
        layer.backward(y, saved)
        ns.muon_set_kernel_timing(h.value, False)
        st = ns.muon_kernel_stats(h.value)
        want = dict(moe_route=2, moe_plan=1, moe_combine=3, fp8_quantize=8, fp8_product=4, fp8_wgrad=2)
        assert {k: st["launches"][k] for k in want} == want
        assert all(st["total_ms"][k] > 0 for k in want)


SCRIPT = """
import hashlib, importlib.util, sys, torch
spec = importlib.util.spec_from_file_location("m", "examples/moe_training_step.py")
m = importlib.util.module_from_spec(spec); spec.loader.exec_module(m)
with m.ns.Handle() as h:
    layer = m.ExpertLayer(h.value, hidden=272, intermediate=144, experts=8, top_k=3, seed=3)
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(900, 272, generator=g, device="cuda").bfloat16()
    y, saved = layer.forward(x)
    gx = layer.backward(y, saved)
    layer.step()
    m.ns.muon_last_device_error(h.value)
    d = hashlib.sha256()
    for t in [y, gx] + layer.grads + layer.weights:
        d.update(t.float().cpu().numpy().tobytes())
print("digest", d.hexdigest())
"""


def test_same_with_and_without_launch_chaining(example):
    """MUON_PDL=0 launches every kernel plainly: the same bits."""
    import subprocess
    import sys
    out = []
    for pdl in ("1", "0"):
        r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, env=dict(os.environ, MUON_PDL=pdl), capture_output=True,
                           text=True, timeout=600)
        assert r.returncode == 0, r.stderr
        out.append(r.stdout.split("digest ")[1].strip())
    assert out[0] == out[1]
