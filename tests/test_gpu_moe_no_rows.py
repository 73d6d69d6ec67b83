"""No rows at all: the weight gradient, its operands, and a layer's step."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_03_gb300 as m
    return m


@pytest.fixture(scope="module")
def h(ns):
    with ns.Handle() as handle:
        yield handle.value


def operands(ns, h, rows, experts, n, k, offsets):
    """Columns of `rows` rows, at the capacity that the binding names."""
    cap = ns.muon_fp8_cols_capacity(rows, experts)
    out = []
    for d in (n, k):
        x = torch.ones(rows, d, dtype=torch.bfloat16, device="cuda")
        q = torch.empty(d, cap, dtype=torch.uint8, device="cuda")
        s = torch.empty(cap // 128, d, dtype=torch.uint8, device="cuda")
        ns.muon_fp8_quantize_cols(h, x, offsets, q, s)
        out += [q, s]
    return out


@pytest.mark.parametrize("experts,n,k", [(1, 16, 16), (3, 272, 240), (64, 48, 512)])
def test_wgrad_without_rows(ns, h, experts, n, k):
    off = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    ops = operands(ns, h, 0, experts, n, k, off)
    assert ops[0].shape == (n, 0) and ops[1].shape == (0, n)
    whole = torch.full((experts + 2, n, k), 7.0, device="cuda")
    ns.muon_fp8_grouped_wgrad(h, *ops, off, whole[1:-1], accumulate=True)
    assert (whole == 7.0).all()                  # nothing to add
    ns.muon_fp8_grouped_wgrad(h, *ops, off, whole[1:-1])
    assert (whole[1:-1] == 0).all() and (whole[0] == 7.0).all() and (whole[-1] == 7.0).all()
    ns.muon_last_device_error(h)


def test_rows_without_room_are_reported(ns, h):
    """Offsets with rows, buffers without a column: an error of both calls, and nothing loaded."""
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    x = torch.ones(5, 32, dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty(32, 0, dtype=torch.uint8, device="cuda"), torch.empty(0, 32, dtype=torch.uint8, device="cuda")
    dw = torch.full((2, 32, 32), 7.0, device="cuda")
    for call in (lambda: ns.muon_fp8_quantize_cols(h, x, off, q, s),
                 lambda: ns.muon_fp8_grouped_wgrad(h, q, s, q, s, off, dw)):
        call()
        with pytest.raises(ns.MuonError) as ei:
            ns.muon_last_device_error(h)
        assert ei.value.status_name == "MUON_ERR_INVALID_ARG"
    with pytest.raises(ns.MuonError):            # still a multiple of 128
        ns.muon_fp8_grouped_wgrad(h, *(torch.zeros(32, 64, dtype=torch.uint8, device="cuda"),
                                       torch.zeros(0, 32, dtype=torch.uint8, device="cuda")) * 2, off, dw)


def test_a_step_without_tokens(ns):
    """An empty micro-batch: empty outputs, gradients of zero."""
    spec = importlib.util.spec_from_file_location("moe_training_step", os.path.join(ROOT, "examples", "moe_training_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    with ns.Handle() as h:
        layer = example.ExpertLayer(h.value, hidden=64, intermediate=32, experts=4, top_k=2)
        for g in layer.grads:
            g.fill_(5.0)
        x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
        y, saved = layer.forward(x)
        gx = layer.backward(y, saved)
        ns.muon_last_device_error(h.value)
        assert y.shape == gx.shape == (0, 64)
        assert all((g == 0).all() for g in layer.grads)
