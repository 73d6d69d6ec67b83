"""The 64-bit statements the GPU tests compare with, checked by themselves:
gradients against differences, the FP8 rounding against PyTorch's."""

import numpy as np
import pytest

from tests import moe_reference as ref


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(softmax, renorm):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(6, 20)) * 2
    x[1, 4] = -np.inf
    grad = rng.normal(size=(6, 5))
    ids, _, _ = ref.route(x, 5, softmax=softmax, renorm=renorm)
    ids[2, 3:] = -1
    ids[3] = -1
    got = ref.route_backward(x, ids, grad, softmax=softmax, renorm=renorm, scale=2.5)

    def value(y):
        return (ref.weights_of(y, ids, softmax=softmax, renorm=renorm, scale=2.5) * grad).sum(1)

    h = 1e-5
    for e in range(20):
        up, dn = x.copy(), x.copy()
        up[:, e] += h
        dn[:, e] -= h
        # Central differences: error about h^2 and rounding 1e-16 / h.
        np.testing.assert_allclose(got[:, e], (value(up) - value(dn)) / (2 * h), atol=1e-8)


def test_e4m3_rounding_matches_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 20000), rng.normal(size=20000) * 0.02,
                        np.ldexp(np.arange(-448, 449) + 0.5, -9), [0.0, 448.0, -448.0]]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(ref.e4m3(v), want.astype(np.float64))


def test_scale_is_the_least_power_of_two():
    rng = np.random.default_rng(1)
    m = np.exp(rng.uniform(-60, 60, 5000))
    m = np.concatenate([m, np.ldexp(448.0, np.arange(-40, 41)), np.ldexp(np.nextafter(448.0, 500.0), np.arange(-40, 41))])
    e = ref.exponent(m)
    assert (m / np.ldexp(1.0, e) <= 448).all()
    assert (m / np.ldexp(1.0, e - 1) > 448).all()
    assert ref.exponent(np.zeros(1))[0] == 0


def test_binding_refuses_wrong_tensors():
    """Shapes and types are checked before the library is asked."""
    torch = pytest.importorskip("torch")
    import newton_schulz_03_gb300 as ns
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    w = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ns.muon_moe_route(1, x, ids, w)
    with pytest.raises(ValueError, match="logits must be"):
        ns.muon_moe_route(1, x.half(), ids, w)
    with pytest.raises(ValueError, match="4 rows"):
        ns.muon_fp8_quantize_rows(1, x, torch.zeros(5, 32, dtype=torch.uint8), torch.zeros(5, 1, dtype=torch.uint8))


@pytest.mark.parametrize("rows,experts", [(0, 8), (1, 8), (7, 512), (128, 1), (1000, 8), (57337, 512)])
def test_column_capacity_holds_any_routing(rows, experts):
    import newton_schulz_03_gb300 as ns
    cap = ns.muon_fp8_cols_capacity(rows, experts)
    assert cap % 128 == 0
    # The worst routing: one row over a multiple of 128 on as many experts as can be.
    counts = np.zeros(experts, dtype=np.int64)
    left = rows
    for e in range(experts):
        if left > 0:
            counts[e] = 1
            left -= 1
    counts[0] += left
    assert (-(-counts // 128)).sum() * 128 <= cap


def test_null_handle_is_refused():
    """Every entry point of the layer checks its handle before anything else."""
    import newton_schulz_03_gb300 as ns
    from newton_schulz_03_gb300 import _native
    lib = ns.load_library()
    names = [n for n in ns.EXPORTED if n.startswith(("muon_moe_", "muon_fp8_"))]
    assert len(names) == 10
    for name in names:
        fn = getattr(lib, name)
        args = [None if t in (_native.ctypes.c_void_p,) or hasattr(t, "contents") else 0 for t in fn.argtypes]
        assert fn(*args) == 1, name                  # MUON_ERR_INVALID_ARG
        assert "handle" in ns.muon_last_error_message()
