"""Routing to experts and its backward pass against the 64-bit statement."""

import numpy as np
import pytest

from tests import moe_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_03_gb300 as m
    return m


@pytest.fixture(scope="module")
def h(ns):
    with ns.Handle() as handle:
        yield handle.value


def run(ns, h, x, k, bias=None, mask=None, softmax=False, renorm=True, scale=1.0, **kw):
    t = x.shape[0]
    ids = torch.full((t, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((t, k), float("nan"), device="cuda")
    ns.muon_moe_route(h, x, ids, w, score=ns.SCORE_SOFTMAX if softmax else ns.SCORE_SIGMOID, bias=bias, mask=mask,
                      renormalize=renorm, scale=scale, **kw)
    return ids.cpu().numpy(), w.double().cpu().numpy()


CASES = [
    # tokens, experts, k, softmax, bias, groups, top_groups, group_top, renorm
    (1, 512, 7, False, True, 1, 1, 1, True),
    (5, 512, 7, True, False, 1, 1, 1, True),
    (33, 64, 1, True, False, 1, 1, 1, False),
    (129, 8, 8, False, False, 1, 1, 1, True),
    (257, 96, 4, False, True, 4, 2, 2, True),
    (64, 1000, 32, False, True, 8, 8, 1, False),
    (64, 1024, 16, True, True, 32, 5, 2, True),
    (77, 7, 3, True, False, 7, 4, 1, True),
    (50, 33, 5, False, False, 3, 1, 2, False),
    (31, 1, 1, True, False, 1, 1, 1, False),
    (40, 510, 6, True, False, 6, 2, 1, False),
]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("case", CASES)
def test_route(ns, h, case, dtype):
    t, e, k, softmax, with_bias, groups, top_groups, group_top, renorm = case
    g = torch.Generator("cuda").manual_seed(t * 1000 + e)
    x = (torch.randn(t, e, generator=g, device="cuda") * 2).to(getattr(torch, dtype))
    bias = torch.randn(e, generator=g, device="cuda") * 0.1 if with_bias else None
    ids, w = run(ns, h, x, k, bias, softmax=softmax, renorm=renorm, scale=1.7, groups=groups, top_groups=top_groups,
                 group_top=group_top)
    x64 = x.double().cpu().numpy()
    want, _, c = ref.route(x64, k, softmax=softmax, bias=None if bias is None else bias.double().cpu().numpy(),
                           groups=groups, top_groups=top_groups, group_top=group_top, renorm=renorm)
    # Choice values are at most about 1.5 and computed in FP32 to a few ulp
    # (exp 2, division 1, sums of up to 1024 terms and of two values): where
    # the choice differs from 64 bits, the two values lie within 2e-6.
    assert (ids >= 0).all() and (np.sort(ids, 1)[:, 1:] != np.sort(ids, 1)[:, :-1]).all()
    diff = ids != want
    if diff.any():
        full = ref.choice_values(x64, softmax, None if bias is None else bias.double().cpu().numpy(), group_top,
                                 softmax and bias is None and (group_top == 1 or groups == 1))
        a, b = np.take_along_axis(full, ids, 1), np.take_along_axis(full, want, 1)
        if groups == 1:
            assert np.abs(a - b)[diff].max() <= 2e-6
        else:
            # A near-tie of two groups replaces whole groups: rows may differ,
            # but not many of them.
            assert diff.any(1).mean() <= 0.02
    # Weights of the choice made: exp, division and two sums in FP32.
    np.testing.assert_allclose(w, ref.weights_of(x64, ids, softmax=softmax, renorm=renorm, scale=1.7), rtol=3e-6, atol=1e-30)
    ns.muon_last_device_error(h)


def test_ties_go_to_the_lowest_expert(ns, h):
    """Small whole logits: equal scores are equal in FP32 too, and the choice is exact."""
    g = torch.Generator("cuda").manual_seed(5)
    for e, groups, top in ((512, 1, 1), (96, 8, 3), (7, 1, 1)):
        x = torch.randint(-2, 3, (200, e), generator=g, device="cuda").float()
        x[0] = 1.0
        x[1, :] = 0.0
        x[1, ::2] = -0.0
        for softmax in (False, True):
            ids, _ = run(ns, h, x, 5, softmax=softmax, groups=groups, top_groups=top)
            want, _, _ = ref.route(x.double().cpu().numpy() + 0.0, 5, softmax=softmax, groups=groups, top_groups=top)
            np.testing.assert_array_equal(ids, want)


def test_masked_tokens_and_closed_experts(ns, h):
    g = torch.Generator("cuda").manual_seed(6)
    t, e, k = 40, 64, 6
    x = torch.randn(t, e, generator=g, device="cuda")
    x[0] = float("-inf")                     # nothing open
    x[1, 3:] = float("-inf")                 # three open, six wanted
    x[2] = torch.finfo(torch.float32).min    # the type's lowest value is a value
    x[3, 10:] = torch.finfo(torch.float32).min
    mask = torch.ones(t, dtype=torch.uint8, device="cuda")
    mask[7] = 0
    mask[39] = 0
    x[7] = float("nan")                      # not looked at
    for softmax in (False, True):
        for groups, top in ((1, 1), (8, 2)):
            ids, w = run(ns, h, x, k, mask=mask, softmax=softmax, groups=groups, top_groups=top)
            x64 = x.double().cpu().numpy()
            x64[7] = 0.0
            want, ww, _ = ref.route(x64, k, softmax=softmax, mask=mask.cpu().numpy(), groups=groups, top_groups=top)
            np.testing.assert_array_equal(ids, want)
            assert (ids[0] == -1).all() and (ids[7] == -1).all() and (ids[1, 3:] == -1).all()
            np.testing.assert_allclose(w, ww, rtol=3e-6, atol=1e-30)
            assert np.isfinite(w).all() and (w[ids < 0] == 0).all()
    ns.muon_last_device_error(h)


@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_nonfinite_logits_are_reported_and_closed(ns, h, bad):
    x = torch.randn(9, 32, device="cuda")
    x[4, 8] = float(bad)
    for softmax in (False, True):
        ids, w = run(ns, h, x, 4, softmax=softmax)
        assert not (ids[4] == 8).any() and np.isfinite(w).all()
        with pytest.raises(ns.MuonError) as ei:
            ns.muon_last_device_error(h)
        assert ei.value.status_name == "MUON_ERR_NONFINITE"
        ns.muon_last_device_error(h)         # reading it clears it


def test_large_logits_have_finite_weights(ns, h):
    """Scores that underflow or saturate: no NaN, renormalised or not."""
    x = torch.full((4, 16), -200.0, device="cuda")
    x[1] = 200.0
    x[2, :8] = 3e38
    x[3, 0] = -3e38
    for softmax in (False, True):
        for renorm in (False, True):
            ids, w = run(ns, h, x, 3, softmax=softmax, renorm=renorm)
            assert np.isfinite(w).all()
            np.testing.assert_allclose(w, ref.weights_of(np.maximum(x.double().cpu().numpy(), -700), ids, softmax=softmax,
                                                         renorm=renorm, scale=1.0) * (w != 0), rtol=3e-6, atol=1e-30)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("t,e,k", [(1, 512, 7), (65, 96, 4), (30, 7, 3), (20, 1000, 32), (3, 1, 1)])
def test_route_backward(ns, h, dtype, softmax, renorm, t, e, k):
    g = torch.Generator("cuda").manual_seed(e + k)
    x = (torch.randn(t, e, generator=g, device="cuda") * 2).to(getattr(torch, dtype))
    if t > 2 and e > 8:
        x[1, 2:9] = float("-inf")
    ids, _ = run(ns, h, x, k, softmax=softmax, renorm=renorm, scale=2.5)
    if t > 2:
        ids[2] = -1
    grad = torch.randn(t, k, generator=g, device="cuda")
    out = torch.full((t, e), float("nan"), dtype=x.dtype, device="cuda")
    ns.muon_moe_route_backward(h, x, torch.from_numpy(ids).cuda(), grad, out,
                               score=ns.SCORE_SOFTMAX if softmax else ns.SCORE_SIGMOID, renormalize=renorm, scale=2.5)
    want = ref.route_backward(x.double().cpu().numpy(), ids, grad.double().cpu().numpy(), softmax=softmax, renorm=renorm, scale=2.5)
    got = out.double().cpu().numpy()
    # FP32: a few ulp of each term, whose differences may cancel: terms are at
    # most scale |g| times a score.  BF16 adds half an ulp, 2^-9.
    size = 2.5 * np.abs(grad.cpu().numpy()).max(1, keepdims=True)
    if renorm and not softmax:
        # Terms carry 1 / S, with S the chosen sigmoids' sum.
        p = ref.weights_of(x.double().cpu().numpy(), ids, softmax=False, renorm=False, scale=1.0).sum(1, keepdims=True)
        size = size / np.where(p > 0, np.minimum(p, 1.0), 1.0)
    tol = 4e-6 * size + (np.abs(want) / 256 if dtype == "bfloat16" else 0.0)
    assert (np.abs(got - want) <= tol).all()
    ns.muon_last_device_error(h)


@pytest.mark.parametrize("softmax", [False, True])
def test_a_single_renormalised_choice_has_no_gradient(ns, h, softmax):
    """Its weight is `scale` whatever the logits are."""
    x = torch.randn(500, 64, device="cuda") * 3
    for k in (1, 3):
        ids = torch.full((500, k), -1, dtype=torch.int32, device="cuda")
        ids[:, k - 1] = torch.randint(0, 64, (500,), dtype=torch.int32, device="cuda")
        out = torch.full_like(x, float("nan"))
        ns.muon_moe_route_backward(h, x, ids, torch.randn(500, k, device="cuda"), out,
                                   score=ns.SCORE_SOFTMAX if softmax else ns.SCORE_SIGMOID, scale=1.5)
        assert (out == 0).all()


def test_backward_of_a_bad_id_is_reported(ns, h):
    x = torch.randn(2, 16, device="cuda")
    ids = torch.tensor([[0, 16], [3, -2]], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    ns.muon_moe_route_backward(h, x, ids, torch.ones(2, 2, device="cuda"), out)
    with pytest.raises(ns.MuonError) as ei:
        ns.muon_last_device_error(h)
    assert ei.value.status_name == "MUON_ERR_INVALID_ARG"
    assert torch.isfinite(out).all()


def test_another_stream_and_no_tokens(ns, h):
    x = torch.randn(300, 128, device="cuda")
    ids = torch.empty(300, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(300, 4, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ns.muon_moe_route(h, x, ids, w, stream=s)
    s.synchronize()
    want, _, _ = ref.route(x.double().cpu().numpy(), 4, softmax=False)
    assert (ids.cpu().numpy() == want).mean() > 0.999
    ns.muon_moe_route(h, x[:0], ids[:0], w[:0])


@pytest.mark.parametrize("kw,experts,k", [
    (dict(groups=3), 32, 4), (dict(groups=33), 66, 4), (dict(groups=4, top_groups=5), 32, 4), (dict(groups=0), 32, 4),
    (dict(groups=8, top_groups=1), 32, 5), (dict(group_top=3), 32, 4), (dict(score=9), 32, 4), (dict(scale=float("nan")), 32, 4),
    (dict(), 1025, 4), (dict(), 64, 33), (dict(), 4, 5),
])
def test_refusals(ns, h, kw, experts, k):
    x = torch.zeros(2, experts, device="cuda")
    ids = torch.zeros(2, k, dtype=torch.int32, device="cuda")
    w = torch.zeros(2, k, device="cuda")
    with pytest.raises(ns.MuonError) as ei:
        ns.muon_moe_route(h, x, ids, w, **kw)
    assert ei.value.status_name == "MUON_ERR_INVALID_ARG"


def test_binding_refusals(ns, h):
    x = torch.zeros(4, 32, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    for bad in (dict(logits=x.half()), dict(ids=ids.long()), dict(weights=w.double()), dict(logits=x.t().contiguous().t()),
                dict(weights=w[:, :1].contiguous()), dict(bias=torch.zeros(31, device="cuda")), dict(logits=x.cpu()),
                dict(mask=torch.ones(4, device="cuda"))):
        kw = dict(dict(logits=x, ids=ids, weights=w), **bad)
        with pytest.raises(ValueError):
            ns.muon_moe_route(h, kw.pop("logits"), kw.pop("ids"), kw.pop("weights"), **kw)
    with pytest.raises(ns.MuonError):
        ns.muon_moe_route(h, x.view(-1)[1:].clone().as_strided((1, 32), (32, 1), 1), ids[:1], w[:1])  # not 16-byte aligned


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("k", [2, 5])
def test_small_scores_have_finite_gradients(ns, h, dtype, k):
    """All chosen sigmoids between 1e-39 and 1e-30, gradients up to a loss
    scale's: the renormalised weights are ordinary, and so is their gradient."""
    t, e, scale = 400, 64, 2.5
    g = torch.Generator("cuda").manual_seed(k)
    x = (-70.0 - 18.5 * torch.rand(t, e, generator=g, device="cuda")).to(getattr(torch, dtype))
    x[0], x[1] = -88.5, -80.0
    ids, w = run(ns, h, x, k, scale=scale)
    x64 = x.double().cpu().numpy()
    # A score is off by 2 ulp of the exponential, half an ulp of the sum, of the
    # reciprocal and of the subnormal result (2^-149 of 3.7e-39): 6e-7; a weight by
    # two scores', the sum's and the division's: 1.5e-6.
    share = ref.weights_of(x64, ids, softmax=False, renorm=True, scale=1.0)
    np.testing.assert_allclose(w, scale * share, rtol=3e-6)
    grad = torch.randn(t, k, generator=g, device="cuda")
    grad[1::2] *= 2e4
    out = torch.full((t, e), float("nan"), dtype=x.dtype, device="cuda")
    ns.muon_moe_route_backward(h, x, torch.from_numpy(ids).cuda(), grad, out, scale=scale)
    got, want = out.double().cpu().numpy(), ref.route_backward(x64, ids, grad.double().cpu().numpy(), softmax=False,
                                                               renorm=True, scale=scale)
    assert np.isfinite(got).all() and np.abs(want).max() > 1e3
    # dx = w (g - <g, w>) (1 - s): the weight's 1.5e-6 of a difference of up to
    # twice the largest gradient, and the sum's 2e-6 of it; BF16 adds half an ulp.
    full = np.zeros_like(want)
    np.put_along_axis(full, ids.astype(np.int64), share, 1)
    tol = 8e-6 * scale * np.abs(grad.double().cpu().numpy()).max(1, keepdims=True) * full
    assert (np.abs(got - want) <= tol + (np.abs(want) / 256 if dtype == "bfloat16" else 0.0)).all()
    ns.muon_last_device_error(h)
