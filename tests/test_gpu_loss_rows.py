"""Every element of every row of the streamed losses, against the calls that take one row
to a block; rows that have no softmax; buffers side by side."""

import numpy as np
import pytest

from tests import loss_reference as ref
from tests.test_gpu_loss import STEP, failure, logits_of, pieces_of, policy_case, refused, run_distill, run_policy, targets_of

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF16, FP32 = torch.bfloat16, torch.float32
U = ref.U


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_03_gb300 as m
    return m


@pytest.fixture(scope="module")
def h(ns):
    with ns.Handle() as handle:
        yield handle.value


def compare(a, b, z, temperature, dense, sparse, at):
    """Gradients a and b within twice of what either may be off by the formula: of any
    element a rounding, the value of the gap to the row's largest (5 U of it) and of its
    sum (ref.q_tol), and ``dense`` q by the row's factor; at the elements ``at`` [rows,
    targets] (-1: none), whose terms cancel, ``sparse`` [rows] more."""
    v = z.shape[1]
    for i in range(0, z.shape[0], 256):
        rows = slice(i, min(i + 256, z.shape[0]))
        x, y, zz = a[rows].double(), b[rows].double(), z[rows].double() / temperature
        top = zz.amax(1, keepdim=True)
        lse = torch.logsumexp(zz, 1, keepdim=True)
        most = max(float(lse.abs().max()), float(top.abs().max()))
        # (lse_tol and q_tol grow with |lse| and |top|: their largest here)
        rel = (top - zz) * 5 * U + 2.0**-22 + ref.lse_tol(v, most, most, pieces_of(v, z.dtype)) + 8 * U * most + 6 * U
        tol = y.abs() * (2 * STEP[z.dtype] + 2 * rel) + 2 * dense[rows, None].double() * torch.exp(zz - lse) + 2.0**-124
        if at is not None:
            ids = at[rows].long()
            tol.scatter_add_(1, ids.clamp(min=0), torch.where(ids >= 0, sparse[rows, None].double(), 0.0).expand(ids.shape))
        assert bool(((x - y).abs() <= tol).all()), i


# Rings of 2, 4, 8 and 16 warps, kept whole and in part.
SIZES = [(1700, 5, BF16), (3300, 333, FP32), (1521, 4099, FP32), (930, 9001, BF16), (609, 50257, BF16), (340, 50257, FP32),
         (309, 131072, BF16)]


@pytest.mark.parametrize("tokens,vocab,dtype", SIZES)
def test_every_element_of_the_distillation(ns, h, tokens, vocab, dtype):
    z, g = logits_of(tokens, vocab, dtype, vocab + 1)
    teacher, ids = targets_of(tokens, vocab, 20, g)
    ids[::9] = -1
    mask = torch.rand(tokens, generator=g, device="cuda") < 0.8 if tokens % 2 else None
    w = torch.randn(tokens, generator=g, device="cuda")
    how = dict(temperature=1.5, scale=2.0, mask=mask)
    grads = [torch.full_like(z, torch.nan) for _ in range(2)]
    for mode, grad in zip(("both", "two"), grads):
        run_distill(ns, h, z, teacher, ids, mode, grad, grad_loss=w, **how)
        assert not bool(torch.isnan(grad).any())
    coef = (w * 2.0 / 1.5).abs()
    # The targets' weights: distill_grad_tol's, for 20 of them whose logits are a few
    # units apart, within 250 U of at most 1, in each call.
    compare(*grads, z, 1.5, torch.zeros_like(w), coef * 512 * U, ids)
    out = (ids < 0).all(1) if mask is None else (ids < 0).all(1) | ~mask
    assert bool((grads[0][out] == 0).all()) and bool((grads[0][~out] != 0).any(1).all())
    ns.muon_last_device_error(h)


@pytest.mark.parametrize("tokens,vocab,dtype", SIZES)
def test_every_element_of_the_policy_loss(ns, h, tokens, vocab, dtype):
    z, actions, adv, old, refp, g = policy_case(tokens, vocab, dtype, vocab + 2, 1.0)
    mask = torch.rand(tokens, generator=g, device="cuda") < 0.8 if tokens % 2 else None
    w = torch.randn(tokens, generator=g, device="cuda")
    how = dict(temperature=1.0, kl_coef=0.1, mask=mask)
    grads = [torch.full_like(z, torch.nan) for _ in range(2)]
    for mode, grad in zip(("both", "two"), grads):
        logp = run_policy(ns, h, z, actions, adv, old, refp, mode, grad, grad_loss=w, **how)[1]
        assert not bool(torch.isnan(grad).any())
    # Slopes of either call: policy_tols's, by the largest error of a log probability.
    n = pieces_of(vocab, dtype)
    e_lp = ref.sum_tol(vocab, n) + 6 * U * (2 * float(logp.abs().max()) + np.log(vocab))
    slope = (adv.abs() * torch.exp(logp - old) + 0.1 * torch.exp(refp - logp)) * (e_lp + 12 * U + 2.0**-22)
    live = actions >= 0 if mask is None else (actions >= 0) & mask
    slope = torch.where(live, slope, 0.0)
    compare(*grads, z, 1.0, w.abs() * slope, 2 * w.abs() * (slope + 4 * U * adv.abs()), actions[:, None])
    assert bool((grads[0][~live] == 0).all())
    ns.muon_last_device_error(h)


@pytest.mark.parametrize("tokens", [6, 700])
def test_rows_without_a_softmax(ns, h, tokens):
    """-inf alone, or +inf among the logits: loss, log probability, lse and gradient are NaN."""
    z, g = logits_of(tokens, 20001, BF16, 41)
    teacher, ids = targets_of(tokens, 20001, 3, g)
    ids[:, 0] = 7
    z[1], z[4, 5] = -torch.inf, torch.inf
    w = torch.ones(tokens, device="cuda")
    good = torch.ones(tokens, dtype=torch.bool, device="cuda")
    good[[1, 4]] = False
    for mode in ("both", "two"):
        for run, rest in ((run_distill, (teacher, ids)), (run_policy, (ids[:, 0].contiguous(), w, -9.0 * w, None))):
            grad = torch.zeros_like(z)
            outs = run(ns, h, z, *rest, mode, grad, grad_loss=w)
            assert failure(ns, h) == "MUON_ERR_NONFINITE"
            for o in outs + (grad,):
                assert bool(torch.isnan(o[~good]).all()) and bool(torch.isfinite(o[good]).all())


def test_rows_between_rows_are_refused(ns, h):
    """A pitched buffer counts from its first element to its last: a gradient in the gaps
    of the logits' pitch is an overlap."""
    z, g = logits_of(6, 200, FP32, 42)
    teacher, ids = targets_of(6, 100, 3, g)
    loss, lse, w = (torch.ones(6, device="cuda") for _ in range(3))
    refused(ns, lambda: ns.muon_distill_loss(h, z[:, :100], teacher, ids, loss, lse, grad_loss=w, grad_logits=z[:, 100:]), "overlaps")
    refused(ns, lambda: ns.muon_policy_loss(h, z[:, :100], ids[:, 0].contiguous(), w, loss, torch.ones(6, device="cuda"), lse,
                                            grad_loss=lse.clone(), grad_logits=z[:, 100:]), "overlaps")


def test_equal_ids_take_no_longer_than_others(ns, h):
    """A thousand targets per row on a few entries, on one, and on entries a power of two
    apart, in many rows: the time of a thousand different ones, not that of their pairs."""
    t, v, k = 700, 20000, 1000
    z, g = logits_of(t, v, BF16, 43)
    teacher = torch.randn(t, k, generator=g, device="cuda")
    apart = torch.rand(t, v, generator=g, device="cuda").argsort(1)[:, :k].int()
    few = torch.randint(0, 5, (t, k), generator=g, device="cuda", dtype=torch.int32)
    w, grad = torch.rand(t, generator=g, device="cuda"), torch.empty_like(z)
    outs = [torch.empty(t, device="cuda") for _ in range(2)]

    def took(ids):
        best = float("inf")
        for _ in range(4):
            began, ended = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            began.record()
            ns.muon_distill_loss(h, z, teacher, ids, *outs, grad_loss=w, grad_logits=grad)
            ended.record()
            ended.synchronize()
            best = min(best, began.elapsed_time(ended))
        return best

    usual = took(apart)
    for ids in (few, torch.full_like(few, 7), apart // 256 * 256):
        assert took(ids.contiguous()) <= 4 * usual
    ns.muon_last_device_error(h)
