"""Waits of the streamed losses that run out: the blocks' warps leave together, nothing is
written but rows that were complete, the call is reported and the next one is right."""

import time

import pytest

from tests.test_gpu_loss import failure, logits_of, targets_of

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF16, FP32 = torch.bfloat16, torch.float32
LOGITS, TARGETS = 1, 2


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_03_gb300 as m
    return m


@pytest.fixture(scope="module")
def h(ns):
    with ns.Handle() as handle:
        yield handle.value


def call(ns, h, kind, z, teacher, ids, w, mask):
    """The gradient in a wider buffer of 9, filled with 5, and the other outputs."""
    t, v = z.shape
    wide = torch.full((t, v + 16), 9.0, dtype=z.dtype, device="cuda")
    grad = wide[:, 8:8 + v]
    grad.fill_(5.0)
    outs = [torch.full((t,), 7.0, device="cuda") for _ in range(2 + (kind == "policy"))]
    how = dict(mask=mask, grad_loss=w, grad_logits=grad)
    if kind == "distill":
        ns.muon_distill_loss(h, z, teacher, ids, *outs, **how)
    else:
        ns.muon_policy_loss(h, z, ids[:, 0].contiguous(), w, *outs, **how)
    return wide, grad, outs


# Two rows and more for every block; short rows in their order, several blocks per SM, and
# long rows behind a mask, ranked first.
@pytest.mark.parametrize("kind,what,tokens,vocab,dtype,masked", [
    ("distill", LOGITS, 1700, 301, BF16, False), ("distill", TARGETS, 700, 32003, BF16, True),
    ("policy", TARGETS, 1700, 301, FP32, True), ("policy", LOGITS, 400, 70001, BF16, True)])
def test_a_wait_runs_out(ns, h, kind, what, tokens, vocab, dtype, masked):
    z, g = logits_of(tokens, vocab, dtype, 31)
    teacher, ids = targets_of(tokens, vocab, 40, g)
    ids[:, 0] = torch.randint(0, vocab, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(tokens, generator=g, device="cuda") + 0.5
    mask = (torch.arange(tokens, device="cuda") % 16 != 3).to(torch.uint8) if masked else None
    wide, clean, outs = call(ns, h, kind, z, teacher, ids, w, mask)
    ns.muon_last_device_error(h)
    ns.muon_selftest_loss_wait(h, what)
    began = time.perf_counter()
    wide2, grad, outs2 = call(ns, h, kind, z, teacher, ids, w, mask)
    assert failure(ns, h) == "MUON_ERR_TIMEOUT"
    assert time.perf_counter() - began < 15.0
    done, untouched = (grad == clean).all(1), (grad == 5.0).all(1)
    assert bool((done ^ untouched).all())
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert int(done.sum()) >= sms and int(untouched.sum()) >= 8
    for a, b in zip(outs2, outs):
        assert torch.equal(a[done], b[done]) and bool((a[untouched] == 7.0).all())
    assert bool((wide2[:, :8] == 9.0).all()) and bool((wide2[:, 8 + vocab:] == 9.0).all())
    # The next call is an ordinary one.
    _, again, outs3 = call(ns, h, kind, z, teacher, ids, w, mask)
    ns.muon_last_device_error(h)
    assert torch.equal(again, clean) and all(torch.equal(*p) for p in zip(outs3, outs))


def test_a_call_of_few_rows_takes_it_off(ns, h):
    z, g = logits_of(5, 301, FP32, 32)
    teacher, ids = targets_of(5, 301, 3, g)
    w = torch.ones(5, device="cuda")
    want = call(ns, h, "distill", z, teacher, ids, w, None)
    ns.muon_selftest_loss_wait(h, LOGITS)
    got = call(ns, h, "distill", z, teacher, ids, w, None)
    assert torch.equal(got[0], want[0])
    z, g = logits_of(1700, 301, FP32, 33)
    teacher, ids = targets_of(1700, 301, 3, g)
    call(ns, h, "distill", z, teacher, ids, torch.ones(1700, device="cuda"), None)
    ns.muon_last_device_error(h)


def test_refusals(ns, h):
    for bad in (0, 3, -1):
        with pytest.raises(ns.MuonError) as ei:
            ns.muon_selftest_loss_wait(h, bad)
        assert ei.value.status_name == "MUON_ERR_INVALID_ARG"
    with pytest.raises(ns.MuonError):
        ns.muon_selftest_loss_wait(0, LOGITS)
