"""Grouping of routed tokens and the weighted sum back, against plain statements."""

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


def plan(ns, h, ids, experts, stream=None):
    n = ids.numel()
    o = torch.full((experts + 1,), -7, dtype=torch.int32, device="cuda")
    s = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    p = torch.full(tuple(ids.shape), -7, dtype=torch.int32, device="cuda")
    ns.muon_moe_plan(h, ids, o, s, p, stream=stream)
    return o, s, p


@pytest.mark.parametrize("n", [0, 1, 31, 1024, 1025, 2048, 2049, 4095, 4096, 4097, 8192, 50001, 131073, 300000])
@pytest.mark.parametrize("experts", [1, 7, 512, 1024])
def test_plan(ns, h, n, experts):
    rng = np.random.default_rng(n + experts)
    ids = rng.integers(0, experts, n).astype(np.int32)
    if n > 100:
        ids[rng.random(n) < 0.1] = -1
        ids[n // 2:n // 2 + 40] = 0
    o, s, p = plan(ns, h, torch.from_numpy(ids).cuda(), experts)
    for got, want in zip((o, s, p), ref.plan(ids, experts)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    ns.muon_last_device_error(h)


def test_plan_without_any_expert(ns, h):
    for n in (100, 6000):
        o, s, p = plan(ns, h, torch.full((n,), -1, dtype=torch.int32, device="cuda"), 16)
        assert (o == 0).all() and (s == -1).all() and (p == -1).all()


def test_plan_reports_bad_ids(ns, h):
    for n in (100, 6000):
        ids = torch.zeros(n, dtype=torch.int32, device="cuda")
        ids[5], ids[6] = 16, -9
        o, s, p = plan(ns, h, ids, 16)
        with pytest.raises(ns.MuonError) as ei:
            ns.muon_last_device_error(h)
        assert ei.value.status_name == "MUON_ERR_INVALID_ARG"
        assert int(o[-1]) == n - 2 and int(p[5]) == -1 and int(p[6]) == -1


def make(t, k, d, experts, seed, off=0.1):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(experts)[:k] for _ in range(t)]).astype(np.int32).reshape(t, k)
    ids[rng.random((t, k)) < off] = -1
    if t > 2:
        ids[1] = -1                      # a token without experts
    _, _, pos = ref.plan(ids, experts)
    pos = pos.reshape(t, k)
    y = torch.from_numpy(rng.normal(size=(t * k, d)).astype(np.float32)).cuda().bfloat16()
    y[int((ids >= 0).sum()):] = float("nan")   # rows that no slot has are not read
    w = torch.from_numpy(rng.normal(size=(t, k)).astype(np.float32)).cuda()
    w[torch.from_numpy(ids < 0).cuda()] = float("nan")
    return pos, torch.from_numpy(pos.astype(np.int32)).cuda(), y, w


SHAPES = [(1, 7, 4096, 512), (37, 2, 144, 8), (3, 1, 16, 4), (129, 8, 2064, 64), (20, 32, 48, 40), (5, 9, 8704, 10)]


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("t,k,d,experts", SHAPES)
def test_combine(ns, h, t, k, d, experts, weighted):
    pos, pos_d, y, w = make(t, k, d, experts, t + d)
    out = torch.full((t, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    ns.muon_moe_combine(h, y, pos_d, w if weighted else None, out)
    yf, live = y.double().cpu().numpy(), pos >= 0
    wf = np.where(live, w.double().cpu().numpy() if weighted else 1.0, 0.0)
    terms = np.where(live[..., None], yf[np.maximum(pos, 0)], 0.0) * wf[..., None]
    want, size = terms.sum(1), np.abs(terms).sum(1)
    # FP32 sums of k terms, then half an ulp of BF16.
    assert (np.abs(out.double().cpu().numpy() - want) <= np.abs(want) / 256 + k * 2.0**-23 * size).all()
    ns.muon_last_device_error(h)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("t,k,d,experts", SHAPES)
def test_combine_backward(ns, h, t, k, d, experts, weighted):
    pos, pos_d, y, w = make(t, k, d, experts, t + d + 1)
    g = torch.randn(t, d, device="cuda", dtype=torch.bfloat16)
    gy = torch.full_like(y, 5.0)
    gw = torch.full((t, k), float("nan"), device="cuda")
    ns.muon_moe_combine_backward(h, g, y, pos_d, w if weighted else None, gy, gw)
    live = pos >= 0
    gf, yf = g.double().cpu().numpy(), y.double().cpu().numpy()
    rows = np.where(live[..., None], yf[np.maximum(pos, 0)], 0.0)
    want = (rows * gf[:, None]).sum(2)
    tol = d * 2.0**-23 * np.abs(rows * gf[:, None]).sum(2)
    assert (np.abs(gw.double().cpu().numpy() - want) <= tol).all()
    wf = np.where(live, w.double().cpu().numpy() if weighted else 1.0, 0.0)
    want_y = np.full(tuple(y.shape), 5.0)                # rows without a slot keep what they hold
    want_y[pos[live]] = (gf[:, None] * wf[..., None])[live]
    assert (np.abs(gy.double().cpu().numpy() - want_y) <= np.abs(want_y) / 256).all()
    ns.muon_moe_combine_backward(h, g, None, pos_d, w if weighted else None, gy.fill_(5.0))
    assert (np.abs(gy.double().cpu().numpy() - want_y) <= np.abs(want_y) / 256).all()
    ns.muon_last_device_error(h)


def test_combine_gradient_against_differences(ns, h):
    """The directional derivative of sum(out * g) in 64 bits."""
    pos, pos_d, y, w = make(6, 3, 64, 8, 2, off=0.0)
    w = torch.where(torch.isnan(w), torch.zeros_like(w), w)
    y = torch.where(torch.isnan(y), torch.zeros_like(y), y)
    g = torch.randn(6, 64, device="cuda", dtype=torch.bfloat16)
    gy, gw = torch.zeros_like(y), torch.zeros_like(w)
    ns.muon_moe_combine_backward(h, g, y, pos_d, w, gy, gw)
    live = pos >= 0

    def value(yv, wv):
        return ((np.where(live[..., None], yv[np.maximum(pos, 0)], 0.0) * wv[..., None]).sum(1) * g.double().cpu().numpy()).sum()

    rng = np.random.default_rng(0)
    yv, wv = y.double().cpu().numpy(), w.double().cpu().numpy()
    dy, dw = rng.normal(size=yv.shape), rng.normal(size=wv.shape)
    e = 1e-6
    num = (value(yv + e * dy, wv + e * dw) - value(yv - e * dy, wv - e * dw)) / (2 * e)
    a, b = gy.double().cpu().numpy() * dy, gw.double().cpu().numpy() * dw
    # grad_y is held in BF16: 2^-9 of each term.
    assert abs(num - a.sum() - b.sum()) <= 2.0**-9 * np.abs(a).sum() + 1e-5 * np.abs(b).sum()


def test_bad_rows_are_reported(ns, h):
    y = torch.ones(4, 16, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([[0, 4], [-3, 1]], dtype=torch.int32, device="cuda")
    out = torch.empty(2, 16, dtype=torch.bfloat16, device="cuda")
    ns.muon_moe_combine(h, y, pos, None, out)
    assert (out == 1).all()
    with pytest.raises(ns.MuonError):
        ns.muon_last_device_error(h)


def test_rows_past_32_bit_offsets(ns, h):
    """Rows that start past 2^31 elements."""
    d, rows = 65536, 33000
    y = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    y[32990] = torch.arange(d, device="cuda") % 128
    y[3] = 1
    pos = torch.tensor([[32990, 3]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 2.0]], device="cuda")
    out = torch.empty(1, d, dtype=torch.bfloat16, device="cuda")
    ns.muon_moe_combine(h, y, pos, w, out)
    want = (torch.arange(d, device="cuda") % 128) * 0.5 + 2
    assert torch.equal(out[0].float(), want)
    gy = torch.zeros_like(y)
    ns.muon_moe_combine_backward(h, out, None, pos, w, gy)
    assert torch.equal(gy[32990].float(), want * 0.5) and torch.equal(gy[3].float(), want * 2)


def test_plan_on_another_stream_is_the_same(ns, h):
    ids = torch.randint(0, 64, (20000,), dtype=torch.int32, device="cuda")
    a = plan(ns, h, ids, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = plan(ns, h, ids, 64, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals(ns, h):
    y = torch.zeros(8, 24, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ns.MuonError):            # hidden not a multiple of 16
        ns.muon_moe_combine(h, y, pos, None, torch.zeros(4, 24, dtype=torch.bfloat16, device="cuda"))
    y = torch.zeros(8, 32, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ns.MuonError):            # out over y
        ns.muon_moe_combine(h, y, pos, None, y[:4])
    with pytest.raises(ValueError):
        ns.muon_moe_combine(h, y.float(), pos, None, y[:4])
    with pytest.raises(ValueError):
        ns.muon_moe_combine(h, y, pos, torch.zeros(4, 3, device="cuda"), y[:4])
    wide = torch.zeros(4, 33, dtype=torch.int32, device="cuda")
    with pytest.raises(ns.MuonError):            # too many choices
        ns.muon_moe_combine(h, y, wide, None, torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda"))
    ids = torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(ns.MuonError):            # outputs over one another
        ns.muon_moe_plan(h, ids, torch.zeros(17, dtype=torch.int32, device="cuda"), ids, torch.zeros_like(ids))
    with pytest.raises(ns.MuonError):            # too many experts
        ns.muon_moe_plan(h, ids, torch.zeros(1026, dtype=torch.int32, device="cuda"), torch.zeros_like(ids), torch.zeros_like(ids))
    with pytest.raises(ValueError):              # y of another shape than its gradient
        ns.muon_moe_combine_backward(h, torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda"), y[:4], pos, None,
                                     torch.zeros(8, 32, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 2, device="cuda"))
