"""Grouped FP8 products against 64-bit sums of the values that the bytes stand for."""

import numpy as np
import pytest

from tests import moe_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_03_gb300 as m
    return m


@pytest.fixture(scope="module")
def h(ns):
    with ns.Handle() as handle:
        yield handle.value


def fp8(shape, g):
    return (torch.randn(shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(F8)


def scales(shape, g):
    return torch.randint(117, 137, shape, generator=g, device="cuda", dtype=torch.uint8)


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def product_case(counts, n, k, seed, extra_rows=0):
    g = torch.Generator("cuda").manual_seed(seed)
    off = offsets_of(counts)
    r, e = int(off[-1]) + extra_rows, len(counts)
    x, w = fp8((r, k), g), fp8((e, n, k), g)
    xs, ws = scales((r, -(-k // 128)), g), scales((e, -(-n // 128), -(-k // 128)), g)
    return off, x, xs, w, ws


def exact_product(off, x, xs, w, ws):
    """(y, sum of magnitudes) in 64 bits."""
    xv = ref.rows_values(x.float().double().cpu().numpy(), xs.cpu().numpy())
    n = w.shape[1]
    y, size = np.zeros((x.shape[0], n)), np.zeros((x.shape[0], n))
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if a < b:
            wv = ref.rows_values(w[e].float().double().cpu().numpy(), np.repeat(ws[e].cpu().numpy(), 128, 0)[:n])
            y[a:b] = xv[a:b] @ wv.T
            size[a:b] = np.abs(xv[a:b]) @ np.abs(wv).T
    return y, size


# The sums are held in 32 bits or more by the tensor cores, each step adding 32
# products: K / 32 + 32 roundings or truncations of at most 2^-23 of the sum of
# magnitudes.  BF16 adds half an ulp, 2^-9 of the value.
def tolerance(k):
    return (k / 32 + 32) * 2.0**-23


COUNTS = [
    [1], [5], [31, 33], [224], [225, 0, 1], [0, 0, 0, 7], [64, 96, 160, 192, 449], [1000], [0] * 100 + [2] * 50 + [0] * 362,
]


@pytest.mark.parametrize("n,k", [(256, 128), (16, 16), (272, 144), (528, 1040), (1536, 512)])
@pytest.mark.parametrize("counts", COUNTS)
def test_product(ns, h, counts, n, k):
    if len(counts) > 100 and n > 300:
        n, k = 48, 272
    off, x, xs, w, ws = product_case(counts, n, k, n + k + len(counts), extra_rows=3)
    y = torch.full((x.shape[0], n), 123.0, dtype=torch.bfloat16, device="cuda")
    ns.muon_fp8_grouped_matmul(h, x, xs, w, ws, torch.from_numpy(off).cuda(), y)
    want, size = exact_product(off, x, xs, w, ws)
    got = y.double().cpu().numpy()
    r = off[-1]
    assert (np.abs(got - want)[:r] <= (np.abs(want) / 256 + tolerance(k) * size)[:r]).all()
    assert (got[r:] == 123.0).all()          # rows of no expert are not written
    ns.muon_last_device_error(h)


@pytest.mark.parametrize("byte", [0x7F, 0xFF])
def test_other_rows_do_not_matter(ns, h, byte):
    """NaN in rows of no expert, and in other experts' rows, reach no result."""
    off, x, xs, w, ws = product_case([40, 70], 272, 400, 3, extra_rows=9)
    d_off = torch.from_numpy(off).cuda()
    y = torch.empty(x.shape[0], 272, dtype=torch.bfloat16, device="cuda")
    ns.muon_fp8_grouped_matmul(h, x, xs, w, ws, d_off, y)
    keep = y.clone()
    x.view(torch.uint8)[110:] = byte
    xs[110:] = 255
    x.view(torch.uint8)[:40] = byte
    w.view(torch.uint8)[0] = byte
    ns.muon_fp8_grouped_matmul(h, x, xs, w, ws, d_off, y)
    assert torch.equal(y[40:110], keep[40:110])
    assert torch.isnan(y[:40]).all()


def test_extreme_scales(ns, h):
    """Scale bytes at both ends, whose product stays in range."""
    off, x, xs, w, ws = product_case([33], 128, 256, 8)
    xs[:, 0], ws[:, :, 0] = 1, 253
    xs[:, 1], ws[:, :, 1] = 250, 4
    y = torch.empty(33, 128, dtype=torch.bfloat16, device="cuda")
    ns.muon_fp8_grouped_matmul(h, x, xs, w, ws, torch.from_numpy(off).cuda(), y)
    want, size = exact_product(off, x, xs, w, ws)
    assert (np.abs(y.double().cpu().numpy() - want) <= np.abs(want) / 256 + tolerance(256) * size).all()


def test_product_is_the_same_each_time_and_on_another_stream(ns, h):
    off, x, xs, w, ws = product_case([300, 5, 77, 0, 200], 784, 656, 1)
    d_off = torch.from_numpy(off).cuda()
    ys = [torch.empty(x.shape[0], 784, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for y, stream in zip(ys, (None, None, s)):
        ns.muon_fp8_grouped_matmul(h, x, xs, w, ws, d_off, y, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_rows_past_32_bit_offsets(ns, h):
    """Operands and results past 2^31 elements."""
    r, k, n = 530000, 4096, 16
    g = torch.Generator("cuda").manual_seed(2)
    x = fp8((64, k), g).view(torch.uint8).repeat(r // 64 + 1, 1)[:r].view(F8)
    xs = scales((64, 32), g).repeat(r // 64 + 1, 1)[:r].contiguous()
    w, ws = fp8((2, n, k), g), scales((2, 1, 32), g)
    off = torch.tensor([0, 100, r], dtype=torch.int32, device="cuda")
    y = torch.empty(r, n, dtype=torch.bfloat16, device="cuda")
    ns.muon_fp8_grouped_matmul(h, x, xs, w, ws, off, y)
    at = [0, 99, 100, 300000, r - 1]
    for row in at:
        e = 0 if row < 100 else 1
        want, size = exact_product([0, 1], x[row:row + 1], xs[row:row + 1], w[e:e + 1], ws[e:e + 1])
        got = y[row].double().cpu().numpy()
        assert (np.abs(got - want[0]) <= np.abs(want[0]) / 256 + tolerance(k) * size[0]).all()
    # Equal rows of one expert have equal results, wherever they are.
    assert torch.equal(y[128:128 + 64], y[r // 64 * 64 - 64:r // 64 * 64])


def test_bad_offsets_are_reported(ns, h):
    """Offsets past the rows, negative or falling: nothing outside is written."""
    _, x, xs, w, ws = product_case([50], 64, 128, 4)
    w, ws = w.repeat_interleave(3, 0), ws.repeat_interleave(3, 0)
    whole = torch.full((52, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    for off in ([0, 10, 20, 60], [-5, 10, 20, 50], [0, 30, 20, 50], [0, 10, 2000000000, 50]):
        ns.muon_fp8_grouped_matmul(h, x, xs, w, ws, torch.tensor(off, dtype=torch.int32, device="cuda"), whole[:50])
        with pytest.raises(ns.MuonError) as ei:
            ns.muon_last_device_error(h)
        assert ei.value.status_name == "MUON_ERR_INVALID_ARG"
        assert (whole[50:] == 9.0).all()


def wild_offsets(experts, top):
    """Offsets that no plan makes: falling, negative, past every buffer, rows counted many times."""
    i = torch.arange(experts + 1)
    big = 2**31 - 1
    return [torch.where(i % 2 == 0, 0, top), torch.where(i % 2 == 0, 0, big), torch.where(i % 2 == 0, -big, big),
            torch.where(i % 2 == 0, top, 0), i * (big // (experts + 1)), torch.where(i % 3 == 0, big, i)]


@pytest.mark.parametrize("experts", [8, 600, 1024])
def test_wild_offsets_stay_inside(ns, h, experts):
    """Whatever offsets holds: an error, and not a byte outside the rows."""
    r, n, k = 700, 48, 144
    g = torch.Generator("cuda").manual_seed(1)
    x, xs = fp8((r, k), g), scales((r, 2), g)
    w, ws = fp8((experts, n, k), g), scales((experts, 1, 2), g)
    whole = torch.full((r + 64, n), 9.0, dtype=torch.bfloat16, device="cuda")
    for off in wild_offsets(experts, r):
        ns.muon_fp8_grouped_matmul(h, x, xs, w, ws, off.int().cuda(), whole[32:r + 32])
        with pytest.raises(ns.MuonError) as ei:
            ns.muon_last_device_error(h)
        assert ei.value.status_name == "MUON_ERR_INVALID_ARG"
        assert (whole[:32] == 9.0).all() and (whole[r + 32:] == 9.0).all()


# ------------------------------------------------------------------ weight gradient
def wgrad_case(ns, counts, n, k, seed, extra=0):
    g = torch.Generator("cuda").manual_seed(seed)
    off = offsets_of(counts)
    cap = max(128, ns.muon_fp8_cols_capacity(int(off[-1]), len(counts))) + extra
    starts = ref.padded_starts(off)
    live = np.zeros(cap, dtype=bool)
    for e in range(len(counts)):
        live[starts[e]:starts[e] + counts[e]] = True
    used = np.zeros(cap, dtype=bool)
    used[:starts[-1]] = ref.written_columns(off)
    out = []
    for rows in (n, k):
        q = fp8((rows, cap), g)
        q.view(torch.uint8)[:, torch.from_numpy(~live).cuda()] = 0
        q.view(torch.uint8)[:, torch.from_numpy(~used).cuda()] = 0x7F   # never written: NaN must reach nothing
        out += [q, scales((cap // 128, rows), g)]
    return off, starts, out


def exact_wgrad(off, starts, yt, ys, xt, xs):
    a = ref.cols_values(yt.float().double().cpu().numpy(), ys.cpu().numpy())
    b = ref.cols_values(xt.float().double().cpu().numpy(), xs.cpu().numpy())
    e = len(off) - 1
    dw = np.zeros((e, a.shape[0], b.shape[0]))
    size = np.zeros_like(dw)
    for i in range(e):
        s = slice(starts[i], starts[i] + off[i + 1] - off[i])
        dw[i] = a[:, s] @ b[:, s].T
        size[i] = np.abs(a[:, s]) @ np.abs(b[:, s]).T
    return dw, size


@pytest.mark.parametrize("n,k", [(256, 192), (16, 16), (272, 208), (144, 1040)])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 129, 128], [700], [2] * 40 + [0] * 10, [0, 0]])
def test_wgrad(ns, h, counts, n, k):
    off, starts, (yt, ys, xt, xs) = wgrad_case(ns, counts, n, k, n + k)
    d_off = torch.from_numpy(off).cuda()
    dw = torch.full((len(counts), n, k), float("nan"), device="cuda")
    ns.muon_fp8_grouped_wgrad(h, yt, ys, xt, xs, d_off, dw)
    want, size = exact_wgrad(off, starts, yt, ys, xt, xs)
    tol = tolerance(max(counts) + 128) * size
    got = dw.double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all()       # experts without rows: exact zeros
    again = torch.empty_like(dw)
    ns.muon_fp8_grouped_wgrad(h, yt, ys, xt, xs, d_off, again)
    assert torch.equal(dw, again)
    # Added to what is there: one more rounding to FP32.
    base = torch.randn_like(dw)
    acc = base.clone()
    ns.muon_fp8_grouped_wgrad(h, yt, ys, xt, xs, d_off, acc, accumulate=True)
    assert torch.equal(acc, base + dw)
    ns.muon_last_device_error(h)


def test_wgrad_capacity_too_small_is_reported(ns, h):
    off, starts, (yt, ys, xt, xs) = wgrad_case(ns, [200, 10], 64, 64, 1)
    cut = [v[:, :256].contiguous() if v.dtype == F8 else v[:2].contiguous() for v in (yt, ys, xt, xs)]
    dw = torch.empty(2, 64, 64, device="cuda")
    ns.muon_fp8_grouped_wgrad(h, *cut, torch.from_numpy(off).cuda(), dw)
    with pytest.raises(ns.MuonError) as ei:
        ns.muon_last_device_error(h)
    assert ei.value.status_name == "MUON_ERR_INVALID_ARG"


@pytest.mark.parametrize("experts", [8, 600, 1024])
def test_wgrad_wild_offsets_stay_inside(ns, h, experts):
    n, k, cap = 64, 80, 1024
    g = torch.Generator("cuda").manual_seed(1)
    ops = [fp8((n, cap), g), scales((cap // 128, n), g), fp8((k, cap), g), scales((cap // 128, k), g)]
    whole = torch.full((experts + 2, n, k), 9.0, device="cuda")
    for off in wild_offsets(experts, 700):
        ns.muon_fp8_grouped_wgrad(h, *ops, off.int().cuda(), whole[1:experts + 1])
        with pytest.raises(ns.MuonError) as ei:
            ns.muon_last_device_error(h)
        assert ei.value.status_name == "MUON_ERR_INVALID_ARG"
        assert (whole[0] == 9.0).all() and (whole[-1] == 9.0).all()


def test_quantised_gradient_against_differences(ns, h):
    """dY^T X of quantised operands is the derivative of sum(dY * (X W^T)) by W, taken on the quantised values."""
    counts, n, k = [37, 0, 20], 48, 32
    off = offsets_of(counts)
    r = int(off[-1])
    g = torch.Generator("cuda").manual_seed(0)
    dy = torch.randn(r, n, generator=g, device="cuda").bfloat16()
    x = torch.randn(r, k, generator=g, device="cuda").bfloat16()
    cap = ns.muon_fp8_cols_capacity(r, 3)
    d_off = torch.from_numpy(off).cuda()
    ops = []
    for t, d in ((dy, n), (x, k)):
        q = torch.zeros(d, cap, dtype=torch.uint8, device="cuda").view(F8)
        s = torch.zeros(cap // 128, d, dtype=torch.uint8, device="cuda")
        ns.muon_fp8_quantize_cols(h, t, d_off, q, s)
        ops += [q, s]
    dw = torch.empty(3, n, k, device="cuda")
    ns.muon_fp8_grouped_wgrad(h, *ops, d_off, dw)
    starts = ref.padded_starts(off)
    dyv, xv = (ref.cols_values(q.float().double().cpu().numpy(), s.cpu().numpy()) for q, s in (ops[:2], ops[2:]))
    rng = np.random.default_rng(1)
    w, d = rng.normal(size=(3, n, k)), rng.normal(size=(3, n, k))

    def value(wv):
        total = 0.0
        for e in range(3):
            s = slice(starts[e], starts[e] + counts[e])
            total += ((wv[e] @ xv[:, s]) * dyv[:, s]).sum()
        return total

    eps = 1e-4
    num = (value(w + eps * d) - value(w - eps * d)) / (2 * eps)
    a = dw.double().cpu().numpy() * d
    assert abs(num - a.sum()) <= 1e-6 * np.abs(a).sum()


def test_refusals(ns, h):
    def call(r=4, e=2, n=32, k=32, offs=3, **bad):
        t = dict(x=torch.zeros(r, k, dtype=torch.uint8, device="cuda"), xs=torch.zeros(r, -(-k // 128), dtype=torch.uint8, device="cuda"),
                 w=torch.zeros(e, n, k, dtype=torch.uint8, device="cuda"),
                 ws=torch.zeros(e, -(-n // 128), -(-k // 128), dtype=torch.uint8, device="cuda"),
                 off=torch.zeros(offs, dtype=torch.int32, device="cuda"), y=torch.zeros(r, n, dtype=torch.bfloat16, device="cuda"))
        t.update(bad)
        ns.muon_fp8_grouped_matmul(h, *(t[i] for i in ("x", "xs", "w", "ws", "off", "y")))

    call()
    for kw in (dict(n=24), dict(k=24), dict(e=1025, offs=1026)):
        with pytest.raises(ns.MuonError) as ei:
            call(**kw)
        assert ei.value.status_name == "MUON_ERR_INVALID_ARG"
    for kw in (dict(offs=2), dict(y=torch.zeros(4, 32, device="cuda")), dict(x=torch.zeros(4, 32, device="cuda")),
               dict(ws=torch.zeros(2, 1, 2, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    call(r=0)                                   # no rows: nothing to do
