"""FP8 quantisation against the plain statement: every byte is determined."""

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


def values(rows, d, seed):
    """BF16 values over many scales, with zero blocks, exact limits and single large values."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, d, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-40, 40, (rows, 1), generator=g, device="cuda").float())
    x = x.bfloat16()
    if rows > 4:
        x[0] = 0
        x[1] = 0
        x[1, -1] = 448.0                       # the largest value: scale 1
        x[2, :16] = 450.0                      # just above: scale 2
        x[3] = 1e-38                           # near the smallest normal value
        x[4, ::3] = -3.0e38
    return x


def host(t):
    return t.float().double().cpu().numpy()


def q_of(t):
    return t.float().double().cpu().numpy()


@pytest.mark.parametrize("rows,d", [(1, 4096), (7, 16), (33, 144), (300, 1040), (5, 8704)])
def test_rows(ns, h, rows, d):
    x = values(rows, d, rows + d)
    q = torch.empty(rows, d, dtype=F8, device="cuda")
    s = torch.empty(rows, -(-d // 128), dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_rows(h, x, q, s)
    want, ws = ref.quantize_rows(host(x))
    np.testing.assert_array_equal(s.cpu().numpy(), ws)
    np.testing.assert_array_equal(q_of(q), want)
    ns.muon_last_device_error(h)


def test_rows_past_the_last_expert_are_left_alone(ns, h):
    x = values(40, 272, 9)
    x[25:] = float("nan")
    off = torch.tensor([0, 3, 25], dtype=torch.int32, device="cuda")
    q = torch.full((40, 272), 9.0, device="cuda").to(F8)
    s = torch.full((40, 3), 200, dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_rows(h, x, q, s, offsets=off)
    ns.muon_last_device_error(h)
    want, ws = ref.quantize_rows(host(x[:25]))
    np.testing.assert_array_equal(q_of(q)[:25], want)
    np.testing.assert_array_equal(s.cpu().numpy()[:25], ws)
    assert (q_of(q)[25:] == 9.0).all() and (s[25:] == 200).all()


@pytest.mark.parametrize("t,k,d", [(9, 3, 272), (1, 7, 4096), (65, 2, 16)])
def test_rows_sent_to_experts(ns, h, t, k, d):
    x = values(t, d, t)
    rng = np.random.default_rng(t)
    pos = rng.permutation(t * k).reshape(t, k).astype(np.int32)
    pos[rng.random((t, k)) < 0.2] = -1
    r = t * k
    q = torch.full((r, d), 9.0, device="cuda").to(F8)
    s = torch.full((r, -(-d // 128)), 200, dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_rows(h, x, q, s, pos=torch.from_numpy(pos).cuda())
    a, b = ref.quantize_rows(host(x))
    want, ws = np.full((r, d), 9.0), np.full(s.shape, 200)
    live = pos >= 0
    want[pos[live]] = np.repeat(a[:, None], k, 1)[live]
    ws[pos[live]] = np.repeat(b[:, None], k, 1)[live]
    np.testing.assert_array_equal(q_of(q), want)
    np.testing.assert_array_equal(s.cpu().numpy(), ws)
    ns.muon_last_device_error(h)
    pos[0, 0] = r
    ns.muon_fp8_quantize_rows(h, x, q, s, pos=torch.from_numpy(pos).cuda())
    with pytest.raises(ns.MuonError) as ei:
        ns.muon_last_device_error(h)
    assert ei.value.status_name == "MUON_ERR_INVALID_ARG"


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("e,n,k", [(1, 128, 128), (3, 16, 16), (2, 272, 400), (1, 2048, 144), (4, 144, 1536)])
def test_blocks(ns, h, dtype, e, n, k):
    g = torch.Generator("cuda").manual_seed(n + k)
    w = torch.randn(e, n, k, generator=g, device="cuda") * 0.02
    w[0, :16, :16] = 0
    w[-1, -1, -1] = 1e30
    w = w.to(getattr(torch, dtype))
    nb, kb = -(-n // 128), -(-k // 128)
    q = torch.empty(e, n, k, dtype=F8, device="cuda")
    s = torch.empty(e, nb, kb, dtype=torch.uint8, device="cuda")
    qt = torch.empty(e, k, n, dtype=F8, device="cuda")
    st = torch.empty(e, kb, nb, dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_blocks(h, w, q, s, qt, st)
    want, ws = ref.quantize_blocks(w.double().cpu().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), ws)
    np.testing.assert_array_equal(st.cpu().numpy(), ws.transpose(0, 2, 1))
    np.testing.assert_array_equal(q_of(q), want)
    np.testing.assert_array_equal(q_of(qt), want.transpose(0, 2, 1))
    q2, s2, qt2, st2 = (torch.empty_like(v) for v in (q, s, qt, st))
    ns.muon_fp8_quantize_blocks(h, w, q2, s2)
    ns.muon_fp8_quantize_blocks(h, w, qt=qt2, scales_t=st2)
    for a, b in ((q, q2), (s, s2), (qt, qt2), (st, st2)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    ns.muon_last_device_error(h)


def counts_to_offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


@pytest.mark.parametrize("counts,d", [
    ([1], 16), ([0, 0, 5, 0], 144), ([128, 1, 127, 129, 0, 300], 272), ([0] * 500 + [3] + [0] * 11, 128), ([2] * 1024, 48),
])
def test_cols(ns, h, counts, d):
    off = counts_to_offsets(counts)
    rows = int(off[-1])
    x = values(rows, d, rows)
    cap = ns.muon_fp8_cols_capacity(rows, len(counts)) + 128
    qt = torch.full((d, cap), 3.0, device="cuda").to(F8)
    s = torch.full((cap // 128, d), 7, dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_cols(h, x, torch.from_numpy(off).cuda(), qt, s)
    want, ws = ref.quantize_cols(host(x), off)
    used = want.shape[1]
    written = ref.written_columns(off)
    got = q_of(qt)
    np.testing.assert_array_equal(got[:, :used][:, written], want[:, written])
    np.testing.assert_array_equal(s.cpu().numpy()[:used // 128], ws)
    assert (got[:, :used][:, ~written] == 3.0).all()
    assert (got[:, used:] == 3.0).all() and (s.cpu().numpy()[used // 128:] == 7).all()
    ns.muon_last_device_error(h)


def test_cols_gathered(ns, h):
    t, k, d, e = 50, 3, 208, 8
    rng = np.random.default_rng(4)
    ids = np.stack([rng.permutation(e)[:k] for _ in range(t)])
    ids[rng.random((t, k)) < 0.2] = -1
    off, slots, _ = ref.plan(ids, e)
    x = values(t, d, 1)
    cap = ns.muon_fp8_cols_capacity(t * k, e)
    qt = torch.zeros(d, cap, dtype=torch.uint8, device="cuda").view(F8)
    s = torch.zeros(cap // 128, d, dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_cols(h, x, torch.from_numpy(off.astype(np.int32)).cuda(), qt, s,
                              slots=torch.from_numpy(slots.astype(np.int32)).cuda(), top_k=k)
    want, ws = ref.quantize_cols(host(x)[slots[:off[-1]] // k], off)
    used = want.shape[1]
    np.testing.assert_array_equal(q_of(qt)[:, :used], want)
    np.testing.assert_array_equal(s.cpu().numpy()[:used // 128], ws)
    ns.muon_last_device_error(h)


def test_too_short_a_buffer_is_reported(ns, h):
    off = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    x = torch.ones(3, 16, dtype=torch.bfloat16, device="cuda")
    qt = torch.zeros(16, 256, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2, 16, dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_cols(h, x, off, qt, s)
    with pytest.raises(ns.MuonError) as ei:
        ns.muon_last_device_error(h)
    assert ei.value.status_name == "MUON_ERR_INVALID_ARG"
    assert (s[:, 0] == 127 - 8).all()


@pytest.mark.parametrize("experts", [8, 600, 1024])
def test_wild_offsets_stay_inside(ns, h, experts):
    """Whatever offsets and slots hold: an error, and not a byte outside the buffers."""
    i = torch.arange(experts + 1)
    big = 2**31 - 1
    x = torch.randn(50, 144, device="cuda").bfloat16()
    slots = torch.randint(-5, 200, (150,), dtype=torch.int32, device="cuda")
    qt = torch.full((146, 1024), 0x11, dtype=torch.uint8, device="cuda")
    s = torch.full((10, 144), 0x22, dtype=torch.uint8, device="cuda")
    for off in (torch.where(i % 2 == 0, 0, 150), torch.where(i % 2 == 0, 0, big), torch.where(i % 2 == 0, -big, big),
                torch.where(i % 2 == 0, 150, 0), i * (big // (experts + 1)), torch.where(i % 3 == 0, big, i)):
        for sl in (None, slots):
            ns.muon_fp8_quantize_cols(h, x, off.int().cuda(), qt[1:145], s[1:9], slots=sl, top_k=3)
            with pytest.raises(ns.MuonError) as ei:
                ns.muon_last_device_error(h)
            assert ei.value.status_name == "MUON_ERR_INVALID_ARG"
            assert (qt[0] == 0x11).all() and (qt[145] == 0x11).all() and (s[0] == 0x22).all() and (s[9] == 0x22).all()


@pytest.mark.parametrize("bad,byte", [(float("nan"), 0x7F), (float("inf"), 0x7E)])
def test_nonfinite_values(ns, h, bad, byte):
    """NaN stays NaN, an infinity saturates; both are reported."""
    x = torch.ones(2, 256, dtype=torch.bfloat16, device="cuda")
    x[0, 5] = bad
    q = torch.empty(2, 256, dtype=torch.uint8, device="cuda")
    s = torch.empty(2, 2, dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_rows(h, x, q, s)
    with pytest.raises(ns.MuonError) as ei:
        ns.muon_last_device_error(h)
    assert ei.value.status_name == "MUON_ERR_NONFINITE"
    assert int(q[0, 5]) & 0x7F == byte
    assert int(s[0, 1]) == 127 - 8 and (q[0, 128:] == q[1, 0]).all()   # other blocks as ever
    if byte == 0x7F:
        assert int(s[0, 0]) == 127 - 8


def finite_reference(x):
    """Each value with NaN as zero and infinities as the largest BF16: what sets the scales."""
    return np.nan_to_num(x, nan=0.0, posinf=3.3895314e38, neginf=-3.3895314e38)


def test_nonfinite_columns(ns, h):
    """One NaN, one infinity: their own columns' bytes, every scale and all other bytes as ever."""
    off = np.array([0, 40, 40, 200], dtype=np.int32)
    x = values(200, 272, 5)
    x[3, 7] = float("nan")
    x[199, 8] = float("inf")
    x[60, 271] = float("-inf")
    x[61, 271] = float("nan")
    cap = ns.muon_fp8_cols_capacity(200, 3)
    qt = torch.zeros(272, cap, dtype=torch.uint8, device="cuda")
    s = torch.zeros(cap // 128, 272, dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_cols(h, x, torch.from_numpy(off).cuda(), qt, s)
    with pytest.raises(ns.MuonError) as ei:
        ns.muon_last_device_error(h)
    assert ei.value.status_name == "MUON_ERR_NONFINITE"
    want, ws = ref.quantize_cols(finite_reference(host(x)), off)
    used, written = want.shape[1], ref.written_columns(off)
    np.testing.assert_array_equal(s.cpu().numpy()[:used // 128], ws)
    got, bytes_ = q_of(qt.view(F8))[:, :used], qt.cpu().numpy()
    ok = np.tile(written, (272, 1))
    starts = ref.padded_starts(off)
    for row, col, byte in ((3, 7, 0x7F), (199, 8, 0x7E), (60, 271, 0xFE), (61, 271, 0x7F)):
        e = 0 if row < 40 else 2
        at = starts[e] + row - off[e]
        assert bytes_[col, at] & (0x7F if byte == 0x7F else 0xFF) == byte
        ok[col, at] = False
    np.testing.assert_array_equal(got[ok], want[ok])


def test_nonfinite_weights(ns, h):
    w = torch.randn(2, 144, 272, device="cuda")
    w[1, 130, 3] = float("nan")
    w[0, 5, 200] = float("-inf")
    q = torch.empty(2, 144, 272, dtype=torch.uint8, device="cuda")
    s = torch.empty(2, 2, 3, dtype=torch.uint8, device="cuda")
    qt = torch.empty(2, 272, 144, dtype=torch.uint8, device="cuda")
    st = torch.empty(2, 3, 2, dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_blocks(h, w, q, s, qt, st)
    with pytest.raises(ns.MuonError) as ei:
        ns.muon_last_device_error(h)
    assert ei.value.status_name == "MUON_ERR_NONFINITE"
    want, ws = ref.quantize_blocks(np.nan_to_num(w.double().cpu().numpy(), nan=0.0, neginf=-3.4028234e38))
    np.testing.assert_array_equal(s.cpu().numpy(), ws)
    assert int(q[1, 130, 3]) & 0x7F == 0x7F and int(q[0, 5, 200]) == 0xFE
    assert torch.equal(qt, q.transpose(1, 2)) and torch.equal(st, s.transpose(1, 2))
    got = q_of(q.view(F8))
    ok = np.ones_like(want, dtype=bool)
    ok[1, 130, 3] = ok[0, 5, 200] = False
    np.testing.assert_array_equal(got[ok], want[ok])


def test_subnormal_values(ns, h):
    w = torch.zeros(1, 128, 128, device="cuda")
    w[0, 3, 4] = 2.0 ** -140
    w[0, 5, 6] = -(2.0 ** -133)
    q = torch.empty(1, 128, 128, dtype=F8, device="cuda")
    s = torch.empty(1, 1, 1, dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_blocks(h, w, q, s)
    want, ws = ref.quantize_blocks(w.double().cpu().numpy())
    assert int(s) == int(ws[0, 0, 0]) == 0
    np.testing.assert_array_equal(q_of(q), want)


def test_more_than_32_bits_of_values(ns, h):
    """A row buffer past 2^31 values: the last rows are right."""
    rows, d = 33000, 65536
    q = torch.empty(rows, d, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, d // 128, dtype=torch.uint8, device="cuda")
    x = torch.randn(2, d, device="cuda", dtype=torch.bfloat16)
    pos = torch.tensor([[rows - 1], [0]], dtype=torch.int32, device="cuda")
    ns.muon_fp8_quantize_rows(h, x, q, s, pos=pos)
    want, ws = ref.quantize_rows(host(x))
    for i, r in ((0, rows - 1), (1, 0)):
        np.testing.assert_array_equal(q_of(q[r].view(F8)), want[i])
        np.testing.assert_array_equal(s[r].cpu().numpy(), ws[i])


def test_refusals(ns, h):
    x = torch.zeros(4, 24, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ns.MuonError):      # not a multiple of 16
        ns.muon_fp8_quantize_rows(h, x, torch.zeros(4, 24, dtype=torch.uint8, device="cuda"),
                                  torch.zeros(4, 1, dtype=torch.uint8, device="cuda"))
    w = torch.zeros(1, 16, 16, device="cuda")
    with pytest.raises(ns.MuonError):      # no output
        ns.muon_fp8_quantize_blocks(h, w)
    with pytest.raises(ns.MuonError):      # values without scales
        ns.muon_fp8_quantize_blocks(h, w, q=torch.zeros(1, 16, 16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ns.muon_fp8_quantize_blocks(h, w.half())
    x = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ns.MuonError):      # capacity
        ns.muon_fp8_quantize_cols(h, x, off, torch.zeros(32, 100, dtype=torch.uint8, device="cuda"),
                                  torch.zeros(0, 32, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ns.muon_fp8_quantize_rows(h, x.float(), torch.zeros(4, 32, dtype=torch.uint8, device="cuda"),
                                  torch.zeros(4, 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_nonfinite_weights_of_either_type(ns, h, dtype):
    """NaN and infinities in blocks of their own and together: the scale is the
    finite values', or the largest one where an infinity is; all else as ever."""
    w = (torch.randn(2, 272, 400, generator=torch.Generator("cuda").manual_seed(8), device="cuda") * 3).to(getattr(torch, dtype))
    places = [(0, 0, 0, "nan"), (0, 127, 127, "nan"), (0, 200, 140, "inf"), (0, 271, 399, "-inf"), (1, 5, 6, "nan"), (1, 7, 8, "-inf"),
              (1, 260, 300, "nan"), (1, 261, 303, "-nan")]
    for e, r, c, v in places:
        w[e, r, c] = float(v.replace("-nan", "nan")) * (-1 if v == "-nan" else 1)
    q, qt = torch.empty(2, 272, 400, dtype=torch.uint8, device="cuda"), torch.empty(2, 400, 272, dtype=torch.uint8, device="cuda")
    s, st = torch.empty(2, 3, 4, dtype=torch.uint8, device="cuda"), torch.empty(2, 4, 3, dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_blocks(h, w, q, s, qt, st)
    with pytest.raises(ns.MuonError) as ei:
        ns.muon_last_device_error(h)
    assert ei.value.status_name == "MUON_ERR_NONFINITE"
    want, ws = ref.quantize_blocks(finite_reference(w.double().cpu().numpy()))
    np.testing.assert_array_equal(s.cpu().numpy(), ws)
    assert torch.equal(qt, q.transpose(1, 2)) and torch.equal(st, s.transpose(1, 2))
    ok = np.ones(want.shape, dtype=bool)
    for e, r, c, v in places:
        ok[e, r, c] = False
        if v.endswith("nan"):
            assert int(q[e, r, c]) & 0x7F == 0x7F
        else:
            assert int(q[e, r, c]) == (0xFE if v == "-inf" else 0x7E)
    np.testing.assert_array_equal(q_of(q.view(F8))[ok], want[ok])
    # A block of nothing but NaN has no magnitude: scale 1.
    w = torch.full((1, 16, 16), float("nan"), dtype=w.dtype, device="cuda")
    q, s = torch.empty(1, 16, 16, dtype=torch.uint8, device="cuda"), torch.empty(1, 1, 1, dtype=torch.uint8, device="cuda")
    ns.muon_fp8_quantize_blocks(h, w, q, s)
    assert int(s) == 127 and ((q & 0x7F) == 0x7F).all()
    with pytest.raises(ns.MuonError):
        ns.muon_last_device_error(h)
