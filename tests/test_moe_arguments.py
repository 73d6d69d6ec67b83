"""Pointers and sizes of the expert layer's entry points that would reach past
a buffer: refused on the host, before anything is launched."""

import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_03_gb300 as m
    return m


@pytest.fixture(scope="module")
def h(ns):
    with ns.Handle() as handle:
        yield handle.value


def test_empty_offsets_are_refused(ns):
    """Their last element would be four bytes before the buffer."""
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="offsets must not be empty"):
        ns.muon_fp8_quantize_rows(1, x, q, s, offsets=torch.zeros(0, dtype=torch.int32))


@pytest.mark.gpu
def test_live_rows_are_checked(ns, h):
    """Aligned to four bytes and outside the outputs."""
    x = torch.ones(4, 32, dtype=torch.bfloat16, device="cuda")
    q, s = torch.zeros(4, 32, dtype=torch.uint8, device="cuda"), torch.zeros(64, dtype=torch.uint8, device="cuda")
    live = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
    fn = ns.load_library().muon_fp8_quantize_rows
    p = ctypes.c_void_p

    def call(at):
        return fn(h, 4, 32, p(x.data_ptr()), p(0), 0, 4, p(at), p(q.data_ptr()), p(s.data_ptr()), p(0))

    for at in (live.data_ptr() + 1, live.data_ptr() + 2, q.data_ptr() + 64, s.data_ptr()):
        assert call(at) == 1 and ns.muon_last_error_message()
    torch.cuda.synchronize()
    assert (q == 0).all()
    assert call(live.data_ptr() + 4) == 0          # the end of offsets is seldom 16-byte aligned
    torch.cuda.synchronize()
    assert (q[:2] != 0).all() and (q[2:] == 0).all()
    ns.muon_last_device_error(h)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,k", [(1 << 60, 16), (1 << 59, 32), (1 << 62, 4), ((1 << 63) - 1, 2), ((1 << 31) - (1 << 20) + 1, 1),
                                      (-1, 1), (-(1 << 62), 4)])
def test_token_counts_whose_slots_do_not_fit(ns, h, tokens, k):
    """tokens x top_k past 2^31 is refused, past 2^64 too (the product would
    come out as zero).  No buffer is behind the pointers: nothing is launched."""
    lib, p = ns.load_library(), ctypes.c_void_p
    a = [p(4096 * (i + 1)) for i in range(6)]
    opts = (ctypes.c_int32 * 6)(0, 1, 1, 1, 1, 0x3F800000)
    opts = ctypes.cast(opts, lib.muon_moe_route.argtypes[8])
    before = ns.muon_kernel_stats(h)["total_launches"]
    assert lib.muon_moe_route(h, tokens, 64, k, a[0], 0, p(0), p(0), opts, a[1], a[2], p(0)) == 1
    assert lib.muon_moe_route_backward(h, tokens, 64, k, a[0], 0, a[1], a[2], opts, a[3], p(0)) == 1
    assert lib.muon_moe_combine(h, tokens, k, 8, 32, a[0], a[1], p(0), a[2], p(0)) == 1
    assert lib.muon_moe_combine_backward(h, tokens, k, 8, 32, a[0], p(0), a[1], p(0), a[2], p(0), p(0)) == 1
    assert lib.muon_fp8_quantize_rows(h, tokens, 32, a[0], a[1], k, 8, p(0), a[2], a[3], p(0)) == 1
    assert "tokens out of range" in ns.muon_last_error_message()
    assert ns.muon_kernel_stats(h)["total_launches"] == before


@pytest.mark.gpu
def test_the_mask_is_not_an_output(ns, h):
    """A mask under ids or weights would be overwritten while others read it."""
    x = torch.randn(64, 32, device="cuda")
    ids, w = torch.zeros(64, 2, dtype=torch.int32, device="cuda"), torch.zeros(64, 2, device="cuda")
    for out in (ids, w):
        for first in (0, 7, 448):
            mask = out.view(torch.uint8).view(-1)[first:first + 64]
            with pytest.raises(ns.MuonError) as ei:
                ns.muon_moe_route(h, x, ids, w, mask=mask)
            assert ei.value.status_name == "MUON_ERR_INVALID_ARG"
    # A mask may start at any byte.
    mask = torch.ones(67, dtype=torch.uint8, device="cuda")
    mask[3] = 0
    ns.muon_moe_route(h, x, ids, w, mask=mask[3:])
    assert (ids[0] == -1).all() and (ids[1:] >= 0).all()
    ns.muon_last_device_error(h)


def test_offsets_do_not_go_with_pos(ns):
    """They count rows: as a count of tokens they would leave out the tokens
    past the number of rows, though these have rows of their own."""
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8)
    pos = torch.tensor([[-1], [-1], [-1], [0]], dtype=torch.int32)
    with pytest.raises(ValueError, match="do not go with pos"):
        ns.muon_fp8_quantize_rows(1, x, q, s, pos=pos, offsets=torch.tensor([0, 1], dtype=torch.int32))
