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
