"""A captured grouping stays valid whatever the handle does after the capture."""

import numpy as np
import pytest

from tests import moe_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_03_gb300 as m
    return m


def buffers(n, experts):
    return [torch.empty(m, dtype=torch.int32, device="cuda") for m in (experts + 1, n, n)]


def random_ids(n, experts, seed):
    return torch.from_numpy(np.random.default_rng(seed).integers(-1, experts, n).astype(np.int32))


@pytest.mark.parametrize("grow", ["step", "plan", "both"])
def test_replay_after_the_handle_has_grown(ns, grow):
    """Captured with 8000 slots; then a step takes its workspace and a longer
    grouping takes scratch; then replayed on other ids."""
    n, experts = 8000, 512
    with ns.Handle() as h:
        ids, out = random_ids(n, experts, 0).cuda(), buffers(n, experts)
        ns.muon_moe_plan(h.value, ids, *out)              # takes the scratch
        torch.cuda.synchronize()
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=s):
            ns.muon_moe_plan(h.value, ids, *out)
        keep = []
        if grow in ("plan", "both"):
            # More than 2^20 slots: past what the first call took.
            m, e = 3 << 20, 1024
            ns.muon_moe_plan(h.value, torch.zeros(m, dtype=torch.int32, device="cuda"), *buffers(m, e))
            torch.cuda.synchronize()
        if grow in ("step", "both"):
            w, mo, g = (torch.randn(8, 512, 1024, device="cuda") for _ in range(3))
            ns.muon_step(h.value, [(512, 1024, 8)], [mo], [g], [w], 0.02, 0.0, 0.9)
            torch.cuda.synchronize()
        for seed in (1, 2):
            # What was freed meanwhile belongs to others, whose values must stay.
            keep.append(torch.full((1 << 20,), seed, dtype=torch.int32, device="cuda"))
            fresh = random_ids(n, experts, seed)
            ids.copy_(fresh)
            graph.replay()
            torch.cuda.synchronize()
            for got, want in zip(out, ref.plan(fresh.numpy(), experts)):
                np.testing.assert_array_equal(got.cpu().numpy(), want)
        assert all((k == i + 1).all() for i, k in enumerate(keep))
        ns.muon_last_device_error(h.value)


def test_the_example_steps_between_capture_and_replay(ns):
    """Serving captured on a handle that trains on: forward, capture, step, replay."""
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("moe_training_step", os.path.join(root, "examples", "moe_training_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    with ns.Handle() as h:
        layer = example.ExpertLayer(h.value, hidden=256, intermediate=128, experts=16, top_k=4, seed=9)
        x = torch.randn(2000, 256, generator=torch.Generator("cuda").manual_seed(3), device="cuda").bfloat16()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            layer.forward(x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            y, _ = layer.forward(x)
        out, saved = layer.forward(x)
        layer.backward(out, saved)
        layer.step()                                      # new weights and FP8 copies in place
        graph.replay()
        torch.cuda.synchronize()
        want, _ = layer.forward(x)
        a, b = y.double(), want.double()
        # The router's FP32 product may run another kernel under capture: two
        # roundings to BF16, and a choice on the edge in few tokens.
        assert float((a - b).norm() / b.norm()) <= 2.0**-7
        ns.muon_last_device_error(h.value)


def test_scratch_keeps_to_the_cap(ns):
    """workspace_bytes_max bounds what groupings take, all buffers together."""
    experts = 1024

    def call(h, n):
        ids, out = random_ids(n, experts, n).cuda(), buffers(n, experts)
        ns.muon_moe_plan(h.value, ids, *out)
        for got, want in zip(out, ref.plan(ids.cpu().numpy(), experts)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)

    # A chunk of 1024 slots takes a 4 KiB histogram here (up to 128 of them).
    with ns.Handle(workspace_bytes_max=40960) as h:
        call(h, 2048)                                     # no scratch
        call(h, 10 * 1024)                                # all of the cap
        with pytest.raises(ns.MuonError) as ei:
            call(h, 10 * 1024 + 1)
        assert ei.value.status_name == "MUON_ERR_NOMEM"
        call(h, 10 * 1024)                                # as before
    with ns.Handle(workspace_bytes_max=40960 - 1) as h:
        with pytest.raises(ns.MuonError) as ei:
            call(h, 10 * 1024)
        assert ei.value.status_name == "MUON_ERR_NOMEM"
    with ns.Handle(workspace_bytes_max=3 << 20) as h:
        call(h, 1 << 20)                                  # 512 KiB
        call(h, (1 << 20) + 1)                            # 1 MiB beside it
        with pytest.raises(ns.MuonError):
            call(h, 4 << 20)                              # 2 MiB are more than what is left
        call(h, 3 << 20)                                  # 1.5 MiB are not: all that is left


@pytest.mark.parametrize("stepped", [False, True])
def test_the_first_grouping_may_be_a_captured_one(ns, stepped):
    """Scratch is taken during the capture where the handle has none yet."""
    n, experts = 8000, 512
    with ns.Handle() as h:
        if stepped:
            w, mo, g = (torch.randn(2, 128, 256, device="cuda") for _ in range(3))
            ns.muon_step(h.value, [(128, 256, 2)], [mo], [g], [w], 0.02, 0.0, 0.9)
        ids, out = random_ids(n, experts, 0).cuda(), buffers(n, experts)
        torch.cuda.synchronize()
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=s):
            ns.muon_moe_plan(h.value, ids, *out)
        for seed in (1, 2):
            fresh = random_ids(n, experts, seed)
            ids.copy_(fresh)
            graph.replay()
            torch.cuda.synchronize()
            for got, want in zip(out, ref.plan(fresh.numpy(), experts)):
                np.testing.assert_array_equal(got.cpu().numpy(), want)
        ns.muon_last_device_error(h.value)
