"""The choice of expert groups near its ties: what a group may be passed over
for, and by how little, against the 64-bit values."""

import numpy as np
import pytest

from tests import moe_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# A sigmoid is off by 2 ulp of the exponential times s (1 - s), half an ulp of
# the sum and of the reciprocal: below 2e-7; a choice value by half an ulp of 1.5
# more, 2.5e-7; the sum of two by both and half an ulp of 3, 6.2e-7; the
# difference of two groups by twice that.
BOUND = 2e-6


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_03_gb300 as m
    return m


@pytest.fixture(scope="module")
def h(ns):
    with ns.Handle() as handle:
        yield handle.value


def route(ns, h, x, k, bias, groups, top_groups, group_top):
    ids = torch.full((x.shape[0], k), 77, dtype=torch.int32, device="cuda")
    w = torch.empty(x.shape[0], k, device="cuda")
    ns.muon_moe_route(h, x, ids, w, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top)
    ns.muon_last_device_error(h)
    return ids.cpu().numpy()


def check(x, bias, ids, groups, top_groups, group_top, bound=BOUND):
    """Every row's choice against its 64-bit values; returns how many rows
    differ from the 64-bit choice."""
    x64 = x.double().cpu().numpy()
    b64 = None if bias is None else bias.double().cpu().numpy()
    t, e = x64.shape
    size, k = e // groups, ids.shape[1]
    c = ref.choice_values(x64, False, b64, group_top, False)
    value = -np.sort(-c.reshape(t, groups, size), axis=2)[:, :, :group_top].sum(2)
    want, _, _ = ref.route(x64, k, softmax=False, bias=b64, groups=groups, top_groups=top_groups, group_top=group_top)
    differ = 0
    for i in range(t):
        got = ids[i]
        assert (got >= 0).all() and (got < e).all() and len(set(got)) == k
        order = np.argsort(-value[i], kind="stable")
        kept, left = order[:top_groups], order[top_groups:]
        lowest = value[i, kept].min()
        highest = value[i, left].max() if len(left) else -np.inf
        used = set(got // size)
        assert len(used) <= top_groups
        # No group that is clearly below the last one kept.
        assert all(value[i, g] >= lowest - bound for g in used), i
        # Of the groups that are clearly above the first one left, the best experts.
        least = c[i, got].min()
        for g in kept:
            if value[i, g] > highest + bound:
                rest = np.setdiff1d(np.arange(g * size, (g + 1) * size), got)
                assert not len(rest) or c[i, rest].max() <= least + bound, i
        assert (np.diff(c[i, got]) <= bound).all(), i
        if lowest > highest + bound:             # no tie of groups: the 64-bit choice
            assert np.abs(c[i, got] - c[i, want[i]]).max() <= bound, i
        differ += int((got != want[i]).any())
    return differ


SHAPES = [(64, 8, 3), (512, 16, 4), (96, 8, 2), (77, 7, 3), (1024, 32, 1)]


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("e,groups,top_groups", SHAPES)
def test_random_rows(ns, h, e, groups, top_groups, dtype, group_top):
    g = torch.Generator("cuda").manual_seed(e + group_top)
    x = (torch.randn(600, e, generator=g, device="cuda") * 1.5).to(getattr(torch, dtype))
    bias = torch.randn(e, generator=g, device="cuda") * 0.1
    k = min(7, top_groups * (e // groups))
    ids = route(ns, h, x, k, bias, groups, top_groups, group_top)
    differ = check(x, bias, ids, groups, top_groups, group_top)
    # Two values within the bound are a matter of a few in a million.
    assert differ <= 6, differ


def tied_rows(t, e, groups, top_groups, seed):
    """Rows whose last kept and first left group are a few 1e-6 apart (the
    difference, up to 2e-5 either way, is each row's own; every eighth row: equal)."""
    rng = np.random.default_rng(seed)
    size = e // groups
    s = rng.uniform(0.05, 0.3, (t, groups, size))
    rows = np.arange(t)
    place = np.argsort(rng.random((t, groups)), axis=1)          # groups in order of value
    for j in range(groups):
        g = place[:, j]
        top = 0.80 - 0.01 * j if j < top_groups - 1 else 0.70 - (0.01 * (j - top_groups) if j > top_groups else 0.0)
        s[rows, g, rng.integers(0, size // 2, t)] = top
        s[rows, g, size // 2 + rng.integers(0, size - size // 2, t)] = 0.6
    delta = rng.uniform(-2e-5, 2e-5, t) * rng.choice([0.05, 0.3, 1.0], t)
    delta[::8] = 0.0
    g = place[:, top_groups]
    best = s[rows, g].argmax(1)
    s[rows, g, best] += delta
    return np.log(s / (1 - s)).reshape(t, e).astype(np.float32)


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("e,groups,top_groups", [(64, 8, 3), (512, 16, 2), (96, 8, 2), (77, 7, 3), (1024, 32, 1)])
def test_groups_a_few_millionths_apart(ns, h, e, groups, top_groups, group_top):
    x = torch.from_numpy(tied_rows(1200, e, groups, top_groups, e + group_top)).cuda()
    size = e // groups
    k = min(32, top_groups * size)                # all experts of the groups kept, or most
    for bias in (None, torch.full((e,), 0.125, device="cuda")):
        ids = route(ns, h, x, k, bias, groups, top_groups, group_top)
        check(x, bias, ids, groups, top_groups, group_top)


def test_equal_groups_go_to_the_lowest(ns, h):
    """Equal logits have equal values: the choice is exact."""
    g = torch.Generator("cuda").manual_seed(1)
    for e, groups, top in ((512, 16, 4), (96, 8, 3), (77, 7, 2)):
        size = e // groups
        # Steps of 1/64: values that are not equal are far apart.
        pattern = torch.round(torch.randn(300, 1, size, generator=g, device="cuda") * 64) / 64
        x = pattern.repeat(1, groups, 1)
        worse = torch.rand(300, groups, generator=g, device="cuda") < 0.4
        x = torch.where(worse[:, :, None], x - 1.0, x).reshape(300, e).contiguous()
        for group_top in (1, 2):
            ids = route(ns, h, x, min(5, top * size), None, groups, top, group_top)
            want, _, _ = ref.route(x.double().cpu().numpy(), ids.shape[1], softmax=False, groups=groups, top_groups=top,
                                   group_top=group_top)
            np.testing.assert_array_equal(ids, want)
