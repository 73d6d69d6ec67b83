"""The kernel statistics' layouts: programs built against the header with nine
classes get what that header declares, programs built against this one all
classes."""

import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NINE = 9 * 8 + 9 * 8 + 8

# What a program built against the header of version 0.1.0 contains.
OLD = """
typedef struct { double total_ms[9]; long long launches[9]; long long total_launches; } old_t;
"""

PROGRAM = OLD + """
#include <stdio.h>
#include <string.h>
#include "muon.h"
#define STR2(x) #x
#define STR(x) STR2(x)
int main(void) {
  printf("%zu %zu %zu %d %s\\n", sizeof(old_t), sizeof(muon_kernel_stats_v1_t), sizeof(muon_kernel_stats_t),
         (int)MUON_KERNEL_COUNT, STR(muon_kernel_stats));
  return 0;
}
"""


def test_layouts_and_names_in_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text(PROGRAM)
    exe = tmp_path / "t"
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got[:3]] == [NINE, NINE, int(got[3]) * 16 + 8]
    assert int(got[3]) > 9
    # Sources that include the header reach the function that fits the structure.
    assert got[4] == "muon_kernel_stats_v2"


def test_binding_matches_the_header():
    import newton_schulz_03_gb300 as ns
    from newton_schulz_03_gb300 import _native
    assert ctypes.sizeof(_native._StatsV1) == NINE
    assert ctypes.sizeof(_native._Stats) == len(ns.KERNEL_NAMES) * 16 + 8
    assert "0.1.0" not in ns.muon_version()


@pytest.mark.gpu
def test_the_old_symbol_writes_nine_classes():
    """Its caller's buffer is as long as the old structure: nothing behind it is touched."""
    torch = pytest.importorskip("torch")
    import newton_schulz_03_gb300 as ns
    with ns.Handle() as h:
        w, m, g = (torch.randn(2, 128, 256, device="cuda") for _ in range(3))
        ns.muon_step(h.value, [(128, 256, 2)], [m], [g], [w], 0.02, 0.1, 0.95)
        ids = torch.zeros(64, dtype=torch.int32, device="cuda")
        ns.muon_moe_plan(h.value, ids, torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty_like(ids), torch.empty_like(ids))
        buf = (ctypes.c_uint8 * 4096)(*([0xAB] * 4096))
        fn = ctypes.CDLL(ns.LIB_PATH).muon_kernel_stats
        assert fn(ctypes.c_void_p(h.value), buf) == 0
        assert all(b == 0xAB for b in buf[NINE:])
        launches = (ctypes.c_int64 * 10).from_buffer(buf, 9 * 8)
        new = ns.muon_kernel_stats(h.value)
        assert list(launches[:9]) == [new["launches"][k] for k in ns.KERNEL_NAMES[:9]]
        assert launches[9] == new["total_launches"] == 19      # 18 of the step, one of the grouping
        assert new["launches"]["moe_plan"] == 1 and new["launches"]["ns_gram"] == 5
        assert fn(ctypes.c_void_p(h.value), None) == 1
        ns.muon_last_device_error(h.value)
