"""The persistent grids of the FP8 products: how many CTA pairs they have is a
handle's, asked of its device when it is made; a question that fails is an
error, not a grid of one pair for good."""

import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
#include <cstdio>
#include "moe.h"
using muon::resident_pairs;
int main() {
  int out = -7, asked = 0;
  auto fails = [&](int* n) { ++asked; *n = 3; return cudaErrorUnknown; };
  auto none = [&](int* n) { ++asked; *n = 0; return cudaSuccess; };
  auto many = [&](int* n) { ++asked; *n = 76; return cudaSuccess; };
  if (resident_pairs(fails, 152, &out) != cudaErrorUnknown || out != -7) return 1;
  if (resident_pairs(none, 152, &out) == cudaSuccess || out != -7) return 2;
  if (resident_pairs(many, 1, &out) == cudaSuccess || out != -7) return 3;
  // Nothing of a failure stays: the next answer counts.
  if (resident_pairs(many, 152, &out) != cudaSuccess || out != 76) return 4;
  if (resident_pairs(many, 148, &out) != cudaSuccess || out != 74) return 5;
  if (asked != 5) return 6;
  std::puts("ok");
  return 0;
}
"""


def test_a_failed_query_is_an_error(tmp_path):
    from newton_schulz_03_gb300 import build_lib
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build_lib.nvcc()))), "include")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-I", include, "-I", build_lib.CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout == "ok\n"


@pytest.mark.gpu
def test_handles_of_several_threads_agree():
    """Handles made and used at the same time, one per thread and stream."""
    import threading
    torch = pytest.importorskip("torch")
    import newton_schulz_03_gb300 as ns
    from tests.test_gpu_fp8_product import exact_product, product_case, tolerance
    off, x, xs, w, ws = product_case([300, 0, 77], 272, 400, 11)
    d_off = torch.from_numpy(off).cuda()
    torch.cuda.synchronize()
    ys, errors = [None] * 6, []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with ns.Handle() as h, torch.cuda.stream(stream):
                y = torch.empty(x.shape[0], 272, dtype=torch.bfloat16, device="cuda")
                ns.muon_fp8_grouped_matmul(h.value, x, xs, w, ws, d_off, y, stream=stream)
                stream.synchronize()
                ns.muon_last_device_error(h.value)
                ys[i] = y
        except Exception as e:               # noqa: BLE001 - reported below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(ys))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert all(torch.equal(y, ys[0]) for y in ys)
    want, size = exact_product(off, x, xs, w, ws)
    assert (np.abs(ys[0].double().cpu().numpy() - want) <= np.abs(want) / 256 + tolerance(400) * size).all()
