"""per_device (csrc/host_common.h): a figure kept for each device, compiled against a cudaGetDevice of the test's own."""
import shutil
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "paged_kv_cache_int64_gb300" / "csrc"
PROGRAM = r"""
#include "host_common.h"
#include <stdlib.h>
#include <thread>
#include <vector>
static thread_local int device = 0;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
static std::atomic<int> asked[100];
static std::atomic<int> known[64];
static int figure() {
  return pkv::per_device(known, [] { ++asked[device]; return 10 + device; });
}
#define CHECK(x) if (!(x)) { printf("line %d: %s\n", __LINE__, #x); exit(1); }
int main() {
  for (int round = 0; round < 3; ++round)
    for (int d : {0, 1, 63, 64, 90}) {  // each device its own figure, whichever was asked last
      device = d;
      CHECK(figure() == 10 + d);
      CHECK(asked[d] == (d < 64 ? 1 : round + 1));
    }
  std::vector<std::thread> all;  // first calls at once
  for (int t = 0; t < 16; ++t)
    all.emplace_back([t] { device = 2 + t % 4; for (int i = 0; i < 1000; ++i) CHECK(figure() == 10 + device); });
  for (auto& t : all) t.join();
  return 0;
}
"""


def test_a_figure_for_each_device(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    include = Path(nvcc).resolve().parent.parent / "include"
    if not shutil.which("g++") or not include.is_dir():
        pytest.skip("no g++ or CUDA headers")
    (tmp_path / "t.cpp").write_text(PROGRAM)
    out = tmp_path / "t"
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", str(CSRC), "-I", str(include), str(tmp_path / "t.cpp"), "-o", str(out)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
