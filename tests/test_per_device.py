"""Kernel attributes and occupancies belong to a device: kept apart for each one a process uses (no GPU)."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from chunked_prefill_paged_cpa_gb300 import build

PROGRAM = r"""
#include "per_device.cuh"
#include <cstdio>
#include <thread>
#include <vector>
static int made[70], limit[70];  // a fake function attribute of every device, and how often it was set
static cpa::PerDevice configured;
static int launch(int device, bool fails = false) {
  return configured.get(device, [&] {
    ++made[device < 0 ? 69 : device];
    if (fails) return 0;
    limit[device < 0 ? 69 : device] = 200;
    return 100 + device;
  });
}
int main() {
#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
  CHECK(launch(0) == 100 && limit[0] == 200);
  CHECK(launch(1) == 101 && limit[1] == 200);   // the second device is set up too
  CHECK(launch(0) == 100 && launch(1) == 101 && made[0] == 1 && made[1] == 1);
  CHECK(launch(2, true) == 0 && limit[2] == 0); // a failure is not kept
  CHECK(launch(2) == 102 && limit[2] == 200 && made[2] == 2);
  CHECK(launch(66) == 166 && launch(66) == 166 && made[66] == 2);  // past the table: made every time
  CHECK(launch(-1) == 99 && launch(-1) == 99 && made[69] == 2);
  static cpa::PerDevice one;
  std::vector<std::thread> t;
  std::atomic<int> wrong{0};
  for (int i = 0; i < 8; ++i)
    t.emplace_back([&] { for (int k = 0; k < 5000; ++k) if (one.get(k % 64, [&] { return 1 + k % 64; }) != 1 + k % 64) ++wrong; });
  for (auto &x : t) x.join();
  CHECK(wrong == 0);
  return 0;
}
"""


def test_a_number_for_each_device(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_nothing_of_a_device_is_kept_per_process():
    """No flag or number found out once for the whole process in the launching code."""
    for path in glob.glob(os.path.join(build.CSRC, "*.cu*")):
        with open(path) as f:
            text = f.read()
        kept = re.findall(r"^\s*static\s+(?:const\s+)?(?:bool|int)\b[^()\n]*=.*$", text, re.M)
        assert not kept, f"{os.path.basename(path)}: {kept}"
