"""What a kernel's launches work out once per device is worked out once, complete for every thread, and again after a
failure (csrc/per_device.h, compiled here; under the thread sanitizer where the compiler has it)."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_mixture_experts_expert_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"
struct Big { int v[64]; };
int main() {
  static nvfp4::PerDevice<Big, int> once;
  static std::atomic<int> fills{0}, bad{0}, failed{0};
  std::atomic<bool> go{false};
  std::vector<std::thread> all;
  for (int t = 0; t < 8; ++t)
    all.emplace_back([&, t] {
      while (!go) {}
      for (int i = 0; i < 2000; ++i) {
        const int dev = (i + t) % 3 * 31;  // 0, 31, 62
        const Big* b = nullptr;
        const int e = once.get(dev, &b, [&](Big& x) {
          if (fills.fetch_add(1) == 1) return 7;  // one attempt fails
          for (int& v : x.v) v = dev + 1;
          return 0;
        });
        if (e) { failed += e == 7 && !b; continue; }
        for (int v : b->v) bad += v != dev + 1;
      }
    });
  go = true;
  for (auto& t : all) t.join();
  printf("%d %d %d\n", fills.load(), bad.load(), failed.load());
}
"""


@pytest.mark.parametrize("flags", [["-O2"], ["-O1", "-fsanitize=thread"]])
def test_filled_once_per_device_and_complete(tmp_path, flags):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-pthread", "-I", CSRC, *flags, str(src), "-o", str(exe)], capture_output=True,
                       text=True)
    if r.returncode and "-fsanitize=thread" in flags:
        pytest.skip("no thread sanitizer")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.split() == ["4", "0", "1"], r.stdout + r.stderr  # 3 devices, one failure


def test_launches_keep_no_state_of_their_own():
    """No kernel file of the FFN-block operators keeps a bare static that threads would share."""
    for name in ("norm_fp8.cu", "fp8_small.cu", "fp8_split.cu", "fp8_gemm.cu", "fp8_mma.cuh", "moe_few.cu"):
        with open(os.path.join(CSRC, name)) as f:
            for line in f:
                words = line.split()
                if words and words[0] == "static" and not words[1].startswith(("constexpr", "PerDevice", "std::atomic", "inline")):
                    assert "(" in line and "=" not in line, (name, line)
