"""The numbering of the recurrence's workgroups (gdn_hybrid.h), compiled for the CPU: every
number gives a slot of the launch or none, whatever the counter in a workspace says that two
calls share."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cstdint>
#include <cstdio>
#include <vector>
#include "gdn_hybrid.h"
int main() {
  for (int tiles : {1, 3, 16384})
    for (int64_t slots : {1, 7, 1000})
      for (bool back : {false, true}) {
        std::vector<int> seen(slots, 0);
        int64_t before = back ? slots : -1;
        for (int64_t s = 0; s < slots; ++s) {
          const int64_t slot = gdn::glr_slot(s * tiles + (s % tiles), tiles, slots, back);
          if (slot < 0 || slot >= slots || seen[slot]++ || (back ? slot >= before : slot <= before)) return 1;
          before = slot;
        }
        // a counter that went on: up to all that 32 bits count
        for (int64_t index : {slots * tiles, slots * tiles + 1, 3 * slots * tiles, int64_t(UINT32_MAX)})
          if (gdn::glr_slot(index, tiles, slots, back) != -1) return 2;
      }
  std::puts("ok");
}
"""


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"), reason="needs g++ and the ROCm headers")
def test_every_number_is_a_slot_or_none(tmp_path):
    src, exe = tmp_path / "slots.cpp", tmp_path / "slots"
    src.write_text(SOURCE)
    r = subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                        "-I" + os.path.join(ROOT, "gated_deltanet_chunked_gdn_amd", "csrc"), str(src), "-o", str(exe)],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok"
