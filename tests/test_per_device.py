"""CPU test of csrc/per_device.h, compiled as it is: numbers are found once per device, a
failure is not kept, and threads may ask at the same time."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_expert_ffn_router_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>

#include "per_device.h"

#define CHECK(x) if (!(x)) return std::printf("line %d: %s\n", __LINE__, #x), 1

static k3moe::PerDevice a, b;

int main() {
  int calls = 0;
  auto find = [&](int n) { return [&calls, n] { ++calls; return n; }; };
  CHECK(a.get(0, find(7)) == 7 && calls == 1);
  CHECK(a.get(0, find(8)) == 7 && calls == 1);       // known
  CHECK(a.get(1, find(0)) == 0 && calls == 2);       // another device's is its own
  CHECK(a.get(1, find(9)) == 0 && calls == 2);       // 0 is a number
  CHECK(a.get(2, find(-1)) == -1 && calls == 3);     // a failure
  CHECK(a.get(2, find(5)) == 5 && calls == 4);       // is not kept
  CHECK(a.get(2, find(-1)) == 5 && calls == 4);
  CHECK(a.get(63, find(4)) == 4 && a.get(63, find(3)) == 4 && calls == 5);
  CHECK(a.get(64, find(1)) == 1 && a.get(64, find(2)) == 2);    // no place for it: found out each time
  CHECK(a.get(-1, find(1)) == 1 && a.get(-1, find(2)) == 2);
  std::vector<std::thread> ts;
  std::atomic<int> wrong{0};
  for (int t = 0; t < 8; ++t)
    ts.emplace_back([&] {
      for (int i = 0; i < 20000; ++i)
        if (b.get(i % 64, [i] { return i % 64 + 1; }) != i % 64 + 1) ++wrong;
    });
  for (auto &t : ts) t.join();
  CHECK(wrong == 0);
  return 0;
}
"""


@pytest.mark.parametrize("flags", [[], ["-fsanitize=thread"]])
def test_per_device(tmp_path, flags):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    build = ["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)] + flags
    r = subprocess.run(build, capture_output=True, text=True)
    if flags and r.returncode:
        pytest.skip("no thread sanitizer here")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    if flags and "FATAL: ThreadSanitizer" in r.stderr:
        pytest.skip("the thread sanitizer does not run here")
    assert r.returncode == 0, r.stdout + r.stderr
