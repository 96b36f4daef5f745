"""Host code of the device-side step without a GPU."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "zero_copy_offloaded_gb300", "csrc")

THREADS = r"""
#include <stdio.h>
#include <thread>
#include <vector>
#include "per_device.h"
static dkv::PerDevice once;
static std::atomic<int> calls[66];
int main() {
  std::vector<std::thread> t;
  for (int i = 0; i < 8; ++i)
    t.emplace_back([i] {
      for (int k = 0; k < 2000; ++k)
        for (int d : {0, 3, 63, 64}) {
          // the first tries on device 3 fail
          const int e = once(d, [d] { return ++calls[d] <= 5 && d == 3 ? 7 : 0; });
          if (e && d != 3) return;
        }
    });
  for (auto& x : t) x.join();
  printf("%d %d %d %d\n", calls[0].load(), calls[3].load(), calls[63].load(), calls[64].load());
}
"""


def test_settings_made_once_a_device_by_any_thread(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    (tmp_path / "probe.cc").write_text("int main() {}\n")
    (tmp_path / "threads.cc").write_text(THREADS)
    build = lambda name: subprocess.run(  # noqa: E731
        [gxx, "-std=c++17", "-O1", "-fsanitize=thread", "-pthread", "-I", CSRC, str(tmp_path / f"{name}.cc"), "-o",
         str(tmp_path / name)], capture_output=True, text=True)
    run = lambda name: subprocess.run([str(tmp_path / name)], capture_output=True, text=True, timeout=120)  # noqa: E731
    if build("probe").returncode or run("probe").returncode:
        pytest.skip("no thread sanitizer")
    b = build("threads")
    assert b.returncode == 0, b.stderr
    r = run("threads")
    assert r.returncode == 0 and "data race" not in r.stderr, r.stderr[:2000]
    first, failing, last, beyond = map(int, r.stdout.split())
    assert 1 <= first <= 8 and 1 <= last <= 8 and 6 <= failing <= 13 and beyond == 16000
