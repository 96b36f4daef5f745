"""Host code of the device-side step without a GPU."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from .step_tiles import CASES, TILE, Tiles

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


# ---- what the tile cases of the attention can see ------------------------------------------------------

@pytest.mark.parametrize("name", CASES)
def test_tile_cases_see_a_lost_or_doubled_tile(name):
    case = Tiles(*CASES[name])
    for b, keys in enumerate(case.lens):
        tiles = -(-keys // TILE)
        if case.rows[b] == 0 or tiles < 2:
            continue
        want = case.reference(b)
        assert case.bad(b, *want, want) == (0, 0)
        piece = -(-tiles // 608)  # as little as one CTA may hold of the sequence
        for at in {0, tiles // 3, tiles // 2, max(0, (keys - case.rows[b]) // TILE - piece)}:
            for off in (dict(without=(at, at + piece)), dict(twice=(at, at + piece)), dict(without=(at, at + 1))):
                out, lse = case.reference(b, **off)
                assert case.bad(b, *want, (out, lse))[1] > 0, (name, b, off)  # lse
        # and outputs short of a piece beside a sum that is not, as far as 16 bits can show it
        piece = -(-tiles // 152)
        out, lse = case.reference(b, without=(tiles // 2, tiles // 2 + piece))
        assert case.bad(b, out * np.exp(lse - want[1])[..., None], want[1], want)[0] > 0, (name, b)
        # a neighbour's tiles in place of one's own
        other = case.reference(b + 1)[0] if b + 1 < len(case.lens) and case.rows[b + 1] == case.rows[b] else None
        if other is not None and case.lens[b + 1]:
            assert case.bad(b, other, want[1], want)[0] > 0
