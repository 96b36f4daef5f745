"""Host code of the 8-bit step without a GPU: how the append's launch is divided."""
import os
import shutil
import subprocess
import sys

import pytest

from zero_copy_offloaded_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_copy_offloaded_gb300", "csrc")

GEOMETRY = r"""
#include <stdio.h>
#include <initializer_list>
#include "append_geometry.h"
int main() {
  for (int rows : {1, 8, 16, 17, 64, 512, 1023, 1024, 1025, 2000, 2048, 4096, 16384, 1 << 20, 1 << 30})
    for (int hq : {0, 1, 7, 32, 33, 65536})
      for (int hkv : {1, 2, 3, 8, 32, 33, 65536})
        for (int d : {64, 128}) {
          const dkv::AppendGeometry g = dkv::append_geometry(rows, hq, hkv, d);
          printf("%d %d %d %d %d %d %d %d %d %d %d %d\n", rows, hq, hkv, d, g.q_items, g.heads, g.span, g.parts,
                 g.block_ctas, g.token_ctas, g.q_ctas, g.grid);
        }
}
"""


def test_the_launch_of_every_size(tmp_path):
    """No division by zero and no overflow (the sanitizer ends the program), every kind of work has CTAs, and short calls
    are told from long ones by `span`."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    (tmp_path / "g.cc").write_text(GEOMETRY)
    b = subprocess.run([gxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC,
                        str(tmp_path / "g.cc"), "-o", str(tmp_path / "g")], capture_output=True, text=True)
    assert b.returncode == 0, b.stderr
    r = subprocess.run([str(tmp_path / "g")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    seen = 0
    for line in r.stdout.splitlines():
        rows, hq, hkv, d, q_items, heads, span, parts, block_ctas, token_ctas, q_ctas, grid = map(int, line.split())
        seen += 1
        assert heads in (1, 2, 4) and 1 <= parts <= 16
        assert q_items == -(-hq // (8 * 32 * 8 // d))
        groups = -(-hkv // (256 // d))
        if rows < 1024:  # a token and a group to a warp
            assert span == 0 and parts == 1 and token_ctas == min(-(-rows * groups // 8), 16 * 3 * 152)
        else:
            assert 1 <= span < 2 * groups and token_ctas <= 16 * 3 * 152
        assert block_ctas >= 1 and token_ctas >= 1 and (q_ctas >= q_items if hq else q_ctas == 0)
        assert q_items == 0 or q_ctas % q_items == 0
        assert grid == 2 * (block_ctas + token_ctas) + q_ctas
    assert seen == 15 * 6 * 7 * 2


@pytest.mark.parametrize("rows", [1, 8, 1023, 1024, 2000, 4096])
def test_an_append_without_a_gpu_says_so(rows):
    """The entry point's own host code, up to the launch: a status, not a signal.  (No device is visible to the process, so
    nothing can be launched.)"""
    build.build()
    code = ("import zero_copy_offloaded_gb300 as dkv\n"
            "from tests.test_block_cpu import APPEND\n"
            f"args = dkv._BLOCK_APPEND.pack(*{{**APPEND, 'rows': {rows}}}.values())\n"
            "print(dkv.lib().dkv_block_append(args, None))\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT,
                       env={**os.environ, "CUDA_VISIBLE_DEVICES": "", "PYTHONPATH": ROOT})
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert int(r.stdout.split()[-1]) not in (0, 1, 2)
