"""The launch plans of tree attention (host only): whatever plan_tree hands to the walk, the
plan that the walk makes of it is one that it can launch."""
import os
import subprocess

import pytest

from w4a16_bit_matmul_amd import _build

PROGRAM = r"""
#include "wq_kv_walk.h"
#include <cstdio>

int main() {
  for (int D : {64, 128, 256})
    for (int Hkv : {2, 8, 16})
      for (int G : {1, 4, 8, 16})
        for (int B : {1, 4, 64, 300, 5000})
          for (int64_t nodes : {1, 4, 16, 64, 125, 600})
            for (int64_t context : {0, 100, 3000, 20000, 1000000}) {
              const wq::KvPlan p = wq::plan_kv(B, G * Hkv, Hkv, D, context, nodes, true);
              const int64_t rows = nodes * G;
              if (p.chunk || (p.RT != 1 && p.RT != 2) || (int64_t)p.rtiles * 16 * p.RT < rows || Hkv % p.HP) {
                printf("D=%d heads %d x %d, %d trees of %ld nodes over %ld: chunk=%d RT=%d rtiles=%d HP=%d\n", D, Hkv, G, B,
                       (long)nodes, (long)context, p.chunk, p.RT, p.rtiles, p.HP);
                return 1;
              }
            }
  return 0;
}
"""


@pytest.mark.skipif(not os.path.exists(_build.HIPCC), reason="hipcc is not installed")
def test_the_walk_can_launch_every_plan_of_a_tree(tmp_path):
    src, exe = tmp_path / "plans.cpp", tmp_path / "plans"
    src.write_text(PROGRAM)
    subprocess.run([_build.HIPCC, "-x", "hip", *_build.COMMON, "-Wno-unused-function", f"-I{_build.CSRC}", str(src), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
