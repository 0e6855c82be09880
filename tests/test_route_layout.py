"""Every number of experts and groups that routing by scores takes: the layout over a warp's lanes
holds each expert once, within the places of the kernel that is taken."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "route_layout.h"
int main() {
  int sizes = 0, bad = 0, most = 0;
  for (int E = 1; E <= 2048; ++E)
    for (int groups = 1; groups <= 32; ++groups) {
      if (E % groups) continue;
      for (int bytes = 2; bytes <= 4; bytes += 2)
        for (int wide = 0; wide < 2; ++wide) {
          const moe::RouteLayout p = moe::route_layout(E, groups, bytes, wide != 0);
          const int places = moe::route_places(p), whole = places & ((1 << p.run) - 1);
          std::vector<int> seen(E);
          bool in_range = p.lanes >= 1 && p.lanes * groups <= 32 && whole == 0 && (groups > 1 || places <= 64);
          for (int lane = 0; lane < 32; ++lane)
            for (int i = 0; i < p.per && i < places; ++i) {
              const int e = moe::route_expert_at(p, i, lane);
              if (e < -1 || e >= E) in_range = false;
              else if (e >= 0) ++seen[e];
            }
          bool once = true;
          for (int n : seen) once = once && n == 1;
          if (p.per > places || !once || !in_range) {
            if (bad++ < 5) std::printf("%d experts in %d groups: %d a lane, %d places\n", E, groups, p.per, places);
          }
          most = p.per > most ? p.per : most;
          ++sizes;
        }
    }
  std::printf("sizes %d bad %d most %d\n", sizes, bad, most);
}
"""


def test_every_size_has_its_places(tmp_path):
    src = tmp_path / "t.cc"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "fp8_block_scale_gb300", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I", csrc, str(src), "-o", str(tmp_path / "t")], check=True)
    said = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, check=True).stdout
    want = 4 * sum(1 for E in range(1, 2049) for g in range(1, 33) if E % g == 0)
    assert said.splitlines()[-1] == f"sizes {want} bad 0 most 120", said
