"""The bound on a softmax score's error that decides which experts are compared in 64 bits."""

import os
import subprocess

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "route_layout.h"
int main() {
  for (int E = 1; E <= 2048; ++E)
    for (int groups = 1; groups <= 32; ++groups) {
      if (E % groups) continue;
      const int places = moe::route_places(moe::route_layout(E, groups, 4, false));
      std::printf("%d %d %.9g\n", E, places, moe::route_softmax_units(E, places));
    }
}
"""


def largest_average(E):
    """The largest average of x >= 0 over weights exp(-x), one of E of them at 0: the others at one x."""
    x = np.linspace(0.0, 12.0, 4801)
    return (((E - 1) * x) / (np.exp(x) + E - 1)).max()


def test_one_distance_is_the_worst():
    rng = np.random.default_rng(1)
    for E in (2, 9, 64, 2048):
        most = largest_average(E)
        for _ in range(300):
            x = rng.random(E) * rng.choice([1.0, 4.0, 8.0, 12.0]) + rng.random() * 6
            x[0] = 0.0
            w = np.exp(-x)
            assert (w * x).sum() / w.sum() <= most + 1e-5


def test_bound_covers_every_source(tmp_path):
    src = tmp_path / "t.cc"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "fp8_block_scale_gb300", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", csrc, str(src), "-o", str(tmp_path / "t")], check=True)
    said = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, check=True).stdout
    averages, x = {}, np.linspace(0.0, 20.0, 2001)
    for line in said.splitlines():
        E, places, units = int(line.split()[0]), int(line.split()[1]), float(line.split()[2])
        if E not in averages:
            averages[E] = largest_average(E)
        total = 2 + 1.7 * averages[E] + (places + 5) / 2 + 1 + 0.5       # terms, additions, reciprocal, product
        need = (np.exp(-x) * (2 + 1.7 * x + total)).max()                # of a score, over that of the largest logit
        assert need <= units <= need + 4, line
