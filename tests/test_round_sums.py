"""The long FP32 sums of squares of a gradient's norm, on the CPU (the header compiled alone): within 16 roundings of
the exact sum for any number of rounds, a large one in front of small ones too."""
import shutil
import subprocess

import pytest

from moe_routing_swiglu_gb300 import _build

PROGRAM = r"""
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include "round_sums.h"

int main() {
  const double limit = 16 * 0x1p-24;
  for (int rounds : {1, 15, 16, 17, 33, 48, 513, 2048, 5000})
    for (int kind = 0; kind < 4; ++kind) {
      moe::RoundSums s;
      double exact = 0.0;
      uint32_t state = 1u + rounds + kind;
      for (int i = 0; i < rounds; ++i) {
        state = state * 1664525u + 1013904223u;
        const float u = 1.0f + (state >> 8) * 0x1p-24f;
        float v = u;                                            // alike
        if (kind == 1) v = i == 0 ? 1.0f : 0x1.fp-25f;          // a large one, then less than half its last bit
        if (kind == 2) v = std::ldexp(u, static_cast<int>(state >> 28) * 3 - 24);   // of all sizes
        if (kind == 3) v = 1.0f + 0x1p-23f;                     // every addition rounds the same way
        exact += v;
        s.add(v);
      }
      const double off = std::fabs(s.near + s.far - exact) / exact;
      if (off > limit) return std::printf("%d rounds, kind %d: off by 2^%.1f\n", rounds, kind, std::log2(off)), 1;
    }
  return 0;
}
"""


def test_sums_are_within_sixteen_roundings(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "sums.cpp", tmp_path / "sums"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", str(_build.CSRC), str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout


def test_the_norm_of_a_gradient_is_summed_that_way():
    text = (_build.CSRC / "newton_schulz.cu").read_text()
    kernel = text[text.index("squares_kernel("):text.index("split_half(")]
    assert "RoundSums total;" in kernel and "total.add(sum);" in kernel and "near +=" not in kernel
