"""The waits that a block owes the asynchronous copies it has in flight when one of its roles gives up: a model of the
barriers' phases on the CPU (the header compiled alone), and that the kernels drain every ring they fill. No GPU is
made to time out for this."""
import re
import shutil
import subprocess

import pytest

from moe_routing_swiglu_gb300 import _build

MODEL = r"""
#include <cstdio>
#include <vector>
#include "ring_drain.h"

// A barrier as its waiters see it: phases end in order; a wait by parity p is over when the current phase's parity
// is not p.
struct Bar { uint32_t armed = 0, ended = 0; };

int main() {
  long cases = 0;
  for (uint32_t depth = 1; depth <= 8; ++depth)
    for (uint32_t issued = 0; issued <= 5 * depth + 1; ++issued) {
      // Stages 0 .. issued - 1 were armed in order, each after its slot's last one had ended. Of the last `depth`
      // any subset is still in flight.
      const uint32_t back = issued < depth ? issued : depth;
      for (uint32_t flying = 0; flying < (1u << back); ++flying) {
        std::vector<Bar> bar(depth);
        std::vector<bool> waited(issued, false);
        for (uint32_t n = 0; n < issued; ++n) {
          Bar& b = bar[n % depth];
          if (b.armed != b.ended || b.armed != n / depth) return std::printf("model\n"), 1;
          ++b.armed;
          const uint32_t i = issued - 1 - n;
          if (i >= back || ((flying >> i) & 1u) == 0) ++b.ended;
        }
        bool bad = false;
        moe::drain_ring(issued, depth, [&](uint32_t slot, uint32_t parity) {
          Bar& b = bar[slot];
          if (b.armed == 0) { bad = true; return; }            // would never end
          if ((b.ended & 1u) == parity) {                      // blocks until the current phase ends
            if (b.armed == b.ended) { bad = true; return; }    // nothing in flight will end it
            ++b.ended;
          }
          waited[(b.armed - 1) * depth + slot] = true;
        });
        for (const Bar& b : bar) bad |= b.armed != b.ended;    // a copy is still in flight
        for (uint32_t n = issued - back; n < issued; ++n) bad |= !waited[n];
        if (bad) return std::printf("depth %u issued %u flying %x\n", depth, issued, flying), 1;
        ++cases;
      }
    }
  std::printf("%ld\n", cases);
  return 0;
}
"""


def test_every_copy_in_flight_is_waited_for(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "model.cpp", tmp_path / "model"
    src.write_text(MODEL)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", str(_build.CSRC), str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
    assert int(run.stdout) > 3000


# file: the "full" barriers of the rings that bulk copies of the file's kernel fill
RINGS = {"experts_mx.cu": {"full", "sf_full"}, "experts_tc.cu": {"full"}, "experts_bwd_tc.cu": {"full"}}


@pytest.mark.parametrize("name", sorted(RINGS))
def test_a_block_that_gives_up_drains_every_ring(name):
    """Every barrier that a bulk copy signals is drained after the block's last barrier under the abort flag, whichever
    role gave up, and no role returns before that."""
    text = re.sub(r"//[^\n]*", "", (_build.CSRC / name).read_text())
    signalled = set(re.findall(r"(?:tma_load_[23]d|tma_gather4|bulk_load)\([^;]*?&(\w*full)\[", text))
    assert signalled == RINGS[name]
    head, tail = text.rsplit("__syncthreads();", 1)
    tail = tail[:tail.index("tmem_dealloc")]
    assert re.search(r"if \(\*abort_flag != 0\)", tail)
    drained = set(re.findall(r"drain_ring\([^;]*?mbar_wait_bounded\(&(\w+)\[", tail))
    assert drained == signalled
    body = head[head.rindex("__global__ void __launch_bounds__"):]
    assert "return;" not in body
