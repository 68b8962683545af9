"""The norms around a block copy rows into a ring while every thread of the block waits round after round, and goes on
when a wait runs out (the rounds have barriers that all must reach). A model of that on the CPU, with the header that
the kernels use: no stage is armed over a copy in flight, and none is in flight when the block exits. No GPU is made to
time out for this."""
import re
import shutil
import subprocess

import pytest

from moe_routing_swiglu_gb300 import _build

MODEL = r"""
#include <cstdio>
#include <vector>
#include "ring_drain.h"

// A barrier's phases end in order; each is armed once.
struct Bar { uint32_t armed = 0, ended = 0; };

// A stage's copy: LANDS before its round's waits; LATE, with the drain only; BETWEEN: another thread has given up on it
// when it lands, before the arming role's own wait.
enum { LANDS = 0, LATE = 1, BETWEEN = 2 };

int main() {
  long cases = 0, gave_up_cases = 0;
  for (uint32_t depth = 2; depth <= 4; ++depth)
    for (uint32_t behind = 0; behind <= 1; ++behind)                   // rounds after whose barrier a stage is free
      for (uint32_t rounds = 1; rounds <= 2 * depth + 1; ++rounds) {
        uint32_t kinds = 1;
        for (uint32_t n = 0; n < rounds; ++n) kinds *= 3;
        for (uint32_t code = 0; code < kinds; ++code) {
          std::vector<int> kind(rounds);
          for (uint32_t n = 0, c = code; n < rounds; ++n, c /= 3) kind[n] = c % 3;
          std::vector<Bar> bar(depth);
          uint32_t issued = 0, next = 0;
          bool flag = false, bad = false;
          auto issue = [&] {
            if (next >= rounds) return;
            Bar& b = bar[issued % depth];
            if (b.armed != b.ended) { bad = true; return; }            // a copy still in flight there
            ++b.armed;
            if (kind[issued] == LANDS) ++b.ended;
            ++issued;
            ++next;
          };
          for (uint32_t i = 0; i < depth; ++i) issue();
          for (uint32_t n = 0; n < rounds + behind && !bad; ++n) {
            if (n < rounds) {                                          // the waits for round n
              Bar& b = bar[n % depth];
              const bool armed = b.armed == n / depth + 1;
              if (!armed || b.ended != b.armed) flag = true;           // another thread's
              if (armed && kind[n] == BETWEEN && b.ended != b.armed) ++b.ended;
              const bool waited = armed && b.ended == b.armed;         // the arming role's
              if (!waited) flag = true;
              moe::issue_only_after(waited || IGNORE_GIVE_UP, next, rounds);
            }
            if (n >= behind) issue();                                  // after the round's barrier
          }
          if (!bad && flag) {
            moe::drain_ring(issued, depth, [&](uint32_t slot, uint32_t parity) {
              Bar& b = bar[slot];
              if (b.armed == 0) { bad = true; return; }
              if ((b.ended & 1u) == parity) {
                if (b.armed == b.ended) { bad = true; return; }        // nothing in flight will end it
                ++b.ended;
              }
            });
            ++gave_up_cases;
          }
          for (const Bar& b : bar) bad |= b.armed != b.ended;
          if (bad) return std::printf("depth %u rounds %u kinds %u\n", depth, rounds, code), 1;
          ++cases;
        }
      }
  std::printf("%ld %ld\n", cases, gave_up_cases);
  return 0;
}
"""


def run_model(tmp_path, ignore):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "model.cpp", tmp_path / "model"
    src.write_text(MODEL)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", f"-DIGNORE_GIVE_UP={ignore}", "-I", str(_build.CSRC),
                    str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True)


def test_no_stage_is_armed_after_a_give_up(tmp_path):
    run = run_model(tmp_path, 0)
    assert run.returncode == 0, run.stdout
    cases, gave_up = map(int, run.stdout.split())
    assert gave_up > 50000 and cases > gave_up


def test_the_model_sees_an_issuer_that_goes_on(tmp_path):
    assert run_model(tmp_path, 1).returncode == 1


def test_the_kernels_arm_after_their_own_waits():
    """Every wait for a round tells the arming role, a warp as one, and every ring ends in its drain."""
    text = re.sub(r"//[^\n]*", "", (_build.CSRC / "block_norm.cu").read_text())
    kernels = [text[m.start():] for m in re.finditer(r"__global__ void", text)]
    kernels = [k[:k.index("\n}\n")] for k in kernels if "ring_wait(" in k[:k.index("\n}\n")]]
    assert len(kernels) == 2
    for k in kernels:
        waits = k.count("ring_wait(ring, turn, a.status)")
        by_warp = k.count("issue_only_after(__all_sync(FULL_MASK, ring_wait(ring, turn, a.status)), issue_t0, rows);")
        by_thread = k.count("issue_only_after(ring_wait(ring, turn, a.status), issue_t0, rows);")
        assert waits == by_warp + by_thread > 0
        assert k.count("if (issue_t0 >= rows) return;") == 1
        assert k.count("ring_end(ring, issued, stages, a.status);") == waits
    # one thread arms (and waits) alone where rows are aligned in the backward, else a whole warp does
    assert "const bool issuer = BULK && threadIdx.x < (VEC ? 1 : 32) && threadIdx.y == 0;" in kernels[1]
    assert kernels[1].index("issue_only_after(ring_wait") > kernels[1].index("if (BULK && VEC) {")


def test_elements_stored_by_hand_are_ordered_before_the_arrive():
    """loose_row stores the elements of a tensor's partial granules lane by lane, and lane 0 arrives for the warp: only
    __syncwarp orders the one before the other (a reduction gathers the lanes without ordering their stores)."""
    text = re.sub(r"//[^\n]*", "", (_build.CSRC / "block_norm.cu").read_text())
    found = 0
    for m in re.finditer(r"loose_row<T>\(dst", text):
        before_arrive = text[m.end():].split("mbar_arrive_expect_tx(", 1)[0]
        assert re.search(r"__syncwarp\(\);\s*if \(lane == 0\) $", before_arrive)
        found += 1
    assert found == 2
