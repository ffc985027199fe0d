"""Waits that give up: the warp's own waits (compiled for the host with a wait that runs out at a
chosen call), and that no role of the chunk kernels which works as a warp waits lane by lane."""

import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_decode_attention_gqa_gb300", "csrc")

# a kernel's loop over pieces and tiles with lane 0 .. 31 run one after the other is not possible
# on the host; one lane whose vote is scripted is: vote[i] is the whole warp's answer to wait i
HOST = r"""
#include <stdint.h>
#include <stdio.h>
#define __device__
#define __forceinline__ inline
static int waits = 0, votes = 0, fail_at = 0, lane_sees = 1;
static bool mbar_wait(uint64_t*, uint32_t, unsigned int*, unsigned int) { ++waits; return lane_sees != 0; }
static int __all_sync(unsigned int mask, bool x) {
  ++votes;
  return mask == 0xffffffffu && x && votes != fail_at;
}
#include "warp_wait.cuh"
int main() {
  unsigned int err = 0;
  uint64_t bar = 0;
  for (lane_sees = 0; lane_sees < 2; ++lane_sees)
    for (fail_at = 1; fail_at < 6; ++fail_at) {
      waits = votes = 0;
      skv::WarpWait wait(&err);
      int taken = 0;
      for (int piece = 0; piece < 3; ++piece)
        for (int tile = 0; tile < 4; ++tile) {
          if (!wait(&bar, tile & 1, 1u)) break;
          ++taken;
        }
      const int first = lane_sees ? fail_at : 1;  // the first wait that the warp gives up
      if (waits != first || votes != first || taken != first - 1 || wait.ok) {
        printf("sees %d fail %d: %d waits, %d votes, %d taken\n", lane_sees, fail_at, waits, votes, taken);
        return 1;
      }
    }
  return 0;
}
"""


def test_a_warp_that_gave_up_waits_no_more(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "w.cpp", tmp_path / "w"
    src.write_text(HOST)
    subprocess.run([cxx, "-std=c++17", "-Wno-unknown-pragmas", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


# Roles in which a lane may wait by itself: the last copies of a loader, and lane 0 of the loader of
# chunk_rows, whose answer the other lanes take from it.
ALONE = {"chunk_rows.cu": 2, "chunk_tc.cu": 2, "qk_norm_rope.cu": 1}


@pytest.mark.parametrize("name", ALONE)
def test_waits_are_the_warps(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    calls = [m.start() for m in re.finditer(r"\bmbar_wait\(", text)]
    alone = 0
    for at in calls:
        statement = text[max(text.rfind(";", 0, at), text.rfind("{", 0, at)) + 1:text.index(";", at)]
        if re.search(r"__all_sync\(0xffffffffu,[^;]*mbar_wait\(", statement):
            continue
        after = text[at:at + 400]
        voted = re.search(r"ok = __all_sync\(0xffffffffu, ok\)", after) and "break" not in after[:after.index("ok = __all_sync")]
        if voted:  # both waits of the statement before the vote
            continue
        assert "kDevErrDrainWait" in statement or "x < NSTAGE ||" in statement, statement.strip()
        alone += 1
    assert alone == ALONE[name]
