"""Barriers in the kernels' sources: an aligned barrier counts a warp whose lanes have parted as a whole, so
each is used behind a __syncwarp() only."""

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_decode_attention_gqa_gb300", "csrc")


def test_every_aligned_barrier_follows_a_syncwarp():
    found = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = open(path).read()
        for m in re.finditer(r'asm volatile\("(bar\.sync|barrier\.)', text):
            found += 1
            before = [line.strip() for line in text[: m.start()].splitlines() if line.strip()]
            assert before[-1].startswith("__syncwarp();"), f"{os.path.basename(path)}: {m.group(0)} without a __syncwarp()"
    assert found >= 2
