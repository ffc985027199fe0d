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


def test_the_append_ring_is_handed_back_by_what_was_read():
    """A stage's arrival needs the sum over its heads (arrive_after), not only to stand behind the loads."""
    text = open(os.path.join(CSRC, "qk_norm_rope.cu")).read()
    assert "mbar_arrive(&empty" not in text and text.count("arrive_after(&empty[s], ss)") == 1
