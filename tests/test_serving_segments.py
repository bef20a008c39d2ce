"""Slots of the shared-prefix kernel that hold several segments, on the CPU:
the batches that the GPU tests take do put several into a CTA, and what one
softmax warp still stages of a segment lies in no byte that another warp
writes for the next."""
import os
import shutil
import subprocess

import pytest

from oracle.kv_cache import FP8, FP8_E5M2
from tests.test_serving_plan import _groups, _prefix_plan

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_kv_cache_reshape_gb300", "csrc")

# 80 KV heads: one slot per head on a GPU of 80 to 159 SMs; 40: three or fewer
# prefixes, sequences per group, KV heads, group, head dim, dtype, segments of the fullest slot at least
SEGMENTS = {
    "part_tile_then_full": ([700, 900], [10, 32], 80, 4, 128, FP8, 2),
    "full_tile_then_part": ([900, 700], [32, 9], 80, 4, 128, FP8, 2),
    "two_tiles_then_one": ([500, 700], [60, 9], 80, 4, 128, FP8, 2),
    "one_tile_then_two": ([700, 500], [8, 60], 80, 4, 128, FP8_E5M2, 2),
    "a_warp_each": ([300, 640, 513, 1000], [8, 8, 8, 8], 80, 4, 128, FP8, 4),
    "three_tiles_then_part": ([260, 390], [81, 11], 80, 4, 128, FP8, 3),
    "empty_between": ([300, 0, 1, 200], [8, 3, 9, 17], 80, 4, 128, FP8, 3),
    "wide_group": ([700, 900, 257], [5, 16, 4], 80, 8, 128, FP8_E5M2, 3),
    "short_prefixes": ([384, 300, 400, 250, 300, 200, 300], [4, 5, 3, 4, 4, 3, 4], 40, 4, 128, FP8, 2),
    "part_tile_then_full_d64": ([700, 900], [10, 32], 80, 4, 64, FP8, 2),
    "two_tiles_then_one_d64": ([500, 700, 300], [60, 9, 33], 80, 4, 64, FP8_E5M2, 3),
}


def starts_of(sizes):
    return [sum(sizes[:i]) for i in range(len(sizes) + 1)]


def most_segments(prefixes, sizes, group, slots):
    """Segments with keys in the fullest slot."""
    at = starts_of(sizes)
    segs, _ = _prefix_plan(_groups(group, list(zip(at, at[1:])), prefixes), slots)
    count = {}
    for s, _, _, _, k0, k1 in segs.values():
        count[s] = count.get(s, 0) + (k1 > k0)
    return max(count.values())


@pytest.mark.parametrize("name", list(SEGMENTS))
def test_the_cases_give_a_slot_several_segments(name):
    prefixes, sizes, heads, group, _, _, least = SEGMENTS[name]
    for sms in range(132, 160):
        assert most_segments(prefixes, sizes, group, sms // heads) >= least


PROGRAM = """
#include <cstdio>
#include "kvq_prefix_smem.h"
template <int D> void show() {
  using G = kvq::PrefixSmem<D>;
  std::printf("%d %d %d %d\\n", D, G::OFF_K, G::OFF_VH_END, G::OFF_BAR);
  for (int x = 0; x < 2; ++x)
    for (int q = 0; q < 4; ++q) {
      for (int r = 0; r < 32; ++r) std::printf("%d ", G::stage_row(x, q, r));
      for (int t = 0; t < 2; ++t)
        for (int r = 0; r < 32; ++r) std::printf("%d ", G::q_row(x, t, 32 * q + r));
      std::printf("\\n");
    }
}
int main() { show<64>(); show<128>(); }
"""


def test_staged_rows_keep_to_their_warps_bytes(tmp_path):
    """Nothing orders a stream's softmax warps between a segment's staged output
    and the next segment's query rows, so no byte may be one warp's staging and
    another's query row or staging, nor anything the other roles write."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "m.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, "-o", str(tmp_path / "m"), str(tmp_path / "m.cpp")], check=True)
    lines = subprocess.run([str(tmp_path / "m")], check=True, capture_output=True, text=True).stdout.splitlines()
    for at in (0, 9):
        D, off_k, vh_end, off_bar = map(int, lines[at].split())
        owner = {}  # byte -> the softmax warp that writes it
        for warp, line in enumerate(lines[at + 1:at + 9]):
            rows = list(map(int, line.split()))
            staged = {b for r in rows[:32] for b in range(r, r + 128)}
            queries = {b for r in rows[32:] for b in range(r, r + D)}
            assert len(staged) == 32 * 128 and len(queries) == 64 * D
            assert all(r % 16 == 0 for r in rows)
            for b in staged | queries:
                assert owner.setdefault(b, warp) == warp
                assert b < off_k or vh_end <= b < off_bar
