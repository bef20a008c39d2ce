"""The kernels' own integer plans (kvq_page_plan.h), compiled for the host: the
tiles of the cache's writes and reads take every token once, and the 4-bit
decode's parts, walked as its warps do, leave exactly the rows of partials that
its joining reads."""
import os
import random
import shutil
import subprocess

import pytest

from tests.test_fp4_plan import pieces, spans
from tests.test_tile_tokens import tiles

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_kv_cache_reshape_gb300", "csrc")

PROGRAM = """
#include <cstdio>
#include "kvq_page_plan.h"
int main() {
  char what;
  while (std::scanf(" %c", &what) == 1) {
    long long a, b, c, d, e;
    if (what == 't') {  // lane, slot
      std::scanf("%lld %lld", &a, &b);
      std::printf("%d\\n", kvq::tile_takes(static_cast<int>(a), b));
    } else if (what == 'c') {  // total, parts
      std::scanf("%lld %lld", &a, &b);
      std::printf("%d\\n", kvq::part_pages(a, b));
    } else if (what == 'j') {
      std::scanf("%lld %lld %lld %lld %lld", &a, &b, &c, &d, &e);
      std::printf("%d\\n", kvq::parts_join(a, b, c, d, e));
    } else {
      std::scanf("%lld %lld %lld %lld", &a, &b, &c, &d);
      const kvq::StreamRows r(a, b, c, d);
      std::printf("%d %d", r.first, r.last);
      for (int i = 0; i < r.count; ++i) std::printf(" %d", r.part(i));
      std::printf("\\n");
    }
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """Questions to the compiled plan, a list of tuples, and its answers, a list of lists."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    at = tmp_path_factory.mktemp("plan")
    (at / "p.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, "-o", str(at / "p"),
                    str(at / "p.cpp")], check=True)

    def answer(questions):
        text = "\n".join(" ".join(map(str, q)) for q in questions)
        out = subprocess.run([str(at / "p")], input=text, check=True, capture_output=True, text=True).stdout.splitlines()
        assert len(out) == len(questions)
        return [[int(x) for x in line.split()] for line in out]

    return answer


def test_tiles(ask):
    """Which lane's token a tile takes, for every place in a page, and so the tiles of any slots."""
    slots = [*range(16), 2**31 + 5, 2**40, 2**62 + 15]
    found = ask([("t", lane, s) for s in slots for lane in range(32)])
    for i, s in enumerate(slots):
        assert [bool(x[0]) for x in found[32 * i:32 * i + 32]] == [0 <= lane - s % 16 < 16 for lane in range(32)]
    rng = random.Random(1)
    for T in (1, 17, 100):
        slots = [rng.randrange(0, 5000) for _ in range(T)]
        for tile, want in enumerate(tiles(slots)):
            at = [16 * (tile - 1) + lane for lane in range(32)]
            takes = ask([("t", lane, slots[t]) for lane, t in enumerate(at) if 0 <= t < T])
            assert [t for t, x in zip([t for t in at if 0 <= t < T], takes) if x[0]] == want


@pytest.mark.parametrize("seed", range(60))
def test_stream(ask, seed):
    rng = random.Random(seed)
    B, heads, sms = rng.choice([1, 2, 7, 40]), rng.choice([1, 2, 8]), rng.choice([1, 3, 152])
    cap = rng.choice([1, 5, 100, 1000])
    lens = [rng.choice([0, 1, 16, 17, rng.randint(0, cap * 16)]) for _ in range(B)]
    sp = spans(lens, rng.choice([-1, -1, 1, 40, 500]), cap)
    parts = min(12 * sms, (B * heads * cap + 1) // 2)
    total = heads * sum(n for _, n in sp)
    if total == 0:
        return
    chunk = ask([("c", total, parts)])[0][0]
    assert chunk % 2 == 0 and chunk * parts >= total
    walked = list(pieces(sp, heads, parts))  # (part, sequence, head, first page, pages)
    assert sum(p[-1] for p in walked) == total
    start, x = {}, 0
    for b, (_, n) in enumerate(sp):
        for h in range(heads):
            start[b, h] = (x, n)
            x += n
    # a CTA's warps, each by the piece that its part begins with
    first = {}
    for part, b, h, pg, n in walked:
        first.setdefault(part, (b, h))
    views = dict(zip(first, ask([("j", part // 4 * 4 * chunk, chunk, total, *start[first[part]]) for part in first])))
    left = {}
    for part, b, h, pg, n in walked:
        assert views[part] == views[part // 4 * 4]  # they agree
        if views[part][0]:
            assert first[part // 4 * 4] == (b, h)
            left.setdefault((b, h), set()).add(part // 4 * 4)
        elif n < sp[b][1]:
            left.setdefault((b, h), set()).add(part)
    keys = [key for key, (_, n) in start.items() if n]
    for key, (lo, hi, *rows) in zip(keys, ask([("r", *start[key], total, chunk) for key in keys])):
        if lo == hi:
            assert key not in left
        else:
            assert rows == sorted(left[key])


def test_the_largest_stream_stays_within_32_bits(ask):
    total = 0x7F000000  # the most that the call takes
    for parts in (12 * 152, 12 * 50):  # that long a stream has a part for each warp of the GPU
        chunk = ask([("c", total, parts)])[0][0]
        last = (total - 1) // chunk
        assert ask([("j", last // 4 * 4 * chunk, chunk, total, 0, total)])[0][0] in (0, 1)
        lo, hi, *rows = ask([("r", 0, total, total, chunk)])[0]
        assert (lo, hi) == (0, last) and rows[-1] <= last
