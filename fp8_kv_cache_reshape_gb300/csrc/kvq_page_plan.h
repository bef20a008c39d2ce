// Integer plans of the kernels that walk tokens and pages: the tiles of the cache's
// writes and reads, and the 4-bit decode's page stream (plain C++: they are also
// checked on the host).
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define KVQ_PLAN __host__ __device__ __forceinline__
#else
#define KVQ_PLAN inline
#endif

namespace kvq {

constexpr int kPlanPage = 16;  // tokens per page

// ------------------------------------------------------------------ tiles ---
// A warp looks at the tokens of an aligned tile, 32 from 16 (tile - 1) on; the one
// of lane `lane`, in slot `slot`, is the tile's if its page's first token, were the
// page's tokens in order, is one of the first 16.
KVQ_PLAN bool tile_takes(int lane, int64_t slot) {
  return static_cast<unsigned>(lane - static_cast<int>(slot % kPlanPage)) < static_cast<unsigned>(kPlanPage);
}

// ------------------------------------------------- the decode's page stream ---
constexpr int kStreamWarps = 4;  // warps per CTA, a part each
constexpr int kMinPart = 2;      // pages of a part, at least: a pair

// Pages of a part, an even number: the stream in `parts` equal ones.
KVQ_PLAN int part_pages(int total, int parts) {
  const int n = ((total + parts - 1) / parts + 1) & ~1;
  return n > kMinPart ? n : kMinPart;
}
// Are the parts of the CTA that begins at c0 of the stream, more than one of them,
// all within pages [x0, x0 + n) of one (sequence, KV head)?  Then they leave one row of
// partials.
KVQ_PLAN bool parts_join(int c0, int chunk, int total, int x0, int n) {
  const int end = c0 + kStreamWarps * chunk, c1 = end < total ? end : total;
  return c1 - c0 > chunk && x0 <= c0 && c1 <= x0 + n;
}
// The rows of partials of a (sequence, KV head) with pages [x, x + n), n > 0, of a
// stream of `total`: row i was left by part part(i).  CTAs c0 .. c1 - 1 left one
// each, the parts before and behind them their own.
struct StreamRows {
  int first, last;       // parts; the same: the output was written there
  int lead, full, tail;  // part behind the joined CTAs
  int joined, count;
  KVQ_PLAN StreamRows(int x, int n, int total, int chunk) {
    first = x / chunk;
    last = (x + n - 1) / chunk;
    const int cta = kStreamWarps * chunk;
    const int c0 = (x + cta - 1) / cta;
    int c1 = (x + n) / cta;
    if (x + n == total && total - total / cta * cta > chunk) c1 = total / cta + 1;
    const bool any = c1 > c0;
    joined = kStreamWarps * c0;
    tail = kStreamWarps * c1;
    lead = any ? joined - first : last - first + 1;
    full = any ? c1 - c0 : 0;
    const int behind = last - tail + 1;
    count = lead + full + (any && behind > 0 ? behind : 0);
  }
  KVQ_PLAN int part(int i) const {
    return i < lead ? first + i : i < lead + full ? joined + kStreamWarps * (i - lead) : tail + i - lead - full;
  }
};

}  // namespace kvq
