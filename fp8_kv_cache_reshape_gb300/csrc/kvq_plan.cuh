// The wide balanced plan: the pages of up to kWideBatch sequences laid end to
// end and cut into equal slots (shared by the decode partials and their merge).
#pragma once

#include "kvq_device.cuh"

namespace kvq {

constexpr int kWideBatch = 256;
constexpr int kWidePages = 4;  // least pages per slot, where that leaves a slot per sequence
constexpr int kPartialWarps = 4;  // partials of a segment: one per consumer warp of the decode kernel

// seq_lens[b] clamped to the block table; spec: read before the preceding
// kernel has completed (a hint) or beside it (L2 only: no stale line); otherwise
// after a wait or a fence of the reader's own.
KVQ_DEVINL int wide_len(const int32_t* seq_lens, int b, int max_blocks, bool spec) {
  const int L = spec ? ld_l2only_s32(seq_lens + b) : seq_lens[b];
  return min(max(L, 0), max_blocks * kPage);
}
// Lane i holds the pages of sequences [i * per, (i + 1) * per).
struct WideScan {
  int per, excl, incl, total;
};
KVQ_DEVINL WideScan wide_scan(const int32_t* seq_lens, int B, int max_blocks, int lane, bool spec) {
  WideScan w;
  w.per = (B + 31) / 32;
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kWideBatch / 32; ++i) {
    const int b = lane * w.per + i;
    if (i < w.per && b < B) sum += (wide_len(seq_lens, b, max_blocks, spec) + kPage - 1) / kPage;
  }
  int x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  w.incl = x;
  w.excl = x - sum;
  w.total = __shfl_sync(0xffffffffu, x, 31);
  return w;
}
// Slots that hold pages: of a batch of short sequences as many as sequences (a
// segment costs about 2 us whatever its length).
__host__ __device__ __forceinline__ int wide_slots(int num_slots, int B, int total) {
  int n = (total + kWidePages - 1) / kWidePages;
  const int seqs = B < total ? B : total;
  if (n < seqs) n = seqs;
  return n < num_slots ? n : num_slots;
}
// The sequence b that stream page `pos` (< total) lies in, or an empty one
// before it, and b's first stream page.
KVQ_DEVINL void wide_find(const int32_t* seq_lens, int B, int max_blocks, const WideScan& w, int pos, int lane, bool spec,
                          int& b, int& start) {
  const int at = __popc(__ballot_sync(0xffffffffu, w.incl <= pos)) & 31;  // the lane whose sequences hold pos
  b = at * w.per;
  start = __shfl_sync(0xffffffffu, w.excl, at);
  // pages of that lane's sequences, one per lane
  const bool mine = lane < w.per && b + lane < B;
  int x = mine ? (wide_len(seq_lens, b + lane, max_blocks, spec) + kPage - 1) / kPage : 0;
  const int pages = x;
#pragma unroll
  for (int o = 1; o < kWideBatch / 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  const int skip = __popc(__ballot_sync(0xffffffffu, mine && start + x <= pos));  // whole sequences before pos
  const int from = __shfl_sync(0xffffffffu, x - pages, skip & 31);
  b += skip;
  start += from;
}
// Sequence b's first stream page and page count.
KVQ_DEVINL void wide_locate(const int32_t* seq_lens, int B, int max_blocks, const WideScan& w, int b, int lane, int& start,
                            int& pages) {
  const int at = b / w.per, in = b - at * w.per;
  const int x = lane <= in ? (wide_len(seq_lens, at * w.per + lane, max_blocks, true) + kPage - 1) / kPage : 0;
  start = __shfl_sync(0xffffffffu, w.excl, at) + __reduce_add_sync(0xffffffffu, lane < in ? x : 0);
  pages = __shfl_sync(0xffffffffu, x, in);
}

}  // namespace kvq
