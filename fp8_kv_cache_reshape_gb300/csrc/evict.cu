// kvq_evict_tokens: cut each sequence's cache to its heaviest tokens.
//
// Two kernels.  Selection: per (sequence, KV head), the n - s - r largest of
// the L - s - r weights between the protected first s and last r tokens, ties
// to the lowest position: a radix selection of the threshold (11, 11 and 10
// bits of an order-preserving integer image of the weight), then an ordered
// compaction of the positions.  Move: the kept tokens' K rows and V columns
// are copied into the destination pages.
#include <cooperative_groups.h>

#include "kvq_device.cuh"
#include "kvq_host.h"

namespace kvq {

namespace {

namespace cg = cooperative_groups;

struct EvictParams {
  const float* weights;
  int64_t weights_stride;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int64_t k_str, v_str;  // bytes between consecutive (block, KV head) pages of each cache
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* keep_lens;
  const int32_t* dst_table;
  float* dst_weights;
  int64_t dst_stride;
  int32_t* dst_lens;
  int32_t* kept;  // [B][Hkv][max_dst * P] source positions, ascending
  int Hkv, max_blocks, max_dst;
  int64_t num_blocks;
  int sink, recent;
  int seg_cap;  // keys of a CTA's segment held in shared memory (0: read from global memory each pass)
  int* dev_status;
};

// ------------------------------------------------------------- selection ---
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;

// Order-preserving image of a weight: a < b <=> image(a) < image(b); the two
// zeros are equal, NaN ranks below everything.
KVQ_DEVINL uint32_t weight_key(float x) {
  uint32_t u = __float_as_uint(x);
  if (x != x) return 0u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// What sequence b keeps: L tokens cut to n, of which the first s and the last
// r are protected.
struct Cut {
  int L, n, s, r;
};
KVQ_DEVINL Cut cut_of(const EvictParams& p, int b, bool report) {
  Cut c;
  c.L = p.seq_lens[b];
  const int cap = p.max_blocks * kPage, dst_cap = p.max_dst * kPage;
  bool bad = false;
  if (c.L < 0 || c.L > cap) {
    bad = true;
    c.L = c.L < 0 ? 0 : cap;
  }
  int keep = p.keep_lens[b];
  if (keep < 0) {
    bad = true;
    keep = 0;
  }
  c.n = min(c.L, keep);
  if (c.n > dst_cap) {
    bad = true;
    c.n = dst_cap;
  }
  if (bad && report) set_status(p.dev_status, KVQ_DEV_BAD_SEQLEN);
  c.s = min(p.sink, c.n);
  c.r = min(p.recent, c.n - c.s);
  return c;
}

// Exclusive prefix over the warp of x; total in the last argument.
KVQ_DEVINL int warp_scan_excl(int x, int lane, int& total) {
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  total = __shfl_sync(0xffffffffu, v, 31);
  return v - x;
}

// Grid (cluster size, Hkv, B), one cluster per (sequence, KV head): CTA k of C
// owns the k-th of C equal segments of the candidate positions.  Histograms
// and counts meet through distributed shared memory.  Bound by latency:
// four cluster barriers (eight in clusters of more than two) and three passes
// over the segment, 16 us for 64 pairs of 20K candidates (their 5.2 MB of weights
// would take 0.8 us).
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t held_k[];  // [seg_cap] the segment's keys
  __shared__ __align__(8) uint32_t hist[3][kBins];  // counts, one histogram per pass
  __shared__ int warp_gt[kSelWarps], warp_eq[kSelWarps];
  __shared__ int2 totals[kMaxCluster];  // each CTA's counts above and at the threshold
  __shared__ uint32_t found[3][2];      // per pass: chosen bin, keys still needed inside it
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  grid_dependency_wait();
  const Cut cut = cut_of(p, b, tid == 0 && rank == 0 && h == 0);
  const size_t pair = static_cast<size_t>(b) * p.Hkv + h;
  const float* w = p.weights + pair * p.weights_stride;
  float* dw = p.dst_weights + pair * p.dst_stride;
  int32_t* kept = p.kept + pair * p.max_dst * kPage;
  const int N = cut.L - cut.r - cut.s;   // candidates
  const int m = cut.n - cut.r - cut.s;   // chosen among them
  if (rank == 0 && h == 0 && tid == 0) p.dst_lens[b] = cut.n;
  // the protected ends, and zeros behind the kept tokens: thread i of n
  auto ends = [&](int i, int n) {
    for (int j = i; j < cut.s; j += n) {
      kept[j] = j;
      dw[j] = w[j];
    }
    for (int j = i; j < cut.r; j += n) {
      const int src = cut.L - cut.r + j, pos = cut.n - cut.r + j;
      kept[pos] = src;
      dw[pos] = w[src];
    }
    for (int64_t j = cut.n + i; j < p.dst_stride; j += n) dw[j] = 0.f;
  };
  const int gtid = rank * kSelThreads + tid, gthreads = C * kSelThreads;
  if (m <= 0 || m == N) ends(gtid, gthreads);
  if (m <= 0) return;  // uniform over the cluster
  if (m == N) {
    for (int i = gtid; i < N; i += gthreads) {
      kept[cut.s + i] = cut.s + i;
      dw[cut.s + i] = w[cut.s + i];
    }
    return;
  }
  const int seg = (N + C - 1) / C;
  const int i0 = min(N, rank * seg), i1 = min(N, i0 + seg), len = i1 - i0;
  const float* wseg = w + cut.s + i0;
  const bool held = len <= p.seg_cap;
  for (int i = tid; i < 3 * kBins; i += kSelThreads) hist[0][i] = 0;
  __syncthreads();
  const bool lead = C > 2;  // see the passes
  if (lead) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  // the keys, and their first digit's histogram on the way
#pragma unroll 8
  for (int i = tid; i < len; i += kSelThreads) {
    const uint32_t k = weight_key(wseg[i]);
    if (held) held_k[i] = k;
    atomicAdd(&hist[0][k >> 21], 1u);
  }
  auto key_at = [&](int i) { return held ? held_k[i] : weight_key(wseg[i]); };
  if (lead) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the leader's histograms are zeroed

  // threshold: the m-th largest key, digit by digit from the top.  In a pair of
  // CTAs each adds the other's counts to its own and finds the digit for itself,
  // with one barrier a pass (8 x 20K: 73.6 us a call, 75.0 with a leader).  In a
  // larger cluster the others add their counts (bins that hold any: few) to the
  // leader's histogram, and it finds the digit and hands it out (128K in clusters
  // of eight: 51.1 us a call; every CTA reading all the histograms: 54.6).
  uint32_t prefix = 0, mask = 0;
  int need = m;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass < 2 ? 2048 : 1024;
    if (pass) {
      auto add = [&](uint32_t k) {
        if ((k & mask) == prefix) atomicAdd(&hist[pass][(k >> shift) & (bins - 1)], 1u);
      };
      if (held) {
        const int quads = len >> 2;
#pragma unroll 2
        for (int i = tid; i < quads; i += kSelThreads) {
          const uint4 k = reinterpret_cast<const uint4*>(held_k)[i];
          add(k.x);
          add(k.y);
          add(k.z);
          add(k.w);
        }
        for (int i = 4 * quads + tid; i < len; i += kSelThreads) add(held_k[i]);
      } else {
#pragma unroll 4
        for (int i = tid; i < len; i += kSelThreads) add(weight_key(wseg[i]));
      }
    }
    if (lead && rank != 0) {
      __syncthreads();
      uint32_t* theirs = cluster.map_shared_rank(&hist[pass][0], 0);
      for (int i = tid; i < bins; i += kSelThreads) {
        const uint32_t c = hist[pass][i];
        if (c) atomicAdd(theirs + i, c);
      }
    }
    if (C == 1) __syncthreads();
    else cluster.sync();
    if (!lead || rank == 0) {
      // bin pairs from the top: thread t sums bins kBins - 1 - 2t and the one below
      const int hi = kBins - 1 - 2 * tid;
      uint2 c = *reinterpret_cast<const uint2*>(&hist[pass][hi - 1]);
      if (C == 2) {
        const uint2 o = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&hist[pass][hi - 1], rank ^ 1));
        c.x += o.x;
        c.y += o.y;
      }
      int tot;
      const int excl = warp_scan_excl(static_cast<int>(c.x + c.y), lane, tot);
      if (lane == 0) warp_gt[wid] = tot;
      __syncthreads();
      int all;
      const int wx = warp_scan_excl(warp_gt[lane], lane, all);
      const int before = excl + __shfl_sync(0xffffffffu, wx, wid);
      if (before < need && before + static_cast<int>(c.x + c.y) >= need) {  // exactly one thread
        const bool first = before + static_cast<int>(c.y) >= need;
        const uint32_t bin = first ? hi : hi - 1, left = need - (first ? before : before + static_cast<int>(c.y));
        found[pass][0] = bin;
        found[pass][1] = left;
        for (int k = 1; lead && k < C; ++k) {
          uint32_t* f = cluster.map_shared_rank(&found[pass][0], k);
          f[0] = bin;
          f[1] = left;
        }
      }
    }
    if (lead) cluster.sync();
    else __syncthreads();
    prefix |= found[pass][0] << shift;
    mask |= static_cast<uint32_t>(bins - 1) << shift;
    need = static_cast<int>(found[pass][1]);
  }
  // prefix is the threshold; of the keys equal to it the first `need` are taken.
  // A warp takes a run of the segment, each lane four neighbours at a time.
  const int sub = (((len + kSelWarps - 1) / kSelWarps) + 127) / 128 * 128;
  const int j0 = min(len, wid * sub), j1 = min(len, j0 + sub);
  auto keys4 = [&](int i, uint32_t (&k)[4]) {  // keys i .. i + 3 (0, and not counted, past the run)
    if (held && i + 4 <= j1) {
      const uint4 v = *reinterpret_cast<const uint4*>(held_k + i);
      k[0] = v.x;
      k[1] = v.y;
      k[2] = v.z;
      k[3] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) k[e] = i + e < j1 ? key_at(i + e) : 0u;
    }
  };
  auto is_eq = [&](int i, int e, uint32_t k) { return k == prefix && i + e < j1; };
  int gt = 0, eq = 0;
  for (int j = j0; j < j1; j += 128) {
    const int i = j + 4 * lane;
    uint32_t k[4];
    keys4(i, k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gt += k[e] > prefix;
      eq += is_eq(i, e, k[e]);
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    warp_gt[wid] = gt;
    warp_eq[wid] = eq;
  }
  __syncthreads();
  int gt_all, eq_all;
  const int gx = warp_scan_excl(warp_gt[lane], lane, gt_all), ex = warp_scan_excl(warp_eq[lane], lane, eq_all);
  int gt_before = __shfl_sync(0xffffffffu, gx, wid), eq_before = __shfl_sync(0xffffffffu, ex, wid);
  if (C > 1) {
    if (tid < C) *cluster.map_shared_rank(&totals[rank], tid) = make_int2(gt_all, eq_all);
    cluster.sync();  // the last access to another CTA's memory is behind it
    const int2 other = lane < rank ? totals[lane] : make_int2(0, 0);  // at most 8 CTAs
    gt_before += __reduce_add_sync(0xffffffffu, other.x);
    eq_before += __reduce_add_sync(0xffffffffu, other.y);
  }
  // stores to global memory only after the last barrier, which would wait for them
  ends(gtid, gthreads);
  for (int j = j0; j < j1; j += 128) {
    const int i = j + 4 * lane;
    uint32_t k[4];
    keys4(i, k);
    int g = 0, q = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      g += k[e] > prefix;
      q += is_eq(i, e, k[e]);
    }
    int both;  // counts of the lanes before this one: at most 128 each
    const int before = warp_scan_excl(g | (q << 16), lane, both);
    int gp = gt_before + (before & 0xFFFF), qp = eq_before + (before >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool is_g = k[e] > prefix, is_q = is_eq(i, e, k[e]);
      if (is_g || (is_q && qp < need)) {
        const int pos = cut.s + gp + min(qp, need);
        kept[pos] = cut.s + i0 + i + e;
        // the weight back from its key; what the key does not tell (which zero,
        // which NaN) is read again
        const uint32_t u = (k[e] & 0x80000000u) ? (k[e] & 0x7FFFFFFFu) : ~k[e];
        dw[pos] = (k[e] == 0u || k[e] == 0x80000000u) ? wseg[i + e] : __uint_as_float(u);
      }
      gp += is_g;
      qp += is_q;
    }
    gt_before += both & 0xFFFF;
    eq_before += both >> 16;
  }
}

// ------------------------------------------------------------------ move ---
constexpr int kMoveWarps = 4;
KVQ_DEVINL void load16(const uint8_t* src, uint32_t* w) {
  const uint4 v = __ldcg(reinterpret_cast<const uint4*>(src));
  w[0] = v.x;
  w[1] = v.y;
  w[2] = v.z;
  w[3] = v.w;
}

// One warp per (sequence, KV head, destination page).  K: 16-byte chunks, row
// by row, each swizzled for its source and its destination row.  V: the lanes
// hold the rows (dimensions) of one source page at a time, read whole, and put
// the kept tokens' bytes into their destination rows with byte permutes.
// (Reading one 32-bit word per row and token instead touches every sector as
// often as the page holds kept tokens: 80 against 64 us for 8 x 20K to 8K when
// it was tried.)  Bound by DRAM: 8 x 20K to 8K reads nearly every V page and 0.4
// of the K rows, 333 MB with what it writes, in 59 us (5.7 TB/s).  Two warps per
// page (79 to 85 us a call), and prefetches of the V pages into L2 during the
// selection (80 to 85) or one page ahead, gained nothing.
template <int D, int ESZ, bool PT>
__global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int ROWB = D * ESZ;
  constexpr int CH = ROWB / 16;           // chunks per K row
  constexpr int PAGE_BYTES = kPage * ROWB;
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y, b = blockIdx.z;
  const int page = blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  // the length, the destination page and the tokens' positions in one round trip
  if (page >= p.max_dst) return;
  const size_t pair = static_cast<size_t>(b) * p.Hkv + h;
  const int n = __ldcg(p.dst_lens + b);
  const int dst_blk = __ldg(p.dst_table + static_cast<size_t>(b) * p.max_dst + page);
  const int pos = lane < kPage ? __ldcg(p.kept + pair * p.max_dst * kPage + page * kPage + lane) : 0;
  if (page * kPage >= n) return;
  if (dst_blk < 0 || static_cast<int64_t>(dst_blk) >= p.num_blocks) {
    if (lane == 0) set_status(p.dev_status, KVQ_DEV_BAD_BLOCK);
    return;
  }
  // lane t < 16: token t's source page (block * Hkv + h) and offset in it
  int64_t src_page = -1;
  int src_off = 0;
  if (lane < kPage && page * kPage + lane < n) {
    const int blk = __ldg(p.block_table + static_cast<size_t>(b) * p.max_blocks + pos / kPage);
    src_off = pos % kPage;
    if (blk < 0 || static_cast<int64_t>(blk) >= p.num_blocks)
      set_status(p.dev_status, KVQ_DEV_BAD_BLOCK);
    else
      src_page = static_cast<int64_t>(blk) * p.Hkv + h;
  }
  const uint32_t live = __ballot_sync(0xffffffffu, src_page >= 0);
  // this lane's token in its pages: the V row slot it is read from, and the pages
  const int from_slot = ESZ == 1 ? fp8_v_slot(src_off) : src_off;
  const uint8_t* k_src = p.k_cache + max(src_page, int64_t(0)) * p.k_str;
  const uint8_t* v_src = p.v_cache + max(src_page, int64_t(0)) * p.v_str;
  auto shfl_ptr = [](const uint8_t* x, int t) {
    return reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(x), t));
  };
  const int64_t dst_page = static_cast<int64_t>(dst_blk) * p.Hkv + h;
  auto k_off = [](int t, int j) { return ESZ == 1 ? fp8_k_offset(t, j, D) : k_chunk_offset(t, j, ROWB); };
  uint8_t* kd = p.k_cache + dst_page * p.k_str;
  uint8_t* vd = p.v_cache + dst_page * p.v_str;
  // first tokens of each source page, in order
  const int64_t prev = __shfl_up_sync(0xffffffffu, src_page, 1);
  const uint32_t heads = __ballot_sync(0xffffffffu, src_page >= 0 && (lane == 0 || src_page != prev));
  constexpr int KU = kPage * CH / 32;
  uint4 kk[KU];
#pragma unroll
  for (int u = 0; u < KU; ++u) {
    const int t = (u * 32 + lane) / CH, j = (u * 32 + lane) % CH;
    const int so = __shfl_sync(0xffffffffu, src_off, t);
    kk[u] = __ldcg(reinterpret_cast<const uint4*>(shfl_ptr(k_src, t) + k_off(so, j)));
  }
  auto store_k = [&]() {
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const int t = (u * 32 + lane) / CH, j = (u * 32 + lane) % CH;
      if ((live >> t) & 1) *reinterpret_cast<uint4*>(kd + k_off(t, j)) = kk[u];
    }
  };
  if constexpr (ESZ == 2) store_k();  // twice the registers: not held beside V
  constexpr int WORDS = kPage * ESZ / 4;  // 32-bit words of a V row
  constexpr int VEC = WORDS / 4;          // 16-byte pieces of a V row
  constexpr int RPL = D / 32 < 4 / VEC ? D / 32 : 4 / VEC;  // rows per lane at a time
#pragma unroll 1
  for (int d0 = lane; d0 < D; d0 += 32 * RPL) {
    uint32_t row[RPL][WORDS], cur[RPL][WORDS], nxt[RPL][WORDS];
    auto load_page = [&](uint32_t from) {  // of the first token in `from`, into nxt
      if (!from) return;  // uniform
      const uint8_t* src = shfl_ptr(v_src, __ffs(from) - 1);
#pragma unroll
      for (int i = 0; i < RPL; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) load16(src + (d0 + 32 * i) * kPage * ESZ + 16 * v, &nxt[i][4 * v]);
    };
    load_page(heads);
    if (ESZ == 1 && d0 == lane) store_k();
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
      if (live != 0xFFFFu) {  // slots of other tokens stay
#pragma unroll
        for (int v = 0; v < VEC; ++v) load16(vd + (d0 + 32 * i) * kPage * ESZ + 16 * v, &row[i][4 * v]);
      } else {
#pragma unroll
        for (int w = 0; w < WORDS; ++w) row[i][w] = 0u;
      }
    }
#pragma unroll
    for (int t = 0; t < kPage; ++t) {
      const int so = __shfl_sync(0xffffffffu, from_slot, t);
      if (!((live >> t) & 1)) continue;  // uniform
      if ((heads >> t) & 1) {  // the next page's rows are under way while this one's are used
#pragma unroll
        for (int i = 0; i < RPL; ++i)
#pragma unroll
          for (int w = 0; w < WORDS; ++w) cur[i][w] = nxt[i][w];
        load_page(heads & ~((2u << t) - 1u));
      }
#pragma unroll
      for (int i = 0; i < RPL; ++i) {
        if constexpr (ESZ == 1) {
          const int from = so, to = fp8_v_slot(t);  // `to` at compile time
          const uint32_t a = (from & 4) ? cur[i][1] : cur[i][0], b2 = (from & 4) ? cur[i][3] : cur[i][2];
          const uint32_t word = (from & 8) ? b2 : a;
          const uint32_t sel = (0x3210u & ~(0xFu << (4 * (to & 3)))) | ((4u + (from & 3)) << (4 * (to & 3)));
          row[i][to >> 2] = __byte_perm(row[i][to >> 2], word, sel);
        } else {
          // the halves of a row swap with its dimension, alike in source and destination
          const bool swap = ((d0 + 32 * i) >> 2) & 1;
          const int wf = (so >> 1) & 3;
          const bool upper = (so >= 8) != swap;
          const uint32_t lo = (wf & 2) ? ((wf & 1) ? cur[i][3] : cur[i][2]) : ((wf & 1) ? cur[i][1] : cur[i][0]);
          const uint32_t hi = (wf & 2) ? ((wf & 1) ? cur[i][7] : cur[i][6]) : ((wf & 1) ? cur[i][5] : cur[i][4]);
          const uint32_t word = upper ? hi : lo;
          const uint32_t pair_sel = (so & 1) ? 0x76u : 0x54u;
          const uint32_t sel = (t & 1) ? (0x0010u | (pair_sel << 8)) : (0x3200u | pair_sel);
          if (swap) row[i][(t >> 1) ^ 4] = __byte_perm(row[i][(t >> 1) ^ 4], word, sel);
          else row[i][t >> 1] = __byte_perm(row[i][t >> 1], word, sel);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RPL; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        *reinterpret_cast<uint4*>(vd + (d0 + 32 * i) * kPage * ESZ + 16 * v) =
            make_uint4(row[i][4 * v], row[i][4 * v + 1], row[i][4 * v + 2], row[i][4 * v + 3]);
  }
  if constexpr (PT) {
    if (src_page >= 0) {
      const float* st = reinterpret_cast<const float*>(v_src + PAGE_BYTES);
      float* dt = reinterpret_cast<float*>(vd + PAGE_BYTES);
      dt[lane] = st[src_off];
      dt[kPage + lane] = st[kPage + src_off];
    }
  }
}

constexpr int kKeysMax = 48 * 1024;  // keys a CTA holds in shared memory (192 KiB)

// CTAs per (sequence, KV head): clusters as large as the GPU holds at once (a
// CTA fills an SM; further waves cost a whole selection each), with at least
// 2,048 candidates per CTA (1,024 or 8,192 instead: the same within 2 us).  Two
// CTAs to an SM and clusters of up to 16 were slower: the barriers of a
// selection cost more in a larger cluster (128K tokens 60 against 52.5 us a
// call, 8 x 20K 81.5 against 75.8).
int select_cluster(int64_t tokens, int64_t pairs) {
  int c = 1;
  while (c < kMaxCluster && 2 * c * pairs <= sm_count() && tokens >= 4096ll * c) c *= 2;
  return c;
}

template <int D, int ESZ, bool PT>
cudaError_t launch_move(cudaLaunchConfig_t cfg, const EvictParams& p) {
  return cudaLaunchKernelEx(&cfg, evict_move_kernel<D, ESZ, PT>, p);
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace

}  // namespace kvq

using namespace kvq;

extern "C" kvq_status_t kvq_evict_tokens(const float* weights, int64_t weights_stride, void* k_cache, void* v_cache,
                                         const int32_t* block_table, const int32_t* seq_lens,
                                         const int32_t* keep_lens, const int32_t* dst_block_table, float* dst_weights,
                                         int64_t dst_weights_stride, int32_t* dst_seq_lens, int32_t* kept, int B,
                                         int Hkv, int D, int P, int max_blocks, int max_dst_blocks, int64_t num_blocks,
                                         int sink, int recent, kvq_dtype_t cache_dtype, int per_token, int* dev_status,
                                         kvq_stream_t stream) {
  clear_error();
  if (B < 1 || Hkv < 1 || max_blocks < 1 || max_dst_blocks < 1 || num_blocks < 1)
    return fail(KVQ_ERR_INVALID_ARG, "evict_tokens: bad sizes");
  if (sink < 0 || recent < 0) return fail(KVQ_ERR_INVALID_ARG, "evict_tokens: sink and recent must be >= 0");
  if (P != kPage) return fail(KVQ_ERR_UNSUPPORTED, "evict_tokens: page size %d (only 16)", P);
  if (cache_dtype != KVQ_DTYPE_FP8_E4M3 && cache_dtype != KVQ_DTYPE_FP8_E5M2 && cache_dtype != KVQ_DTYPE_BF16)
    return fail(KVQ_ERR_INVALID_ARG, "evict_tokens: bad cache dtype");
  const bool fp8 = cache_dtype != KVQ_DTYPE_BF16;
  if (per_token && !fp8) return fail(KVQ_ERR_INVALID_ARG, "evict_tokens: per-token scales need an FP8 cache");
  if (D != 64 && D != 128 && !(fp8 && !per_token && D == 256))
    return fail(KVQ_ERR_UNSUPPORTED, "evict_tokens: head_dim %d (64 or 128; 256 for FP8 with per-head scales)", D);
  if (B > 65535 || Hkv > 65535) return fail(KVQ_ERR_UNSUPPORTED, "evict_tokens: grid too large");
  const int64_t cap = static_cast<int64_t>(max_blocks) * P, dst_cap = static_cast<int64_t>(max_dst_blocks) * P;
  if (cap > 0x7FFFFFFFll - 65536 || dst_cap > 0x7FFFFFFFll - 65536)
    return fail(KVQ_ERR_UNSUPPORTED, "evict_tokens: block table too long");
  if (weights_stride < cap || dst_weights_stride < dst_cap)
    return fail(KVQ_ERR_INVALID_ARG, "evict_tokens: a weights row is shorter than its block table");
  if (!weights || !k_cache || !v_cache || !block_table || !seq_lens || !keep_lens || !dst_block_table || !dst_weights ||
      !dst_seq_lens || !kept)
    return fail(KVQ_ERR_INVALID_ARG, "evict_tokens: null pointer");
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(weights, 4) || !aligned(dst_weights, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(keep_lens, 4) || !aligned(dst_block_table, 4) ||
      !aligned(dst_seq_lens, 4) || !aligned(kept, 4))
    return fail(KVQ_ERR_INVALID_ARG, "evict_tokens: misaligned pointer");
  const size_t pairs = static_cast<size_t>(B) * Hkv;
  if (overlap(weights, pairs * weights_stride * 4, dst_weights, pairs * dst_weights_stride * 4) ||
      overlap(seq_lens, size_t(B) * 4, dst_seq_lens, size_t(B) * 4) ||
      overlap(keep_lens, size_t(B) * 4, dst_seq_lens, size_t(B) * 4))
    return fail(KVQ_ERR_INVALID_ARG, "evict_tokens: an output overlaps an input");
  EvictParams p;
  p.weights = weights;
  p.weights_stride = weights_stride;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  const int64_t page_b = static_cast<int64_t>(kPage) * D * (fp8 ? 1 : 2);
  const PageStrides ps = page_strides(k_cache, v_cache, page_b, page_b + (per_token ? kScaleTailBytes : 0));
  p.k_str = ps.k;
  p.v_str = ps.v;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.keep_lens = keep_lens;
  p.dst_table = dst_block_table;
  p.dst_weights = dst_weights;
  p.dst_stride = dst_weights_stride;
  p.dst_lens = dst_seq_lens;
  p.kept = kept;
  p.Hkv = Hkv;
  p.max_blocks = max_blocks;
  p.max_dst = max_dst_blocks;
  p.num_blocks = num_blocks;
  p.sink = sink;
  p.recent = recent;
  p.dev_status = dev_status;
  const int C = select_cluster(cap, static_cast<int64_t>(B) * Hkv);
  const int64_t seg = (cap + C - 1) / C;
  p.seg_cap = seg <= kKeysMax ? static_cast<int>(seg) : 0;
  static int configured_mask = 0;  // devices whose attribute is set
  int dev = 0;
  cudaGetDevice(&dev);
  if (!(configured_mask & (1 << (dev & 31)))) {
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysMax * 4);
    if (e != cudaSuccess) return cuda_status(e, "evict_tokens: set shared memory size");
    configured_mask |= 1 << (dev & 31);
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, Hkv, B);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.seg_cap) * 4;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
  if (e != cudaSuccess) return cuda_status(e, "evict_tokens select launch");
  cfg.gridDim = dim3((max_dst_blocks + kMoveWarps - 1) / kMoveWarps, Hkv, B);
  cfg.blockDim = dim3(kMoveWarps * 32);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  if (!fp8)
    e = D == 128 ? launch_move<128, 2, false>(cfg, p) : launch_move<64, 2, false>(cfg, p);
  else if (per_token)
    e = D == 128 ? launch_move<128, 1, true>(cfg, p) : launch_move<64, 1, true>(cfg, p);
  else
    e = D == 256   ? launch_move<256, 1, false>(cfg, p)
        : D == 128 ? launch_move<128, 1, false>(cfg, p)
                   : launch_move<64, 1, false>(cfg, p);
  return cuda_status(e, "evict_tokens move launch");
}
