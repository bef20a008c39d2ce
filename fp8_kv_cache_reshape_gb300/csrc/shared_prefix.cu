// kvq_paged_decode_attention_shared_prefix: decode attention for groups of
// sequences that share a prefix.
//
// softmax over prefix and own tokens splits into partial results (output and
// log-sum-exp) that merge exactly: the sequences' own tokens run through the
// split-KV decode kernel; the prefix is contracted once per group with all
// its sequences' query heads as rows; a combine kernel merges both.
#include <cfloat>
#include <cmath>

#include "kvq_device.cuh"
#include "kvq_host.h"
#include "kvq_plan.cuh"
#include "kvq_prefix_smem.h"
#include "kvq_tcgen05.cuh"

namespace kvq {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int TR = kTileRows;   // query rows per tile
constexpr int TK = kTileKeys;   // keys per tile (8 pages)
constexpr int UNIT = 2 * TR;    // rows of a unit: two tiles over the same keys

struct SharedParams {
  const void* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* prefix_table;
  const int32_t* prefix_lens;
  const int32_t* group_starts;
  float* o_part;    // [Hkv][kseg][UNIT][D]
  float* lse_part;  // [Hkv][kseg][UNIT], log2 units
  int B, G, Hq, Hkv, g, max_prefix;
  int64_t num_blocks;
  float sm_scale;
  int64_t k_str, v_str;
  int slots;      // CTAs per KV head
  int max_units;  // bound of the batch's units
  int kseg;       // slots + max_units
  int* dev_status;
  int first;  // launched before the own tokens' grid
  // merge table, written by the prefix kernel: [B][g], see RowParts
  int4* parts;
  const int32_t* seq_lens;
  int max_blocks, own_slots;
  // failure-path test hook (kvq_debug_set_stall_ns): > 0 makes the softmax
  // warps wait up to this long on a barrier nothing arrives on
  uint64_t stall_ns;
};

// ------------------------------------------------------------------ plan ---
// Rows of group i: its sequences x the query heads of a KV head, in tiles of
// 128; a unit is two tiles (the last of a group maybe one) over the prefix's
// key tiles.  The cost of a unit is tiles x key tiles, after kUnitCost for
// starting it (its queries, its first scores, its output: about as long as that
// many tiles; 8 and 18 were within 2%).  Per KV head the batch's units are
// laid end to end and, less the first unit's start, which every CTA pays, cut
// into equal slots, one per CTA; a slot's part inside a unit is a segment.
constexpr int kUnitCost = 16;
struct Group {
  int a, nb;        // first sequence, sequences
  int L, tiles, K;  // prefix tokens, row tiles, key tiles
  KVQ_DEVINL int units() const { return (tiles + 1) / 2; }
  KVQ_DEVINL int cost() const { return tiles * K > 0 ? tiles * K + units() * kUnitCost : 0; }
};
KVQ_DEVINL Group group_of(const SharedParams& p, int i, bool report) {
  Group r;
  int a = ld_l2only_s32(p.group_starts + i), e = ld_l2only_s32(p.group_starts + i + 1);
  int L = ld_l2only_s32(p.prefix_lens + i);
  int fault = 0;
  if (a < 0 || a > p.B || e < a || e > p.B) {
    fault = KVQ_DEV_BAD_GROUP;
    a = min(max(a, 0), p.B);
    e = min(max(e, a), p.B);
  }
  if (L < 0 || L > p.max_prefix * kPage) {
    fault |= KVQ_DEV_BAD_SEQLEN;
    L = L < 0 ? 0 : p.max_prefix * kPage;
  }
  if (fault && report) set_status(p.dev_status, fault);
  r.a = a;
  r.nb = e - a;
  r.L = L;
  r.tiles = (r.nb * p.g + TR - 1) / TR;
  r.K = (L + TK - 1) / TK;
  return r;
}
// Inclusive warp prefix sums of the cost and the units of 32 groups.
KVQ_DEVINL void scan_groups(int& cost, int& units, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int c = __shfl_up_sync(0xffffffffu, cost, o);
    const int u = __shfl_up_sync(0xffffffffu, units, o);
    if (lane >= o) {
      cost += c;
      units += u;
    }
  }
}
// The cut of the stream [kUnitCost, W) of cost into used slots: the first `rem`
// slots hold q + 1, the others q.  The host checks that W is below 2^31 for
// groups in order; faulty ones, which may overlap, can make it wrap, and what
// follows from it is then clamped or dropped where it would index out of bounds.
struct Cut {
  int q, rem, used;
  KVQ_DEVINL Cut(const SharedParams& p, int W) {
    W -= kUnitCost;
    used = max(0, min(W, p.slots));
    q = used ? static_cast<unsigned>(W) / static_cast<unsigned>(used) : 0;
    rem = used ? W - q * used : 0;
  }
  KVQ_DEVINL int start(int slot) const { return kUnitCost + slot * q + min(slot, rem); }
  KVQ_DEVINL int slot_of(int x) const {
    x -= kUnitCost;
    const int y = x - rem * (q + 1);
    return max(0, min(used - 1, y < 0 ? x / (q + 1) : rem + y / q));
  }
};

struct Segment {
  int a;           // first sequence of the group
  int row0, rows;  // rows [row0, row0 + rows) of the group
  bool once;       // no other unit reads these keys
  int nq;          // tiles: 2, or 1 (then the two row halves take alternate key tiles of the one tile)
  int k0, k1;      // key tiles
  int L;           // prefix tokens
  int group;
  int unit;
};

// The segments of one slot; every lane of the warp holds the same values.
// The groups come 32 at a time, one per lane, so that a batch of at most 32
// groups is read once.
struct SegWalk {
  Group mine;  // group base + lane
  int base;
  int pos, end, gstart;
  int gi, ubase;
  KVQ_DEVINL void load(const SharedParams& p, int at, int lane, bool report) {
    base = at;
    mine = Group{};
    if (at + lane < p.G) mine = group_of(p, at + lane, report);
  }
  KVQ_DEVINL SegWalk(const SharedParams& p, int slot, int lane, bool report) {
    int W = 0;
#pragma unroll 1
    for (int at = 0; at < p.G; at += 32) {
      load(p, at, lane, report);
      W += __reduce_add_sync(0xffffffffu, mine.cost());
    }
    const Cut cut(p, W);
    pos = end = gstart = 0;
    gi = ubase = 0;
    if (slot >= cut.used) return;
    pos = cut.start(slot);
    end = cut.start(slot + 1);
#pragma unroll 1
    for (int at = 0; at < p.G; at += 32) {  // the group that pos lies in
      if (base != at) load(p, at, lane, false);
      int c = mine.cost(), u = mine.units();
      scan_groups(c, u, lane);
      const int before = __popc(__ballot_sync(0xffffffffu, gstart + c <= pos));
      const int last = before < 32 ? before - 1 : 31;
      const int cb = __shfl_sync(0xffffffffu, c, last & 31), ub = __shfl_sync(0xffffffffu, u, last & 31);
      gi = at + before;
      if (before) {
        gstart += cb;
        ubase += ub;
      }
      if (before < 32) return;
    }
  }
  KVQ_DEVINL bool next(const SharedParams& p, Segment& s, int lane) {
#pragma unroll 1
    while (pos < end && gi < p.G) {
      if (__builtin_expect(gi >= base + 32 || gi < base, 0)) load(p, gi & ~31, lane, false);
      const int at = gi - base;
      const int tiles = __shfl_sync(0xffffffffu, mine.tiles, at), K = __shfl_sync(0xffffffffu, mine.K, at);
      const int cost = tiles * K > 0 ? tiles * K + (tiles + 1) / 2 * kUnitCost : 0;
      if (pos >= gstart + cost) {
        gstart += cost;
        ubase += (tiles + 1) / 2;
        ++gi;
        continue;
      }
      int u = 0;
      if (pos - gstart >= 2 * K + kUnitCost) u = static_cast<unsigned>(pos - gstart) / static_cast<unsigned>(2 * K + kUnitCost);
      const int ustart = gstart + u * (2 * K + kUnitCost) + kUnitCost;  // past its starting cost
      s.once = tiles <= 2;
      s.nq = min(2, tiles - 2 * u);
      const int stop = min(end, ustart + s.nq * K);
      // the slot ends before the unit's first tile; or a wrapped stream
      if (stop <= ustart || u < 0 || u >= (tiles + 1) / 2) break;
      pos = max(pos, ustart);
      s.k0 = s.nq == 2 ? (pos - ustart + 1) >> 1 : pos - ustart;
      s.k1 = s.nq == 2 ? (stop - ustart + 1) >> 1 : stop - ustart;
      s.a = __shfl_sync(0xffffffffu, mine.a, at);
      s.row0 = u * UNIT;
      s.rows = min(UNIT, __shfl_sync(0xffffffffu, mine.nb, at) * p.g - s.row0);
      s.L = __shfl_sync(0xffffffffu, mine.L, at);
      s.group = gi;
      s.unit = ubase + u;
      pos = stop;
      // false only with faulty group_starts (reported)
      return s.k0 >= 0 && s.k1 >= s.k0 && s.k1 <= K && s.unit >= 0 && s.unit < p.max_units;
    }
    return false;
  }
};

// Where the partials of row (b, head hi of a KV head's group) are, for every KV
// head alike.  x: index of the first prefix partial (its segment * UNIT + the
// row in its unit); y: their count, and 2 << 24 where a segment holds two
// (alternate key tiles), else 1 << 24; z, w: first segment of the own tokens'
// partials (slot + b) and their count.
// Warp w of n takes every (n * gridDim)-th sequence (one warp for all of a CTA's:
// 1,024 sequences in 512 groups 158 against 124 us a call).
KVQ_DEVINL void write_parts(const SharedParams& p, int lane, int w, int n) {
  const int b0 = blockIdx.x + gridDim.x * w, step = gridDim.x * n;
  if (b0 >= p.B) return;
  WideScan ws = {};
  if (p.own_slots) ws = wide_scan(p.seq_lens, p.B, p.max_blocks, lane, true);
#pragma unroll 1
  for (int b = b0; b < p.B; b += step) {
    int W = 0, gstart = 0, ubase = 0, a = 0, K = 0, tiles = 0;
    bool found = false;
#pragma unroll 1
    for (int base = 0; base < p.G; base += 32) {
      Group r = {};
      if (base + lane < p.G) r = group_of(p, base + lane, false);
      int c = r.cost(), u = r.units();
      scan_groups(c, u, lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, base + lane < p.G && b >= r.a && b < r.a + r.nb);
      if (hit && !found) {
        found = true;
        const int at = __ffs(hit) - 1;
        a = __shfl_sync(0xffffffffu, r.a, at);
        K = __shfl_sync(0xffffffffu, r.K, at);
        tiles = __shfl_sync(0xffffffffu, r.tiles, at);
        gstart += __shfl_sync(0xffffffffu, c - r.cost(), at);
        ubase += __shfl_sync(0xffffffffu, u - r.units(), at);
      }
      const int ct = __shfl_sync(0xffffffffu, c, 31);
      W += ct;
      if (!found) {
        gstart += ct;
        ubase += __shfl_sync(0xffffffffu, u, 31);
      }
    }
    int4 e = make_int4(0, 1 << 24, 0, 0);
    const int row = (b - a) * p.g + lane, un = row / UNIT;
    if (found && K > 0 && lane < p.g && ubase + un >= 0 && ubase + un < p.max_units) {
      const int nq = min(2, tiles - 2 * un), c0 = gstart + un * (2 * K + kUnitCost) + kUnitCost;
      const Cut cut(p, W);
      const int s0 = cut.slot_of(c0), ns = max(1, cut.slot_of(c0 + nq * K - 1) - s0 + 1);
      e.x = (s0 + ubase + un) * UNIT + row % UNIT;
      e.y = nq == 1 ? (2 * ns) | (2 << 24) : ns | (1 << 24);
    }
    if (p.own_slots) {
      int start, pages;
      wide_locate(p.seq_lens, p.B, p.max_blocks, ws, b, lane, start, pages);
      if (pages > 0) {
        const int64_t T = ws.total, N = wide_slots(p.own_slots, p.B, ws.total);
        // the slot of a stream page x: the largest s with s * T / N <= x
        const int s0 = static_cast<int>(((start + 1ll) * N + T - 1) / T) - 1;
        const int s1 = static_cast<int>(((start + static_cast<int64_t>(pages)) * N + T - 1) / T) - 1;
        e.z = s0 + b;
        e.w = (s1 - s0 + 1) * kPartialWarps;
      }
    }
    if (lane < p.g) p.parts[static_cast<size_t>(b) * p.g + lane] = e;
  }
}

// ---------------------------------------------------------------- prefix ---
// One CTA per (KV head, slot).  Two streams, each with its own 128 query rows,
// score buffer and output sum in tensor memory: over a unit of two tiles the
// streams take the two tiles and every key tile; over a unit of one tile both
// take the same rows and alternate key tiles.  While one stream's softmax
// runs, the tensor cores work on the other.
//   S = Q K^T   kind::f8f6f4, K as cached (FP8); the query row enters as the
//               sum of two E4M3 terms of q * sigma, sigma = 2^(7 - floor(log2
//               max|q|)): exact except elements under 2^-9 of the row's
//               maximum, which keep 2^-17 of it;
//   O += P V    kind::f16, P = f16(2^(s - M + 8)) from tensor memory, V
//               converted to f16 (exact) by four warps.  FP8 probabilities
//               would lose long tails (a key at 2^-18 of the largest is half
//               a step of E4M3), and two FP8 terms cost the tensor cores as
//               much as f16.
// M is a row's first tile maximum and moves only when a later one is more than
// 2^kSlack times larger (P then reaches at most 2^(8 + kSlack)), so that the
// rescale of O by tensor-memory round trips is rare.
// Bound by shared memory over long prefixes: a key tile of both streams moves
// 272 KiB through it (Q and K for S twice over the two terms, V for O, the
// copies and the conversion), 2,125 cycles at 128 bytes each; measured 2,850 (64
// sequences of 4 heads after 128K tokens: 108 us, 1.27 PFLOP/s of 1.88).  Over
// short ones by what a unit costs to start and end, about 10 us, most of it the
// first fetch of the code.
// A stream's MMAs, issued by one thread, complete in order, and each S_j commit
// covers the P.V issued before it: its softmax sees O complete when S_j arrives,
// and its P_j may lie over S_j.
static_assert(kSoftWarps == 8, "warps 0-3 stream 0, 4-7 stream 1");
constexpr int kConvWarps = 4;           // 8-11
constexpr int W_K = 12, W_V = 13, W_MMA = 14;  // an issuing warp per stream: 14, 15
constexpr int kPrefixThreads = 512;
// Registers per thread: a softmax thread holds its row's 128 scores (reading
// them twice from tensor memory instead cost 500 cycles a tile).
constexpr int REG_SOFT = 192, REG_CONV = 64, REG_CTRL = 64;
static_assert(kSoftWarps * 32 * REG_SOFT + kConvWarps * 32 * REG_CONV + 128 * REG_CTRL <= 65536, "register split");
constexpr float kSlack = 7.f;
constexpr int kInfo = 16;  // tile flags kept: more than the tiles in flight

template <int D>
using Geo = PrefixSmem<D>;
template <int NST>
struct Bars {
  uint64_t k_full[NST], k_empty[NST], v_full[NST], v_empty[NST];
  uint64_t vh_full[2], vh_empty[2];
  uint64_t q_full[2], s_full[2], o_full[2];
  uint64_t p_full[2][2];  // [stream][half of the tile's keys]
  uint64_t turn[2];  // stream 0 has issued its P.V and next S (even, odd rounds): stream 1 may
  uint64_t done[2], stall;
  uint32_t k_bad[kInfo], v_dead[kInfo];  // bit i: page i of the tile is not there
  uint32_t tmem_base;
  int abort;
};

template <int D, bool E5>
__global__ void __launch_bounds__(kPrefixThreads, 1) prefix_kernel(const __grid_constant__ SharedParams p) {
  using G = Geo<D>;
  constexpr int NST = G::NST;
  using B = Bars<NST>;
  static_assert(sizeof(B) <= G::BAR_BYTES, "barrier block");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023) & ~1023u) - raw);
  const uint32_t sbase = smem_u32(smem);
  B* bars = reinterpret_cast<B*>(smem + G::OFF_BAR);
  volatile int* abort_flag = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.x % p.Hkv, slot = blockIdx.x / p.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 2);  // a release per stream
      mbar_init(&bars->v_full[i], 1);
      mbar_init(&bars->v_empty[i], kConvWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->vh_full[i], kConvWarps);
      mbar_init(&bars->vh_empty[i], 2);
      mbar_init(&bars->q_full[i], 128);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i][0], 128);
      mbar_init(&bars->p_full[i][1], 128);
      mbar_init(&bars->o_full[i], 1);
      mbar_init(&bars->done[i], 1);
      mbar_init(&bars->turn[i], 1);
    }
    mbar_init(&bars->stall, 1);
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == W_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&bars->tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;  // S0 | S1 (128 columns each) | O0 | O1 (D each)
  // Whichever of this grid and the own tokens' is launched first waits for what
  // precedes the call; the other starts after that, runs beside it and waits
  // for it only before it ends (and so reads what precedes the call past L1).
  if (p.first) grid_dependency_wait();
  grid_launch_dependents();

  // a wait of the whole warp; false (for good) after a timeout anywhere
  bool ok = true;
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    if (!ok) return false;
    const bool got = mbar_wait(bar, parity, abort_flag);
    if (!__all_sync(0xffffffffu, got)) {
      ok = false;
      set_status(p.dev_status, KVQ_DEV_TIMEOUT);
      *abort_flag = 1;
    }
    return ok;
  };

  if (warp >= W_K) {
    setmaxnreg_dec<REG_CTRL>();
    if (warp == W_K || warp == W_V) {
      // --------------------------------------------------- K and V producers --
      const bool is_k = warp == W_K;
      SegWalk walk(p, slot, lane, is_k && blockIdx.x == 0);
      uint64_t* full = is_k ? bars->k_full : bars->v_full;
      uint64_t* empty = is_k ? bars->k_empty : bars->v_empty;
      uint32_t* info = is_k ? bars->k_bad : bars->v_dead;
      const uint8_t* cache = is_k ? p.k_cache : p.v_cache;
      const int64_t str = is_k ? p.k_str : p.v_str;
      uint8_t* ring = smem + (is_k ? G::OFF_K : G::OFF_V);
      const uint64_t pol_once = policy_evict_first(), pol_keep = policy_evict_last();
      uint32_t it = 0;  // tiles issued
      for (Segment s; ok && walk.next(p, s, lane);) {
        const int n_pages = (s.L + kPage - 1) / kPage;
        const int32_t* bt = p.prefix_table + static_cast<size_t>(s.group) * p.max_prefix;
        // block ids of four tiles at a time, loaded a group ahead
        auto load_ids = [&](int tile) {
          const int page = tile * (TK / kPage) + lane;
          return tile < s.k1 && page < n_pages ? ld_l2only_s32(bt + page) : -1;
        };
        int ids = load_ids(s.k0), ids_next = load_ids(s.k0 + 4);
        for (int kt = s.k0; kt < s.k1; ++kt, ++it) {
          const int in_group = (kt - s.k0) & 3;
          if (in_group == 0 && kt != s.k0) {
            ids = ids_next;
            ids_next = load_ids(kt + 4);
          }
          const int st = it % NST;
          if (!wait_all(&empty[st], ((it / NST) & 1) ^ 1)) break;
          int blk = __shfl_sync(0xffffffffu, ids, (in_group << 3) | (lane & 7));
          const int page = kt * (TK / kPage) + lane;
          if (lane >= TK / kPage || page >= n_pages) {
            blk = -1;
          } else if (blk < 0 || static_cast<int64_t>(blk) >= p.num_blocks) {
            set_status(p.dev_status, KVQ_DEV_BAD_BLOCK);
            blk = -1;
          }
          const uint32_t there = __ballot_sync(0xffffffffu, blk >= 0);
          if (lane == 0) {
            info[it % kInfo] = ~there & 0xFFu;
            mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(G::PAGE) * __popc(there));
          }
          __syncwarp();
          if (blk >= 0)
            bulk_g2s(ring + st * G::TILE + lane * G::PAGE, cache + (static_cast<size_t>(blk) * p.Hkv + kvh) * str, G::PAGE,
                     &full[st], s.once ? pol_once : pol_keep);
          __syncwarp();
        }
      }
      if (!ok && lane == 0) {  // abandoned: let issued copies land
        for (uint32_t k = it > NST ? it - NST : 0; k < it; ++k) mbar_wait(&full[k % NST], (k / NST) & 1);
      }
    } else {
      // ----------------------------------------------- MMA issuers, per stream --
      constexpr uint32_t IDESC_S = idesc_e4m3(TR, TK, E5);
      constexpr uint32_t IDESC_O = idesc_f16(TR, D);
      const int x = warp - W_MMA;
      // operand descriptors: the address sits in the low bits (16-byte units)
      const uint32_t q_s = sbase + G::OFF_Q + x * 2 * G::QT;
      const uint64_t q_desc = D == 128 ? desc_sw128(q_s) : desc_sw64(q_s);
      const uint64_t k_desc = D == 128 ? desc_sw128(sbase + G::OFF_K) : desc_sw64(sbase + G::OFF_K);
      const uint64_t v_desc = desc_interleave(sbase + G::OFF_VH, D * 16, 128);
      const uint32_t s_t = tmem + x * TK, o_t = tmem + 2 * TK + x * D;
      SegWalk walk(p, slot, lane, false);
      uint32_t tile0 = 0, np = 0, nseg = 0, round = 0;  // tiles of earlier segments, P tiles and queries seen, turns
      uint32_t kn = 0, vn = 0;                          // next K and V tile to pass
      for (Segment s; ok && walk.next(p, s, lane);) {
        const int n = s.k1 - s.k0;
        if (elect_one()) {
          const bool pair = s.nq == 2;
          const int cnt = pair ? n : (n + 1 - x) / 2;
          auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok && !mbar_wait(bar, parity, abort_flag)) {
              ok = false;
              set_status(p.dev_status, KVQ_DEV_TIMEOUT);
              *abort_flag = 1;
            }
            return ok;
          };
          // Each stream passes every tile in order, the other stream's too (wait
          // and release): a parity wait tells only neighbouring phases apart.
          auto pass_k = [&](uint32_t upto) {
            for (; kn < upto && wait(&bars->k_full[kn % NST], (kn / NST) & 1); ++kn) mbar_arrive(&bars->k_empty[kn % NST]);
          };
          auto pass_v = [&](uint32_t upto) {
            for (; vn < upto && wait(&bars->vh_full[vn & 1], (vn >> 1) & 1); ++vn) mbar_arrive(&bars->vh_empty[vn & 1]);
          };
          auto qk = [&](int j) {  // S = Q K^T
            const uint32_t t = tile0 + (pair ? j : 2 * j + x);
            pass_k(t);
            const int st = t % NST;
            if (!wait(&bars->k_full[st], (t / NST) & 1)) return;
            ++kn;
            tc_fence_after();
            const uint64_t kd = k_desc + st * (G::TILE >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
              for (int term = 0; term < 2; ++term)
                umma_f8(s_t, q_desc + ((term * G::QT + kk * 32) >> 4), kd + ((kk * 32) >> 4), IDESC_S, kk + term > 0 ? 1u : 0u);
            umma_commit(&bars->s_full[x]);
            umma_commit(&bars->k_empty[st]);
          };
          if (cnt > 0 && wait(&bars->q_full[x], nseg++ & 1)) qk(0);
          // Stream 1 issues a tile's P.V only after stream 0 has issued its own
          // and its next S: left alone the streams fall into step, and the
          // tensor cores idle while both softmaxes run.  Stream 0 is at most a
          // round ahead (its next V tile needs stream 1 to release one), so two
          // barriers taken in turn keep their phases apart.
          const int rounds = pair ? n : (n + 1) / 2;
          for (int j = 0; ok && j < rounds; ++j, ++round) {
            if (x == 1 && !wait(&bars->turn[round & 1], (round >> 1) & 1)) break;
            if (j < cnt) {
              const uint32_t t = tile0 + (pair ? j : 2 * j + x);
              pass_v(t);
              if (!wait(&bars->vh_full[t & 1], (t >> 1) & 1)) break;
              ++vn;
              // O += P V: a page per MMA (two halves of eight tokens, D * 16 bytes apart)
              const uint64_t vd = v_desc + (t & 1) * (2 * G::TILE >> 4);
              // the first half of the keys while the softmax works on the second
              // (whole tiles: 19% slower over long prefixes; quarters: 25%)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (!wait(&bars->p_full[x][h], np & 1)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = h * 4; kk < h * 4 + 4; ++kk)
                  umma_f16_ta(o_t, s_t + kk * 8, vd + ((kk * 2 * G::PAGE) >> 4), IDESC_O, (j > 0 || kk > 0) ? 1u : 0u);
              }
              if (!ok) break;
              ++np;
              umma_commit(&bars->vh_empty[t & 1]);
              if (j == cnt - 1) umma_commit(&bars->o_full[x]);
              if (j + 1 < cnt) qk(j + 1);
            }
            if (x == 0) mbar_arrive(&bars->turn[round & 1]);
          }
          pass_k(tile0 + n);
          pass_v(tile0 + n);
        }
        tile0 += n;
        ok = __all_sync(0xffffffffu, ok);
      }
      // every MMA has completed before the tensor memory is released
      if (elect_one()) umma_commit(&bars->done[x]);
      __syncwarp();
      mbar_wait(&bars->done[x], 0);
    }
  } else if (warp >= kSoftWarps) {
    setmaxnreg_dec<REG_CONV>();
    // ------------------------------------------------- V to f16 (exact) --
    // A thread per dimension row: 16 codes -> two 16-byte chunks of f16, the
    // no-swizzle K-major operand (token slots 0-7, then 8-15).  Slots of tokens
    // that are not there are zeroed: P is 0 for them, and 0 x NaN is NaN.
    write_parts(p, lane, warp - kSoftWarps, kConvWarps);  // V is not needed before the first softmax is done
    SegWalk walk(p, slot, lane, false);
    const int t = threadIdx.x - kSoftWarps * 32;
    uint32_t it = 0;
    for (Segment s; ok && walk.next(p, s, lane);) {
      for (int kt = s.k0; kt < s.k1; ++kt, ++it) {
        const int st = it % NST;
        if (!wait_all(&bars->v_full[st], (it / NST) & 1)) break;
        if (!wait_all(&bars->vh_empty[it & 1], ((it >> 1) & 1) ^ 1)) break;
        const uint32_t dead = reinterpret_cast<volatile uint32_t*>(bars->v_dead)[it % kInfo];
        const int valid = s.L - kt * TK;  // tokens of the tile, if less than TK
        const uint8_t* src = smem + G::OFF_V + st * G::TILE;
        uint8_t* dst = smem + G::OFF_VH + (it & 1) * 2 * G::TILE;
        constexpr int IT = TK / kPage * D / (kConvWarps * 32);  // rows per thread
        uint4 c[IT];  // all in flight (half of them at a time: 6% slower at head dim 128)
#pragma unroll
        for (int u = 0; u < IT; ++u) c[u] = *reinterpret_cast<const uint4*>(src + (t + u * kConvWarps * 32) * 16);
        if (dead != 0 || valid < TK) {
#pragma unroll 1
          for (int u = 0; u < IT; ++u) {
            const int pg = (t + u * kConvWarps * 32) / D, left = valid - pg * kPage;
            uint32_t m[4] = {0, 0, 0, 0};
            if (!((dead >> pg) & 1)) {
#pragma unroll
              for (int tok = 0; tok < kPage; ++tok) {
                const int sl = fp8_v_slot(tok);
                if (tok < left) m[sl >> 2] |= 0xFFu << (8 * (sl & 3));
              }
            }
#pragma unroll
            for (int k = 0; k < IT; ++k)
              if (k == u) c[k] = make_uint4(c[k].x & m[0], c[k].y & m[1], c[k].z & m[2], c[k].w & m[3]);
          }
        }
#pragma unroll
        for (int u = 0; u < IT; ++u) {
          const int i = t + u * kConvWarps * 32, pg = i / D, d = i % D;
          uint4 lo, hi;
          fp8x4_to_f16x2x2<E5>(c[u].x, lo.x, lo.y);
          fp8x4_to_f16x2x2<E5>(c[u].y, lo.z, lo.w);
          fp8x4_to_f16x2x2<E5>(c[u].z, hi.x, hi.y);
          fp8x4_to_f16x2x2<E5>(c[u].w, hi.z, hi.w);
          uint8_t* o = dst + pg * 2 * G::PAGE + d * 16;
          *reinterpret_cast<uint4*>(o) = lo;
          *reinterpret_cast<uint4*>(o + D * 16) = hi;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars->v_empty[st]);
          mbar_arrive(&bars->vh_full[it & 1]);
        }
      }
    }
  } else {
    setmaxnreg_inc<REG_SOFT>();
    // ------------------------------------------------------------- softmax --
    // A thread per query row (tensor-memory lane), 128 keys of a tile each.
    const int x = warp >> 2;                 // stream
    const int quarter = warp & 3;
    const uint32_t t_lane = static_cast<uint32_t>(quarter * 32) << 16;
    const int row = quarter * 32 + lane;     // of the stream's tile
    const uint32_t s_t = tmem + t_lane + x * TK, o_t = tmem + t_lane + 2 * TK + x * D;
    const float kscale_raw = __ldcg(p.k_scale + kvh), vscale = __ldcg(p.v_scale + kvh);  // used after the walk's loads
    SegWalk walk(p, slot, lane, false);
    const float kscale = __fmul_rn(__fmul_rn(kscale_raw, p.sm_scale), kLog2e);
    uint32_t tile0 = 0, ns = 0, nseg = 0;  // tiles of earlier segments; S tiles seen; O sums taken
    if (!__all_sync(0xffffffffu, stall_wait(&bars->stall, p.stall_ns, abort_flag))) {
      ok = false;
      set_status(p.dev_status, KVQ_DEV_TIMEOUT);
      *abort_flag = 1;
    }
    for (Segment s; ok && walk.next(p, s, lane);) {
      const bool pair = s.nq == 2;
      const int n = s.k1 - s.k0;
      const int cnt = pair ? n : x == 0 ? (n + 1) / 2 : n / 2;
      const int r = (pair ? x * TR : 0) + row;  // row of the unit
      const bool live = r < s.rows;
      const bool warp_live = __any_sync(0xffffffffu, live);
      const size_t idx = (static_cast<size_t>(kvh) * p.kseg + slot + s.unit) * UNIT + x * TR + row;
      if (cnt == 0) {  // nothing for this stream: no queries, no barriers
        if (live) p.lse_part[idx] = -INFINITY;
        tile0 += n;
        continue;
      }
      // ---- the query rows as two E4M3 terms, swizzled K-major: D / 8 lanes per
      // row, eight dimensions each ----
      float coef = 0.f;
      {
        // 16-byte pieces c4, c4 + 4, ... of eight dimensions each: lanes of a row
        // read 64-byte runs, and a lane's pieces convert side by side.  A loop
        // kept small: the first segment pays for fetching its code.
        constexpr int NP = D / 32, NI = 4;  // pieces per lane, steps of eight rows
        const int sub = lane >> 2, c4 = lane & 3;
        const int own = live ? (s.a + (s.row0 + r) / p.g) * p.Hq + kvh * p.g + (s.row0 + r) % p.g : -1;  // q row
        uint4 u[NI][NP];  // every load in flight at once
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int qr = __shfl_sync(0xffffffffu, own, i * 8 + sub);
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + static_cast<size_t>(max(qr, 0)) * D);
#pragma unroll
          for (int k = 0; k < NP; ++k) u[i][k] = qr >= 0 ? __ldcg(src + c4 + 4 * k) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll 1
        for (int i = 0; i < NI; ++i) {
          const int rq = quarter * 32 + i * 8 + sub;  // row of the tile
          uint32_t mb = 0;  // the largest magnitude, as bf16 bits in either half
#pragma unroll
          for (int k = 0; k < NP; ++k)
            mb = __vmaxu2(mb, __vmaxu2(__vmaxu2(u[0][k].x & 0x7FFF7FFFu, u[0][k].y & 0x7FFF7FFFu),
                                       __vmaxu2(u[0][k].z & 0x7FFF7FFFu, u[0][k].w & 0x7FFF7FFFu)));
          mb = __vmaxu2(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
          mb = __vmaxu2(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
          const uint32_t top = max(mb & 0xFFFFu, mb >> 16);
          int e2 = top ? static_cast<int>(top >> 7) - 127 : 0;
          e2 = e2 < -100 ? -100 : (e2 > 127 ? 127 : e2);
          const float sigma = __uint_as_float(static_cast<uint32_t>(127 + 7 - e2) << 23);
          const float inv = __uint_as_float(static_cast<uint32_t>(127 - 7 + e2) << 23);
          const float mine = __shfl_sync(0xffffffffu, inv, (lane & 7) * 4);
          if ((lane >> 3) == i) coef = fmaxf(kscale * mine, FLT_MIN);  // not 0: times a dead key's -inf
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            const uint32_t w[4] = {u[0][k].x, u[0][k].y, u[0][k].z, u[0][k].w};
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float a0 = __uint_as_float(w[2 * e] << 16) * sigma, a1 = __uint_as_float(w[2 * e] & 0xFFFF0000u) * sigma;
              const float a2 = __uint_as_float(w[2 * e + 1] << 16) * sigma, a3 = __uint_as_float(w[2 * e + 1] & 0xFFFF0000u) * sigma;
              hi[e] = f32x2_to_e4m3x2(a0, a1) | (f32x2_to_e4m3x2(a2, a3) << 16);
              uint32_t f0, f1;
              e4m3x4_to_f16x2x2(hi[e], f0, f1);
              const float2 b0 = __half22float2(*reinterpret_cast<__half2*>(&f0)), b1 = __half22float2(*reinterpret_cast<__half2*>(&f1));
              lo[e] = f32x2_to_e4m3x2(a0 - b0.x, a1 - b0.y) | (f32x2_to_e4m3x2(a2 - b1.x, a3 - b1.y) << 16);
            }
            const int c8 = c4 + 4 * k, c = c8 >> 1;  // piece, 16-byte chunk of the row
            uint8_t* qs = smem + G::q_row(x, 0, rq) + ((D == 128 ? c ^ (rq & 7) : c ^ ((rq >> 1) & 3)) << 4) + (c8 & 1) * 8;
            *reinterpret_cast<uint2*>(qs) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(qs + G::QT) = make_uint2(lo[0], lo[1]);
#pragma unroll
            for (int n = 0; n + 1 < NI; ++n) u[n][k] = u[n + 1][k];
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars->q_full[x]);

      float M = -INFINITY, l = 0.f;
      for (int j = 0; j < cnt; ++j, ++ns) {
        if (!wait_all(&bars->s_full[x], ns & 1)) break;
        tc_fence_after();
        if (warp_live) {
          const uint32_t t = tile0 + (pair ? j : 2 * j + x);
          const int kt = s.k0 + (pair ? j : 2 * j + x);
          const uint32_t bad = reinterpret_cast<volatile uint32_t*>(bars->k_bad)[t % kInfo];
          const int valid = s.L - kt * TK;
          const bool edge = bad != 0 || valid < TK;
          uint32_t v[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_nowait(s_t + 32 * c, v[c]);
          tmem_wait_ld();
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_pin32(v[c]);
            if (edge) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * c + i >= valid || ((bad >> (2 * c + i / kPage)) & 1)) v[c][i] = __float_as_uint(-INFINITY);
            }
            float m1[11];
#pragma unroll
            for (int i = 0; i < 10; ++i)
              m1[i] = fmax3(__uint_as_float(v[c][3 * i]), __uint_as_float(v[c][3 * i + 1]), __uint_as_float(v[c][3 * i + 2]));
            m1[10] = fmaxf(__uint_as_float(v[c][30]), __uint_as_float(v[c][31]));
            mx = fmax3(mx, fmax3(fmax3(m1[0], m1[1], m1[2]), fmax3(m1[3], m1[4], m1[5]), fmax3(m1[6], m1[7], m1[8])),
                       fmaxf(m1[9], m1[10]));
          }
          mx *= coef;
          const bool move = live && mx > M + kSlack;  // M = -inf: the first tile with a live key
          if (j > 0 && __any_sync(0xffffffffu, move)) {
            const float a = move ? ex2(M - mx) : 1.f;
            l *= a;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16_async(o_t + 16 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
              tmem_st16(o_t + 16 * c, o);
            }
          }
          if (move) M = mx;
          const float nb = M == -INFINITY ? 0.f : 8.f - M;  // no live key so far: every score is -inf
          const float2 coef2 = make_float2(coef, coef), nb2 = make_float2(nb, nb);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 32 keys (two pages), 16 words of two slots
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int k = (i >> 3) * 16 + (i & 1) * 8 + ((i & 7) >> 1) * 2;  // tokens of slots 2i, 2i + 1
              float2 e = ffma2(make_float2(__uint_as_float(v[c][k]), __uint_as_float(v[c][k + 1])), coef2, nb2);
              e.x = ex2(e.x);
              e.y = ex2(e.y);
              sum = fadd2(sum, e);
              w[i] = pack_f16x2(e.x, e.y);
            }
            tmem_st16(s_t + 16 * c, w);  // over S, which the registers hold
            if (c & 1) {
              tmem_wait_st();
              tc_fence_before();
              mbar_arrive(&bars->p_full[x][c >> 1]);
            }
          }
          l += sum.x + sum.y;
        } else {
          mbar_arrive(&bars->p_full[x][0]);
          mbar_arrive(&bars->p_full[x][1]);
        }
      }
      tile0 += n;
      if (!ok) break;
      {
        if (!wait_all(&bars->o_full[x], nseg & 1)) break;
        ++nseg;
        tc_fence_after();
        const float f = l > 0.f ? vscale / l : 0.f;
        // A lane holds a row; through shared memory the rows leave as 128-byte
        // runs instead of 16-byte ones (which cost 9,000 cycles per segment).
        auto stage = [&](int rr, int col) {  // row of the warp, dimension of the 32
          return reinterpret_cast<float4*>(smem + G::stage_row(x, quarter, rr) + col * 4);
        };
        const int nrow = min(32, s.rows - (pair ? x * TR : 0) - quarter * 32);  // live rows of the warp
        float* dst = p.o_part + (idx - lane) * D;
        if (warp_live) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(o_t + 32 * c, o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *stage(lane, 4 * i) =
                  make_float4(__uint_as_float(o[4 * i]) * f, __uint_as_float(o[4 * i + 1]) * f,
                              __uint_as_float(o[4 * i + 2]) * f, __uint_as_float(o[4 * i + 3]) * f);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = 4 * i + (lane >> 3);
              if (rr < nrow)
                *reinterpret_cast<float4*>(dst + rr * D + 32 * c + 4 * (lane & 7)) = *stage(rr, 4 * (lane & 7));
            }
            __syncwarp();
          }
        }
        tc_fence_before();
      }
      if (live) p.lse_part[idx] = l > 0.f ? M + __log2f(l) - 8.f : -INFINITY;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  if (!p.first) grid_dependency_wait();
}

// --------------------------------------------------------------- combine ---
struct MergeParams {
  SharedParams sp;
  const float* o_own;    // the own tokens' partials (DecodePartialPlan)
  const float* lse_own;
  int own_splits;
  __nv_bfloat16* out;
};
constexpr int kMergeWarps = 4;

// One CTA per row (b, hq): its warps take the row's partials in turn (a lane
// holds D / 32 dimensions), then merge through shared memory.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const __grid_constant__ MergeParams mp) {
  constexpr int E = D / 32;
  __shared__ float m_s[kMergeWarps], l_s[kMergeWarps], o_s[kMergeWarps][D];
  const SharedParams& p = mp.sp;
  const int b = blockIdx.x / p.Hq, hq = blockIdx.x - b * p.Hq;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  grid_dependency_wait();
  const int4 rp = __ldcg(p.parts + static_cast<size_t>(b) * p.g + hq % p.g);
  const int np = rp.y & 0xFFFFFF, halves = rp.y >> 24;
  const size_t first = (static_cast<size_t>(hq / p.g) * p.kseg * UNIT + rp.x);
  const size_t own_first = p.own_slots ? (static_cast<size_t>(hq) * (p.own_slots + p.B - 1) + rp.z) * kPartialWarps
                                       : static_cast<size_t>(blockIdx.x) * mp.own_splits * kPartialWarps;
  const int n_own = p.own_slots ? rp.w : mp.own_splits * kPartialWarps;
  // Partial i of the row: prefix partials first, then the own tokens'.  A warp
  // takes 32 of them at a time: a lane per log-sum-exp, then the outputs of
  // those that carry weight, eight loads in flight.
  const int total = np + n_own;
  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = wid; i0 < total; i0 += 32 * kMergeWarps) {
    const int i = i0 + lane * kMergeWarps;
    const float* op = nullptr;
    float x = -INFINITY;
    if (i < np) {
      const size_t idx = first + static_cast<size_t>(halves == 2 ? i >> 1 : i) * UNIT + (halves == 2 ? (i & 1) * TR : 0);
      x = __ldcg(p.lse_part + idx);
      op = p.o_part + idx * D;
    } else if (i < total) {
      const size_t idx = own_first + (i - np);
      x = __ldcg(mp.lse_own + idx);
      op = mp.o_own + idx * D;
    }
    float mn = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mn = fmaxf(mn, m);
    if (mn == -INFINITY) continue;  // uniform
    const float w = ex2(x - mn), a = ex2(m - mn);
    m = mn;
    l *= a;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= a;
    uint32_t todo = __ballot_sync(0xffffffffu, w > 0.f);
    while (todo) {
      float wk[8];
      float o[8][E];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int src = todo ? __ffs(todo) - 1 : 0;
        const bool on = todo != 0;
        todo &= todo - 1;
        const float* ok_ = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(op), src));
        const float ws = __shfl_sync(0xffffffffu, w, src);
        wk[k] = on ? ws : 0.f;
        if constexpr (E == 4) {
          const float4 t = on ? __ldcg(reinterpret_cast<const float4*>(ok_) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
          o[k][0] = t.x;
          o[k][1] = t.y;
          o[k][2] = t.z;
          o[k][3] = t.w;
        } else {
          const float2 t = on ? __ldcg(reinterpret_cast<const float2*>(ok_) + lane) : make_float2(0.f, 0.f);
          o[k][0] = t.x;
          o[k][1] = t.y;
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        l += wk[k];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wk[k], o[k][e], acc[e]);
      }
    }
  }
  if (lane == 0) {
    m_s[wid] = m;
    l_s[wid] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) o_s[wid][lane * E + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < D) {
    const int d = threadIdx.x;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) M = fmaxf(M, m_s[w]);
    float num = 0.f, den = 0.f;
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        const float f = ex2(m_s[w] - M);
        den = fmaf(f, l_s[w], den);
        num = fmaf(f, o_s[w][d], num);
      }
    }
    mp.out[static_cast<size_t>(blockIdx.x) * D + d] = __float2bfloat16_rn(den > 0.f ? num / den : 0.f);
  }
}

// Slots per KV head: one CTA per SM over all KV heads.
int prefix_slots(int Hkv) {
  const int n = sm_count() / Hkv;
  return n < 1 ? 1 : n;
}
// Units of the batch: every group adds at most one to its share of B * g / 256.
int64_t prefix_units(int B, int G, int g) { return static_cast<int64_t>(B) * g / UNIT + G; }

struct Layout {
  size_t o_part, lse_part, o_own, lse_own, parts, total;  // byte offsets
};
Layout layout_of(int B, int G, int Hq, int Hkv, int D, int max_blocks) {
  const size_t rows = static_cast<size_t>(Hkv) * (prefix_slots(Hkv) + prefix_units(B, G, Hq / Hkv)) * UNIT;
  const DecodePartialPlan own = decode_partial_plan(B, Hq, Hkv, D, max_blocks);
  Layout l;
  l.o_part = 0;
  l.lse_part = rows * D * 4;
  l.o_own = l.lse_part + rows * 4;
  l.lse_own = l.o_own + own.rows * D * 4;
  l.parts = l.lse_own + (own.rows * 4 + 15) / 16 * 16;
  l.total = l.parts + static_cast<size_t>(B) * (Hq / Hkv) * sizeof(int4);
  return l;
}

template <int D, bool E5>
kvq_status_t launch_shared(const SharedParams& p, const MergeParams& mp, const DecodePartialArgs& a,
                           const DecodePartialPlan& own, cudaStream_t s) {
  constexpr int smem = Geo<D>::SMEM;
  auto kern = prefix_kernel<D, E5>;
  static int configured_mask = 0;  // devices whose attribute is set
  int dev = 0;
  cudaGetDevice(&dev);
  if (!(configured_mask & (1 << (dev & 31)))) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_status(e, "shared_prefix: set shared memory size");
    configured_mask |= 1 << (dev & 31);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.slots * p.Hkv);
  cfg.blockDim = dim3(kPrefixThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  if (p.first) e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return cuda_status(e, "shared_prefix launch");
  const kvq_status_t st = decode_partials(a, own, s);
  if (st != KVQ_OK) return st;
  if (!p.first) e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return cuda_status(e, "shared_prefix launch");
  cfg.gridDim = dim3(p.B * p.Hq);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, merge_kernel<D>, mp);
  return cuda_status(e, "shared_prefix merge launch");
}

}  // namespace

}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_shared_prefix_workspace_size(int B, int G, int Hq, int Hkv, int D, int P, int max_prefix_blocks,
                                                   int max_blocks) {
  if (B < 1 || G < 1 || Hq < 1 || Hkv < 1 || D < 1 || P < 1 || max_prefix_blocks < 1 || max_blocks < 1 || Hq % Hkv != 0)
    return 0;
  return layout_of(B, G, Hq, Hkv, D, max_blocks).total;
}

extern "C" kvq_status_t kvq_paged_decode_attention_shared_prefix(
    const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
    const int32_t* prefix_table, const int32_t* prefix_lens, const int32_t* group_starts, const int32_t* block_table,
    const int32_t* seq_lens, void* out, int B, int G, int Hq, int Hkv, int D, int P, int max_prefix_blocks,
    int max_blocks, int64_t num_blocks, float sm_scale, kvq_dtype_t cache_dtype, void* workspace,
    size_t workspace_bytes, int* dev_status, kvq_stream_t stream) {
  clear_error();
  if (B < 1 || G < 1 || Hq < 1 || Hkv < 1 || max_prefix_blocks < 1 || max_blocks < 1 || num_blocks < 1)
    return fail(KVQ_ERR_INVALID_ARG, "shared_prefix: bad sizes");
  if (Hq % Hkv != 0) return fail(KVQ_ERR_INVALID_ARG, "shared_prefix: Hq %% Hkv != 0");
  if (!(sm_scale > 0.f) || !(sm_scale < FLT_MAX)) return fail(KVQ_ERR_INVALID_ARG, "shared_prefix: bad sm_scale");
  if (P != kPage) return fail(KVQ_ERR_UNSUPPORTED, "shared_prefix: page size %d (only 16)", P);
  if (D != 64 && D != 128) return fail(KVQ_ERR_UNSUPPORTED, "shared_prefix: head_dim %d", D);
  if (Hq / Hkv > 8) return fail(KVQ_ERR_UNSUPPORTED, "shared_prefix: GQA ratio %d > 8", Hq / Hkv);
  if (cache_dtype != KVQ_DTYPE_FP8_E4M3 && cache_dtype != KVQ_DTYPE_FP8_E5M2)
    return fail(KVQ_ERR_UNSUPPORTED, "shared_prefix: FP8 (E4M3 or E5M2) caches only");
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !prefix_table || !prefix_lens || !group_starts ||
      !block_table || !seq_lens || !out || !workspace)
    return fail(KVQ_ERR_INVALID_ARG, "shared_prefix: null pointer");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(workspace, 16) || !aligned(out, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(prefix_table, 4) || !aligned(prefix_lens, 4) ||
      !aligned(group_starts, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return fail(KVQ_ERR_INVALID_ARG, "shared_prefix: misaligned pointer");
  const int64_t g = Hq / Hkv;
  if (static_cast<int64_t>(max_prefix_blocks) * P > 0x7FFFFFFFll - TK || static_cast<int64_t>(max_blocks) * P > 0x7FFFFFFFll - TK ||
      static_cast<int64_t>(B) * Hq > 0x7FFFFFFFll || B * g > 0x7FFFFFFFll - TR || (prefix_units(B, G, g) + prefix_slots(Hkv)) * UNIT > 0x7FFFFFFFll ||
      prefix_units(B, G, g) * (2 * ((static_cast<int64_t>(max_prefix_blocks) * P + TK - 1) / TK) + kUnitCost) > 0x7FFFFFFFll)
    return fail(KVQ_ERR_UNSUPPORTED, "shared_prefix: problem too large");
  const DecodePartialPlan own = decode_partial_plan(B, Hq, Hkv, D, max_blocks);
  if (own.items > 0x7FFFFFFFll || static_cast<int64_t>(B) * max_blocks > 0x7FFFFFFFll)
    return fail(KVQ_ERR_UNSUPPORTED, "shared_prefix: problem too large");
  const Layout l = layout_of(B, G, Hq, Hkv, D, max_blocks);
  if (workspace_bytes < l.total)
    return fail(KVQ_ERR_INVALID_ARG, "shared_prefix: workspace %zu bytes < %zu needed", workspace_bytes, l.total);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool e5 = cache_dtype == KVQ_DTYPE_FP8_E5M2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  DecodePartialArgs a;
  a.q = q;
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.o_part = reinterpret_cast<float*>(ws + l.o_own);
  a.lse_part = reinterpret_cast<float*>(ws + l.lse_own);
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.sm_scale = sm_scale;
  a.e5m2 = e5;
  a.dev_status = dev_status;
  SharedParams p;
  p.q = q;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.prefix_table = prefix_table;
  p.prefix_lens = prefix_lens;
  p.group_starts = group_starts;
  p.o_part = reinterpret_cast<float*>(ws + l.o_part);
  p.lse_part = reinterpret_cast<float*>(ws + l.lse_part);
  p.B = B;
  p.G = G;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.g = static_cast<int>(g);
  p.max_prefix = max_prefix_blocks;
  p.num_blocks = num_blocks;
  p.sm_scale = sm_scale;
  const int64_t page_b = static_cast<int64_t>(kPage) * D;
  const PageStrides ps = page_strides(k_cache, v_cache, page_b, page_b);
  p.k_str = ps.k;
  p.v_str = ps.v;
  p.slots = prefix_slots(Hkv);
  p.max_units = static_cast<int>(prefix_units(B, G, p.g));
  p.kseg = p.slots + p.max_units;
  p.dev_status = dev_status;
  p.stall_ns = stall_ns();
  p.parts = reinterpret_cast<int4*>(ws + l.parts);
  p.seq_lens = seq_lens;
  p.max_blocks = max_blocks;
  p.own_slots = own.slots;
  // A long prefix goes first: its CTAs end microseconds apart, and the own
  // tokens' fill what they leave (128 sequences after 32K: 118 us, 125 the other
  // way).  A short one second: the own tokens' grid, small enough to be placed
  // while the preceding kernel still runs, starts faster (32 after 8K: 33 us
  // against 35).  By the tiles per CTA; more sequences than the wide plan takes
  // have no partials that wait late.
  const int64_t tiles = (B * g + TR - 1) / TR * ((static_cast<int64_t>(max_prefix_blocks) * P + TK - 1) / TK);
  p.first = own.slots > 0 && tiles >= 8ll * p.slots;
  a.late = p.first != 0;
  MergeParams mp;
  mp.sp = p;
  mp.o_own = a.o_part;
  mp.lse_own = a.lse_part;
  mp.own_splits = own.splits;
  mp.out = static_cast<__nv_bfloat16*>(out);
  if (e5) return D == 128 ? launch_shared<128, true>(p, mp, a, own, s) : launch_shared<64, true>(p, mp, a, own, s);
  return D == 128 ? launch_shared<128, false>(p, mp, a, own, s) : launch_shared<64, false>(p, mp, a, own, s);
}
