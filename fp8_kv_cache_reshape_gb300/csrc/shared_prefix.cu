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

namespace kvq {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int TR = 128;         // query rows per tile
constexpr int TK = 128;         // keys per tile (8 pages)
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
};

// ------------------------------------------------------------------ plan ---
// Rows of group i: its sequences x the query heads of a KV head, in tiles of
// 128; a unit is two tiles (the last of a group maybe one) over the prefix's
// key tiles.  The cost of a unit is tiles x key tiles.  Per KV head the
// batch's units are laid end to end and cut into equal slots, one per CTA; a
// slot's part inside a unit is a segment.
struct Group {
  int a, nb;     // first sequence, sequences
  int L, tiles, K;  // prefix tokens, row tiles, key tiles
  int units;
  int64_t cost;
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
  r.units = (r.tiles + 1) / 2;
  r.cost = static_cast<int64_t>(r.tiles) * r.K;
  return r;
}
// Inclusive warp prefix sums of the cost and the units of 32 groups.
KVQ_DEVINL void scan_groups(int64_t& cost, int& units, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t c = __shfl_up_sync(0xffffffffu, cost, o);
    const int u = __shfl_up_sync(0xffffffffu, units, o);
    if (lane >= o) {
      cost += c;
      units += u;
    }
  }
}
KVQ_DEVINL int64_t total_cost(const SharedParams& p, int lane, bool report) {
  int64_t W = 0;
  for (int base = 0; base < p.G; base += 32) {
    int64_t c = base + lane < p.G ? group_of(p, base + lane, report).cost : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    W += c;
  }
  return W;
}
KVQ_DEVINL int64_t used_slots(const SharedParams& p, int64_t W) { return W < p.slots ? W : p.slots; }

struct Segment {
  int a;           // first sequence of the group
  int row0, rows;  // rows [row0, row0 + rows) of the group
  int nq;          // tiles: 2, or 1 (then the two row halves take alternate key tiles of the one tile)
  int k0, k1;      // key tiles
  int L;           // prefix tokens
  int group;
  int unit;
};

// The segments of one slot; every lane of the warp holds the same values.
struct SegWalk {
  int64_t pos, end, gstart;
  int gi, ubase;
  KVQ_DEVINL SegWalk(const SharedParams& p, int slot, int lane, bool report) {
    const int64_t W = total_cost(p, lane, report);
    const int64_t N = used_slots(p, W);
    pos = end = gstart = 0;
    gi = ubase = 0;
    if (slot >= N) return;
    pos = slot * W / N;
    end = (slot + 1) * W / N;
    for (int base = 0; base < p.G; base += 32) {  // the group that pos lies in
      int64_t c = 0;
      int u = 0;
      if (base + lane < p.G) {
        const Group r = group_of(p, base + lane, false);
        c = r.cost;
        u = r.units;
      }
      scan_groups(c, u, lane);
      const int before = __popc(__ballot_sync(0xffffffffu, gstart + c <= pos));
      if (before < 32) {
        const int64_t cb = __shfl_sync(0xffffffffu, c, before ? before - 1 : 0);
        const int ub = __shfl_sync(0xffffffffu, u, before ? before - 1 : 0);
        gi = base + before;
        if (before) {
          gstart += cb;
          ubase += ub;
        }
        return;
      }
      gstart += __shfl_sync(0xffffffffu, c, 31);
      ubase += __shfl_sync(0xffffffffu, u, 31);
    }
    gi = p.G;
  }
  KVQ_DEVINL bool next(const SharedParams& p, Segment& s) {
    while (pos < end && gi < p.G) {
      const Group r = group_of(p, gi, false);
      if (pos >= gstart + r.cost) {
        gstart += r.cost;
        ubase += r.units;
        ++gi;
        continue;
      }
      const int u = static_cast<int>((pos - gstart) / (2 * r.K));
      const int64_t ustart = gstart + static_cast<int64_t>(u) * 2 * r.K;
      s.nq = min(2, r.tiles - 2 * u);
      const int64_t uend = ustart + static_cast<int64_t>(s.nq) * r.K;
      const int64_t stop = end < uend ? end : uend;
      s.k0 = static_cast<int>((pos - ustart + s.nq - 1) / s.nq);
      s.k1 = static_cast<int>((stop - ustart + s.nq - 1) / s.nq);
      s.a = r.a;
      s.row0 = u * UNIT;
      s.rows = min(UNIT, r.nb * p.g - s.row0);
      s.L = r.L;
      s.group = gi;
      s.unit = ubase + u;
      pos = stop;
      if (s.unit < p.max_units) return true;
      return false;  // only with faulty group_starts (reported)
    }
    return false;
  }
};

// ---------------------------------------------------------------- prefix ---
// Grid slots * Hkv; a thread per row of the unit.
template <int D, bool E5>
__global__ void __launch_bounds__(256) prefix_kernel(const __grid_constant__ SharedParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  float* ks = reinterpret_cast<float*>(smem);  // [TK][D]
  float* vs = ks + TK * D;                     // [TK][D]
  __nv_bfloat162* qs = reinterpret_cast<__nv_bfloat162*>(vs + TK * D);  // [UNIT][D / 2 + 1]
  __shared__ int bad[TK / kPage];
  const int kvh = blockIdx.x % p.Hkv, slot = blockIdx.x / p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31;
  grid_launch_dependents();
  SegWalk walk(p, slot, lane, blockIdx.x == 0 && tid < 32);
  const float coef = p.k_scale[kvh] * p.sm_scale * kLog2e;
  auto dec = [](uint8_t c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, E5 ? __NV_E5M2 : __NV_E4M3);
    return __half2float(__half(h));
  };
  for (Segment s; walk.next(p, s);) {
    const int half = tid >> 7;
    const int row = s.nq == 2 ? tid : tid & 127;
    const bool live = row < s.rows;
    __syncthreads();
    if (live) {
      const int r = s.row0 + row;
      const __nv_bfloat162* src = reinterpret_cast<const __nv_bfloat162*>(
          static_cast<const __nv_bfloat16*>(p.q) +
          (static_cast<size_t>(s.a + r / p.g) * p.Hq + kvh * p.g + r % p.g) * D);
      for (int d = 0; d < D / 2; ++d) qs[tid * (D / 2 + 1) + d] = src[d];
    }
    float m = -INFINITY, l = 0.f, o[D];
#pragma unroll
    for (int d = 0; d < D; ++d) o[d] = 0.f;
    for (int kt = s.k0; kt < s.k1; ++kt) {
      __syncthreads();
      for (int i = tid; i < TK * D; i += 256) {
        const int key = i / D, d = i % D, tok = kt * TK + key;
        float kx = 0.f, vx = 0.f;
        if (tok < s.L) {
          const int blk = p.prefix_table[static_cast<size_t>(s.group) * p.max_prefix + tok / kPage];
          const bool ok = blk >= 0 && static_cast<int64_t>(blk) < p.num_blocks;
          if (!ok) set_status(p.dev_status, KVQ_DEV_BAD_BLOCK);
          if (d == 0 && key % kPage == 0) bad[key / kPage] = !ok;
          if (ok) {
            const size_t pg = static_cast<size_t>(blk) * p.Hkv + kvh;
            const int t = tok % kPage;
            kx = dec(p.k_cache[pg * p.k_str + fp8_k_offset(t, d / 16, D) + d % 16]);
            vx = dec(p.v_cache[pg * p.v_str + d * kPage + fp8_v_slot(t)]);
          }
        }
        ks[i] = kx;
        vs[i] = vx;
      }
      __syncthreads();
      if (!live || (s.nq == 1 && ((kt - s.k0) & 1) != half)) continue;
      const int n = min(TK, s.L - kt * TK);
      for (int key = 0; key < n; ++key) {
        if (bad[key / kPage]) continue;
        float x = 0.f;
        for (int d = 0; d < D / 2; ++d) {
          const float2 qf = __bfloat1622float2(qs[tid * (D / 2 + 1) + d]);
          x = fmaf(qf.x, ks[key * D + 2 * d], fmaf(qf.y, ks[key * D + 2 * d + 1], x));
        }
        x *= coef;
        const float mn = fmaxf(m, x), a = ex2(m - mn), w = ex2(x - mn);
        l = l * a + w;
#pragma unroll
        for (int d = 0; d < D; ++d) o[d] = fmaf(w, vs[key * D + d], o[d] * a);
        m = mn;
      }
    }
    if (live) {
      const size_t idx = (static_cast<size_t>(kvh) * p.kseg + slot + s.unit) * UNIT + tid;
      const float f = l > 0.f ? p.v_scale[kvh] / l : 0.f;
#pragma unroll
      for (int d = 0; d < D; ++d) p.o_part[idx * D + d] = o[d] * f;
      p.lse_part[idx] = l > 0.f ? m + log2f(l) : -INFINITY;
    }
  }
  // the decode partials' grid precedes this one and may still run: this grid
  // must not complete before it, so that the combine sees both
  grid_dependency_wait();
}

// --------------------------------------------------------------- combine ---
struct MergeParams {
  SharedParams sp;
  const float* o_own;    // [B][Hq][per_row][D]
  const float* lse_own;  // [B][Hq][per_row]
  int per_row;
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
  // the row's prefix partials: slots s0 .. s0 + ns - 1, `halves` of each
  int ns = 0, halves = 1;
  size_t first = 0;
  {
    const int64_t W = total_cost(p, lane, false), N = used_slots(p, W);
    int64_t gstart = 0;
    int ubase = 0;
    for (int base = 0; base < p.G; base += 32) {
      Group r = {};
      if (base + lane < p.G) r = group_of(p, base + lane, false);
      int64_t c = r.cost;
      int u = r.units;
      scan_groups(c, u, lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, base + lane < p.G && b >= r.a && b < r.a + r.nb);
      if (hit) {
        const int at = __ffs(hit) - 1;
        const int a = __shfl_sync(0xffffffffu, r.a, at), K = __shfl_sync(0xffffffffu, r.K, at);
        const int tiles = __shfl_sync(0xffffffffu, r.tiles, at);
        gstart += __shfl_sync(0xffffffffu, c - r.cost, at);
        ubase += __shfl_sync(0xffffffffu, u - r.units, at);
        const int row = (b - a) * p.g + hq % p.g, un = row / UNIT;
        const int nq = min(2, tiles - 2 * un);
        if (K > 0 && ubase + un < p.max_units) {
          const int64_t c0 = gstart + static_cast<int64_t>(un) * 2 * K, c1 = c0 + static_cast<int64_t>(nq) * K;
          const int s0 = static_cast<int>(((c0 + 1) * N + W - 1) / W) - 1;
          const int s1 = static_cast<int>((c1 * N + W - 1) / W) - 1;
          ns = s1 - s0 + 1;
          halves = nq == 1 ? 2 : 1;
          first = (static_cast<size_t>(hq / p.g) * p.kseg + s0 + ubase + un) * UNIT + row % UNIT;
        }
        break;
      }
      gstart += __shfl_sync(0xffffffffu, c, 31);
      ubase += __shfl_sync(0xffffffffu, u, 31);
    }
  }
  grid_dependency_wait();
  const int np = ns * halves, total = np + mp.per_row;
  auto at = [&](int i, const float*& o, const float*& l) {
    if (i < np) {
      const size_t idx = first + static_cast<size_t>(i / halves) * UNIT + (i % halves) * TR;
      o = p.o_part + idx * D;
      l = p.lse_part + idx;
    } else {
      const size_t idx = static_cast<size_t>(blockIdx.x) * mp.per_row + (i - np);
      o = mp.o_own + idx * D;
      l = mp.lse_own + idx;
    }
  };
  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i = wid; i < total; i += kMergeWarps) {
    const float *op, *lp;
    at(i, op, lp);
    const float x = *lp;
    if (x == -INFINITY) continue;
    const float mn = fmaxf(m, x), a = ex2(m - mn), w = ex2(x - mn);
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(w, op[lane * E + e], acc[e] * a);
    m = mn;
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
  size_t o_part, lse_part, o_own, lse_own, total;  // byte offsets
};
Layout layout_of(int B, int G, int Hq, int Hkv, int D, int max_blocks) {
  const size_t rows = static_cast<size_t>(Hkv) * (prefix_slots(Hkv) + prefix_units(B, G, Hq / Hkv)) * UNIT;
  const DecodePartialPlan own = decode_partial_plan(B, Hq, Hkv, D, max_blocks);
  Layout l;
  l.o_part = 0;
  l.lse_part = rows * D * 4;
  l.o_own = l.lse_part + rows * 4;
  l.lse_own = l.o_own + own.rows * D * 4;
  l.total = l.lse_own + (own.rows * 4 + 15) / 16 * 16;
  return l;
}

template <int D, bool E5>
kvq_status_t launch_shared(const SharedParams& p, const MergeParams& mp, cudaStream_t s) {
  constexpr int smem = 2 * TK * D * 4 + UNIT * (D / 2 + 1) * 4;
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
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
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
      static_cast<int64_t>(B) * Hq > 0x7FFFFFFFll || B * g > 0x7FFFFFFFll - TR || prefix_units(B, G, g) > 0x3FFFFFFF)
    return fail(KVQ_ERR_UNSUPPORTED, "shared_prefix: problem too large");
  const DecodePartialPlan own = decode_partial_plan(B, Hq, Hkv, D, max_blocks);
  if (static_cast<int64_t>(B) * Hkv * own.splits > 0x7FFFFFFFll)
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
  a.splits = own.splits;
  a.num_blocks = num_blocks;
  a.sm_scale = sm_scale;
  a.e5m2 = e5;
  a.dev_status = dev_status;
  const kvq_status_t st = decode_partials(a, s);
  if (st != KVQ_OK) return st;

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
  MergeParams mp;
  mp.sp = p;
  mp.o_own = a.o_part;
  mp.lse_own = a.lse_part;
  mp.per_row = own.per_row;
  mp.out = static_cast<__nv_bfloat16*>(out);
  if (e5) return D == 128 ? launch_shared<128, true>(p, mp, s) : launch_shared<64, true>(p, mp, s);
  return D == 128 ? launch_shared<128, false>(p, mp, s) : launch_shared<64, false>(p, mp, s);
}
