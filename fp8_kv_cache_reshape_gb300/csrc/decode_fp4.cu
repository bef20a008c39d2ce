// kvq_paged_decode_attention_fp4: one decode step over a 4-bit paged cache.
//
// Mathematics.  Online softmax in base 2 per query head, split over the cache
// and joined by log-sum-exps: with scores s2 = (q . k) sm_scale log2 e and any
// stabilizer M, a piece's (M, l = sum 2^(s2 - M), O = sum 2^(s2 - M) v) joins
// another's after scaling by 2^(M - M').  K's value is code * block scale *
// head scale; code * block scale has at most six significant bits and is at least
// 2^-10, so it is exact in float16 and K enters the products exactly.  V's block scale
// belongs to a token and 16 dims: with those 16 dims as the rows of one MMA it
// moves to the other operand, P, one multiplication for two weights instead of one
// for every two of V's 16 x 16 values.
//
// Bound: memory, 9/16 byte per element of K and V.
//
// Layout.  A warp takes two pages (32 tokens of a KV head) at a time from two
// stages of its own in shared memory, filled by 16-byte asynchronous copies: no
// barrier, no producer warp, nothing between warps until a piece ends.  The
// page format is the MMA operand order (m16n8k16, tokens as the rows of K Q^T,
// dims as the rows of V^T P^T), so that a lane reads its whole share of a page
// with 16-byte loads: lane 4 r + c holds dims 32 c .. 32 c + 31 (at head dim
// 128) of tokens r and r + 8 of K, and tokens 2c, 2c + 1, 2c + 8, 2c + 9 of
// dims 2r, 2r + 1 of each 16 of V.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "kvq_host.h"
#include "kvq_rows.cuh"

namespace kvq {

namespace {

constexpr int kWarps = 4;             // warps per CTA, each with a ring of its own
constexpr int kCtasPerSm = 3;
constexpr int kMinPart = 4;           // pages of a part, at least
constexpr int kHinted = 16;             // pages that hint_pages() asks for: two pairs per warp
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLag = 3.f;           // by how much scores may pass the stabilizer
constexpr float kBase = 4.f;          // weights are 2^(s2 - M + kBase) <= 2^7: times 448 within float16
constexpr float kNone = -1e30f;
// Sums of code products are below 2^27, so a smaller coefficient gives scores of zero
// either way; one of zero would make a masked score, minus infinity, no number.
constexpr float kLeast = 1e-30f;
#define NEG_INF __int_as_float(0xff800000)

template <int D>
struct Fp4 {
  static constexpr int kCodes = kPage * D / 2;
  static constexpr int kScales = kPage * D / 16;
  static constexpr int kPageB = kCodes + kScales;
  static constexpr int kPairB = 2 * kPageB;            // K page, V page
  static constexpr int kStageB = 2 * kPairB;           // of two pages
  static constexpr int kHalfScales = 2 * kScales * 2;  // both pages' V scales as float16
  static constexpr int kRingB = 2 * kStageB + kHalfScales;
  static constexpr int kSmem = kWarps * kRingB;
  static constexpr int kTiles = D / 16;                // MMAs per page, of K and of V
  static constexpr int kRow = D + 8;                   // floats between the queries of a warp's output in shared memory
  static_assert(kRingB >= 8 * kRow * 4, "a warp's output takes its ring's place");
  static_assert(kSmem <= 47 * 1024, "no more than a launch gets unasked");
};

struct Fp4Params {
  const __nv_bfloat16* q;
  const uint8_t *k_cache, *v_cache;
  int64_t k_str, v_str;
  const float *k_scale, *v_scale;
  const int32_t *block_table, *seq_lens;
  __nv_bfloat16* out;
  float *o_part, *lse_part;
  int32_t* prefix;  // [B + 1]: attended pages of the sequences before b
  int B, Hq, Hkv, g, max_blocks;
  int64_t num_blocks;
  float sm_scale;
  int window;
  int* dev_status;
};

// Attended tokens [lo, len) of a sequence, and their pages [first, first + n).
struct Span {
  int lo, len, first, n;
};
// early: before the preceding kernel has completed (the value may still change, and
// leaves no line in L1).
KVQ_DEVINL Span span_of(const Fp4Params& p, int b, bool report = false, bool early = false) {
  Span s;
  const int L = early ? ld_l2only_s32(p.seq_lens + b) : p.seq_lens[b];
  s.len = min(max(L, 0), p.max_blocks * kPage);
  if (report && s.len != L) set_status(p.dev_status, KVQ_DEV_BAD_SEQLEN);
  s.lo = p.window > 0 && s.len > p.window ? s.len - p.window : 0;
  s.first = s.lo / kPage;
  s.n = (s.len + kPage - 1) / kPage - s.first;
  return s;
}
// Pages of a part: the stream in `parts` equal ones, but at least a page per warp.
KVQ_DEVINL int part_pages(int total, int parts) { return max(kMinPart, (total + parts - 1) / parts); }

// Where a CTA's part [pos, end) of the page stream begins: in sequence b, `before`
// pages (of one KV head) after the stream's start.  A warp finds it alone.
struct Part {
  int pos, end, b, before;
};
KVQ_DEVINL Part find_part(const Fp4Params& p, int lane, bool first_cta, bool early) {
  const int per = (p.B + 31) / 32;
  const int b0 = min(p.B, lane * per), b1 = min(p.B, b0 + per);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += span_of(p, b, first_cta, early).n;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  const int total = __shfl_sync(0xffffffffu, incl, 31);
  if (first_cta) {  // for the combine
    int x = incl - mine;
    for (int b = b0; b < b1; ++b) {
      p.prefix[b] = x;
      x += span_of(p, b).n;
    }
    if (lane == 0) p.prefix[p.B] = total;
  }
  Part r;
  const int chunk = part_pages(total * p.Hkv, gridDim.x);
  r.pos = blockIdx.x * chunk;
  r.end = min(total * p.Hkv, r.pos + chunk);
  r.b = r.before = 0;
  if (r.pos >= r.end) return r;
  // the lane whose sequences hold the part's first page looks for the one
  const bool here = r.pos >= (incl - mine) * p.Hkv && r.pos < incl * p.Hkv;
  int b = b0, x = incl - mine;
  if (here) {
    for (;; ++b) {
      const int n = span_of(p, b, false, early).n;
      if (r.pos < (x + n) * p.Hkv || b + 1 >= b1) break;  // the second: lengths that change meanwhile (early)
      x += n;
    }
  }
  const int who = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  r.b = __shfl_sync(0xffffffffu, b, who);
  r.before = __shfl_sync(0xffffffffu, x, who);
  return r;
}

// While the preceding kernel still runs: brings the first pages of a CTA's part
// into L2.  A hint: what it reads may still change and is read again, and the
// addresses stay inside the table and the caches whatever it holds.
template <int D>
KVQ_DEVINL void hint_pages(const Fp4Params& p, int lane) {
  const Part part = find_part(p, lane, false, true);
  if (part.pos >= part.end) return;
  const Span sp = span_of(p, part.b, false, true);
  if (sp.n == 0) return;
  const int within = max(0, part.pos - part.before * p.Hkv);
  const int h = min(within / sp.n, p.Hkv - 1), pg = within % sp.n + lane;
  if (pg >= sp.n || pg - lane + part.pos >= part.end || lane >= kHinted) return;
  const int id = ld_l2only_s32(p.block_table + static_cast<int64_t>(part.b) * p.max_blocks + min(sp.first + pg, p.max_blocks - 1));
  if (static_cast<unsigned>(id) >= static_cast<uint64_t>(p.num_blocks)) return;
  const int64_t page = static_cast<int64_t>(id) * p.Hkv + h;
  prefetch_l2(p.k_cache + page * p.k_str, Fp4<D>::kPageB);
  prefetch_l2(p.v_cache + page * p.v_str, Fp4<D>::kPageB);
}

KVQ_DEVINL void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
KVQ_DEVINL uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// The four bytes of a word, each two E2M1 codes, as f16x2 (low nibble in the low half).
KVQ_DEVINL void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Bytes 1 and 3 of a word.
KVQ_DEVINL void e2m1x4_to_f16x2(uint32_t w, uint32_t& h1, uint32_t& h3) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b;\n\tcvt.rn.f16x2.e2m1x2 %1, d;\n\t}"
      : "=r"(h1), "=r"(h3)
      : "r"(w));
}
// Two E4M3 codes as f16x2.
KVQ_DEVINL uint32_t e4m3x2_to_f16x2(uint32_t x) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(x));
  return h;
}
KVQ_DEVINL uint32_t both(uint32_t h, bool high) { return __byte_perm(h, h, high ? 0x3232 : 0x1010); }

// A warp's state for the queries of one KV head: lane 4 r + c holds the
// stabilizers and sums of queries 2c, 2c + 1 and, per 16 dims, the outputs
// O[.][0], O[.][1] of dim 2r and O[.][2], O[.][3] of dim 2r + 1.
template <int D>
struct Attend {
  using F = Fp4<D>;
  uint32_t q[D / 8];  // query r, dims (D / 4) c .. + D / 4 - 1
  float coef[2];
  float m[2], mb[2], l[2];  // mb: m - kBase, or kNone, which any score passes
  float O[F::kTiles][4];

  KVQ_DEVINL void start(const Fp4Params& p, int b, int h, int lane) {
    const int r = lane >> 2, c = lane & 3;
    const bool live = r < p.g;
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(b) * p.Hq + h * p.g + (live ? r : 0)) * D +
                                                      c * (D / 4));
    float mx = 0.f;
    float2 x[D / 32][4];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      unpack8_bf16(live ? src[i] : make_uint4(0, 0, 0, 0), x[i]);
      mx = fmaxf(mx, amax8(x[i]));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    int e2 = mx > 0.f ? static_cast<int>((__float_as_uint(mx) >> 23) & 0xFF) - 127 : 0;
    e2 = max(e2, -100);
    const float sigma = __uint_as_float(static_cast<uint32_t>(127 + 7 - e2) << 23);
    const float inv_sigma = __uint_as_float(static_cast<uint32_t>(127 - 7 + e2) << 23);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) q[4 * i + e] = pack_f16x2(x[i][e].x * sigma, x[i][e].y * sigma);
    const float cf = __fmul_rn(__fmul_rn(p.k_scale[h], p.sm_scale), kLog2e);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      coef[i] = cf * __shfl_sync(0xffffffffu, inv_sigma, 8 * c + 4 * i);
      if (coef[i] < kLeast) coef[i] = kLeast;
      m[i] = NEG_INF;
      mb[i] = kNone;
      l[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < F::kTiles; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) O[i][e] = 0.f;
  }

  // Two pages at shared address `stage`; tokens [lo[i], hi[i]) of page i are live
  // (edge: not all are).  `half`: room for V's scales as float16.
  KVQ_DEVINL void take(uint32_t stage, uint32_t half, bool edge, const int (&lo)[2], const int (&hi)[2], int lane) {
    const int r = lane >> 2, c = lane & 3;
    // ---- V's scales, eight to a lane, as float16 for all; those of masked tokens may be anything: zero
    {
      constexpr int kLanes = F::kScales / 8;  // per page
      const int pg = lane / kLanes;           // D = 64: the upper half of the lanes has none
      if (pg < 2) {
        uint2 w = lds64(stage + pg * F::kPairB + F::kPageB + F::kCodes + lane % kLanes * 8);
        if (edge) {
          uint32_t keep = 0xffffffffu;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = 2 * ((lane >> 1) & 3) + (e & 1) + 8 * (e >> 1);
            if (t < (pg ? lo[1] : lo[0]) || t >= (pg ? hi[1] : hi[0])) keep &= ~(0xffu << (8 * e));
          }
          w.x &= keep;
          w.y &= keep;
        }
        uint4 h;
        e4m3x4_to_f16x2x2(w.x, h.x, h.y);
        e4m3x4_to_f16x2x2(w.y, h.z, h.w);
        sts128(half + lane * 16, h);
      }
    }
    // ---- scores: rows are tokens, and each lane's dims share two scales (one at D = 64) per row
    float t[2][4];
#pragma unroll
    for (int pg = 0; pg < 2; ++pg) {
      const uint32_t page = stage + pg * F::kPairB;
      uint32_t kw[2][D / 32], ks[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = r + 8 * i;
        if constexpr (D == 128) {
          const uint4 u = lds128(page + tok * 64 + c * 16);
          kw[i][0] = u.x;
          kw[i][1] = u.y;
          kw[i][2] = u.z;
          kw[i][3] = u.w;
          const uint32_t s = e4m3x2_to_f16x2(lds16(page + F::kCodes + tok * 8 + 2 * c));
          ks[i][0] = both(s, false);
          ks[i][1] = both(s, true);
        } else {
          const uint2 u = lds64(page + tok * 32 + c * 8);
          kw[i][0] = u.x;
          kw[i][1] = u.y;
          ks[i][0] = ks[i][1] = both(e4m3x2_to_f16x2(lds8(page + F::kCodes + tok * 4 + c)), false);
        }
      }
      float s[2][4] = {};
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        uint32_t a[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          e2m1x8_to_f16x2(kw[i][w], a[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) a[i][e] = hmul2(a[i][e], ks[i][w / 2]);
        }
        mma_f16(s[0], a[0][0], a[1][0], a[0][1], a[1][1], q[4 * w], q[4 * w + 1], s[0]);
        mma_f16(s[1], a[0][2], a[1][2], a[0][3], a[1][3], q[4 * w + 2], q[4 * w + 3], s[1]);
      }
      // [0], [1]: token r, queries 2c, 2c + 1; [2], [3]: token r + 8
#pragma unroll
      for (int e = 0; e < 4; ++e) t[pg][e] = s[0][e] + s[1][e];
      if (edge) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = r + 8 * (e >> 1);
          if (tok < lo[pg] || tok >= hi[pg]) t[pg][e] = NEG_INF;
        }
      }
    }
    // ---- stabilizer: moved only when a score passes it by more than kLag
    float x[2][4];
#pragma unroll
    for (int pg = 0; pg < 2; ++pg)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[pg][e] = fmaf(t[pg][e], coef[e & 1], -mb[e & 1]);
    const float top = fmax3(fmax3(x[0][0], x[0][2], fmaxf(x[1][0], x[1][2])), x[0][1], fmax3(x[0][3], x[1][1], x[1][3]));
    if (__any_sync(0xffffffffu, top > kLag + kBase)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float n = fmaxf(fmaxf(t[0][i], t[0][2 + i]), fmaxf(t[1][i], t[1][2 + i])) * coef[i];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
        n = fmaxf(n, m[i]);
        if (n > m[i]) {  // the same in every lane of the query
          const float alpha = ex2(m[i] - n);
          l[i] *= alpha;
#pragma unroll
          for (int d = 0; d < F::kTiles; ++d) {
            O[d][i] *= alpha;
            O[d][2 + i] *= alpha;
          }
          m[i] = n;
          mb[i] = n - kBase;
        }
      }
#pragma unroll
      for (int pg = 0; pg < 2; ++pg)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[pg][e] = fmaf(t[pg][e], coef[e & 1], -mb[e & 1]);
    }
    uint32_t p[2][2];
#pragma unroll
    for (int pg = 0; pg < 2; ++pg) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[pg][e] = ex2(x[pg][e]);
      l[0] += x[pg][0] + x[pg][2];
      l[1] += x[pg][1] + x[pg][3];
      p[pg][0] = movmatrix_t(pack_f16x2(x[pg][0], x[pg][1]));
      p[pg][1] = movmatrix_t(pack_f16x2(x[pg][2], x[pg][3]));
    }
    // ---- outputs: rows are 16 dims that share a token's scale, which multiplies the weights
    __syncwarp();  // the scales are there
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
#pragma unroll
      for (int quad = 0; quad < 2; ++quad) {
        float f[2][4] = {};
#pragma unroll
        for (int pg = 0; pg < 2; ++pg) {
          const uint2 codes = lds64(stage + pg * F::kPairB + F::kPageB + h * 512 + lane * 16 + quad * 8);
          const uint4 scales = lds128(half + pg * (2 * F::kScales) + h * 128 + c * 32 + quad * 16);
          const uint32_t cw[2] = {codes.x, codes.y};
          const uint32_t sw[2][2] = {{scales.x, scales.y}, {scales.z, scales.w}};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // bytes are tokens, nibbles dims 2r and 2r + 1: bytes 1 and 3 of `even`
            // (`odd`) become dim 2r (2r + 1) of tokens 2c, 2c + 1 and of 2c + 8, 2c + 9
            constexpr uint32_t kHigh = 0xF000F000u;
            const uint32_t w4 = cw[i] << 4, w8 = cw[i] << 8;
            const uint32_t even = (w4 & kHigh) | (w8 & ~kHigh), odd = (cw[i] & kHigh) | (w4 & ~kHigh);
            uint32_t a0, a1, a2, a3;
            e2m1x4_to_f16x2(even, a0, a2);
            e2m1x4_to_f16x2(odd, a1, a3);
            mma_f16(f[i], a0, a1, a2, a3, hmul2(p[pg][0], sw[i][0]), hmul2(p[pg][1], sw[i][1]), f[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float(&o)[4] = O[h * 4 + quad * 2 + i];
          const float2 u = fadd2(make_float2(o[0], o[1]), make_float2(f[i][0], f[i][1]));
          const float2 z = fadd2(make_float2(o[2], o[3]), make_float2(f[i][2], f[i][3]));
          o[0] = u.x;
          o[1] = u.y;
          o[2] = z.x;
          o[3] = z.y;
        }
      }
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) decode_fp4_kernel(const Fp4Params p) {
  using F = Fp4<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float s_m[kWarps][8], s_l[kWarps][8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kWarps - 1) hint_pages<D>(p, lane);
  grid_dependency_wait();
  grid_launch_dependents();
  const Part part = find_part(p, lane, blockIdx.x == 0 && warp == 0, false);
  int pos = part.pos, b = part.b, before = part.before;
  const int end = part.end;
  if (pos >= end) return;

  const uint32_t ring = smem_u32(smem) + warp * F::kRingB;
  float* const stage = reinterpret_cast<float*>(smem + warp * F::kRingB);
  Attend<D> at;

  while (pos < end) {
    const Span sp = span_of(p, b);
    if (sp.n == 0) {  // to the next sequence with pages (there is one: pos < end)
      do {
        ++b;
        const unsigned has = __ballot_sync(0xffffffffu, b + lane < p.B && span_of(p, min(b + lane, p.B - 1)).n > 0);
        b += has ? __ffs(has) - 1 : 31;
        if (has) break;
      } while (true);
      continue;
    }
    const int within = pos - before * p.Hkv;
    const int h = within / sp.n, pg0 = within % sp.n;
    const int n = min(end - pos, sp.n - pg0);
    const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks + sp.first + pg0;

    // ---- this warp's pairs of pages: pairs warp, warp + kWarps, ...
    const int pairs = (n + 1) / 2;
    const int count = pairs > warp ? (pairs - warp + kWarps - 1) / kWarps : 0;
    int ids = -1;        // block ids of 16 pairs, one page per lane
    unsigned valid = 0;  // bit 2 s + i: page i of stage s is there
    auto issue = [&](int i) {
      if (i < count) {
        if ((i & 15) == 0) {
          const int j = i + (lane >> 1), page = 2 * (warp + j * kWarps) + (lane & 1);
          ids = j < count && page < n ? table[page] : -1;
        }
        const int st = i & 1;
        valid &= ~(3u << (2 * st));
#pragma unroll
        for (int pg = 0; pg < 2; ++pg) {
          const int id = __shfl_sync(0xffffffffu, ids, 2 * (i & 15) + pg);
          if (static_cast<unsigned>(id) < static_cast<uint64_t>(p.num_blocks)) {
            valid |= 1u << (2 * st + pg);
            const int64_t page = static_cast<int64_t>(id) * p.Hkv + h;
            const uint8_t* k = p.k_cache + page * p.k_str + lane * 16;
            const uint8_t* v = p.v_cache + page * p.v_str + lane * 16;
            const uint32_t at = ring + st * F::kStageB + pg * F::kPairB + lane * 16;
#pragma unroll
            for (int x = 0; x < F::kPageB; x += 512) {
              if (x + 512 <= F::kPageB || x + lane * 16 < F::kPageB) {
                copy16(at + x, k + x);
                copy16(at + F::kPageB + x, v + x);
              }
            }
          } else if (lane == 0 && 2 * (warp + i * kWarps) + pg < n) {
            set_status(p.dev_status, KVQ_DEV_BAD_BLOCK);
          }
        }
      }
      copy_commit();
    };
    issue(0);
    issue(1);
    at.start(p, b, h, lane);
    for (int i = 0; i < count; ++i) {
      copy_wait<1>();
      __syncwarp();  // every lane's copies are there
      const int st = i & 1;
      const unsigned have = valid >> (2 * st) & 3;
      if (have) {
        const int tok = (sp.first + pg0 + 2 * (warp + i * kWarps)) * kPage;
        int lo[2], hi[2];
#pragma unroll
        for (int pg = 0; pg < 2; ++pg) {
          lo[pg] = sp.lo - tok - pg * kPage;
          hi[pg] = have >> pg & 1 ? sp.len - tok - pg * kPage : 0;
        }
        const bool edge = lo[0] > 0 || lo[1] > 0 || hi[0] < kPage || hi[1] < kPage;
        at.take(ring + st * F::kStageB, ring + 2 * F::kStageB, edge, lo, hi, lane);
      }
      __syncwarp();  // every lane is done with the stage
      issue(i + 2);
    }
    copy_wait<0>();
    __syncwarp();

    // ---- the piece's end: the warps' states meet
    {
      const int r = lane >> 2, c = lane & 3;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) at.l[i] += __shfl_xor_sync(0xffffffffu, at.l[i], o);
        if (r == 0) {
          s_m[warp][2 * c + i] = at.m[i];
          s_l[warp][2 * c + i] = at.l[i];
        }
#pragma unroll
        for (int d = 0; d < F::kTiles; ++d)
          *reinterpret_cast<float2*>(stage + (2 * c + i) * F::kRow + 16 * d + 2 * r) = make_float2(at.O[d][i], at.O[d][2 + i]);
      }
    }
    __syncthreads();
    const bool direct = n == sp.n;  // all of the sequence and KV head
    const int64_t id = blockIdx.x + static_cast<int64_t>(b) * p.Hkv + h;
    const float vs = p.v_scale[h];
    for (int x = tid; x < p.g * D; x += kWarps * 32) {
      const int qh = x / D, d = x % D;
      float M = NEG_INF;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][qh]);
      float l = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = s_m[w][qh] == NEG_INF ? 0.f : ex2(s_m[w][qh] - M);
        l = fmaf(s_l[w][qh], f, l);
        if (f != 0.f) o = fmaf(reinterpret_cast<const float*>(smem + w * F::kRingB)[qh * F::kRow + d], f, o);
      }
      o = l > 0.f || l != l ? o / l * vs : 0.f;
      if (direct) {
        p.out[(static_cast<int64_t>(b) * p.Hq + h * p.g + qh) * D + d] = __float2bfloat16(o);
      } else {
        p.o_part[(id * p.g + qh) * D + d] = o;
        if (d == 0) p.lse_part[id * p.g + qh] = l > 0.f || l != l ? M + log2f(l) : NEG_INF;
      }
    }
    __syncthreads();
    pos += n;
    if (within + n == sp.n * p.Hkv) {
      before += sp.n;
      ++b;
    }
  }
}

// Joins the pieces of a row: a CTA per (sequence, query head).  A warp loads
// kAtOnce pieces' log-sum-exps and outputs together, so that a row of up to NW *
// kAtOnce pieces takes one round trip to L2, then joins them against their own
// maximum; the warps meet in shared memory.
constexpr int kAtOnce = 5;
template <int D, int NW>
__global__ void __launch_bounds__(NW * 32) decode_fp4_combine_kernel(const Fp4Params p, int parts) {
  __shared__ float s_max[NW], s_l[NW];
  __shared__ __align__(16) float s_o[NW][D];
  constexpr int V = D / 32;
  using Vec = typename std::conditional<V == 4, float4, float2>::type;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.Hq, hq = blockIdx.x % p.Hq;
  const int h = hq / p.g, qh = hq % p.g;
  grid_dependency_wait();
  grid_launch_dependents();  // the next call's CTAs may come; they wait for this kernel's end
  const int total = p.prefix[p.B], before = p.prefix[b], n = p.prefix[b + 1] - before;
  __nv_bfloat16* out = p.out + (static_cast<int64_t>(b) * p.Hq + hq) * D;
  if (n == 0) {
    for (int d = threadIdx.x; d < D; d += NW * 32) out[d] = __float2bfloat16(0.f);
    return;
  }
  const int chunk = part_pages(total * p.Hkv, parts);
  const int x = before * p.Hkv + h * n;
  const int first = x / chunk, last = (x + n - 1) / chunk;
  if (first == last) return;  // written where it was computed
  const int64_t row = (first + static_cast<int64_t>(b) * p.Hkv + h) * p.g + qh;
  const int count = last - first + 1;
  float m = NEG_INF, l = 0.f, acc[V] = {};
  for (int i0 = warp; i0 < count; i0 += NW * kAtOnce) {
    float e[kAtOnce];
    Vec o[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + k * NW;
      const int64_t at = row + static_cast<int64_t>(min(i, count - 1)) * p.g;
      e[k] = i < count ? p.lse_part[at] : NEG_INF;
      o[k] = reinterpret_cast<const Vec*>(p.o_part + at * D)[lane];
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, e[k]);
    const float base = top == NEG_INF ? 0.f : top;
    const float alpha = ex2(m - base);
    m = top;
    l *= alpha;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= alpha;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const float f = ex2(e[k] - base);
      l += f;
      const float* ov = reinterpret_cast<const float*>(&o[k]);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(ov[v], f, acc[v]);
    }
  }
  if (lane == 0) {
    s_max[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) s_o[warp][lane * V + v] = acc[v];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += NW * 32) {
    float top = NEG_INF;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, s_max[w]);
    const float base = top == NEG_INF ? 0.f : top;
    float sum = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = ex2(s_max[w] - base);
      sum = fmaf(s_l[w], f, sum);
      y = fmaf(s_o[w][d], f, y);
    }
    out[d] = __float2bfloat16(sum > 0.f || sum != sum ? y / sum : 0.f);
  }
}

// CTAs of a call: one wave, and no more than parts of kMinPart pages.
int fp4_parts(int B, int Hkv, int max_blocks) {
  const int64_t most = (static_cast<int64_t>(B) * Hkv * max_blocks + kMinPart - 1) / kMinPart;
  return static_cast<int>(std::min<int64_t>(static_cast<int64_t>(kCtasPerSm) * sm_count(), most));
}
// Rows of partials: piece (part, sequence and KV head) is row part + pair.
int64_t fp4_rows(int B, int Hq, int Hkv, int max_blocks) {
  return (fp4_parts(B, Hkv, max_blocks) + static_cast<int64_t>(B) * Hkv) * (Hq / Hkv);
}
bool fp4_sizes_ok(int B, int Hq, int Hkv, int D, int P, int max_blocks) {
  return B >= 1 && Hq >= 1 && Hkv >= 1 && max_blocks >= 1 && Hq % Hkv == 0 && (D == 64 || D == 128) && P == kPage;
}

template <int D>
kvq_status_t launch_fp4(const Fp4Params& p, cudaStream_t s) {
  using F = Fp4<D>;
  auto kern = decode_fp4_kernel<D>;
  const int parts = fp4_parts(p.B, p.Hkv, p.max_blocks);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = F::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return cuda_status(e, "paged_decode_fp4 launch");
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Hq);
  cfg.dynamicSmemBytes = 0;
  // warps for the pieces of a row
  if (parts / (static_cast<int64_t>(p.B) * p.Hkv) >= 8) {
    cfg.blockDim = dim3(16 * 32);
    e = cudaLaunchKernelEx(&cfg, decode_fp4_combine_kernel<D, 16>, p, parts);
  } else {
    cfg.blockDim = dim3(4 * 32);
    e = cudaLaunchKernelEx(&cfg, decode_fp4_combine_kernel<D, 4>, p, parts);
  }
  return cuda_status(e, "paged_decode_fp4 combine launch");
}

}  // namespace

}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_decode_fp4_workspace_size(int B, int Hq, int Hkv, int D, int P, int max_blocks) {
  if (!fp4_sizes_ok(B, Hq, Hkv, D, P, max_blocks)) return 0;
  const int64_t rows = fp4_rows(B, Hq, Hkv, max_blocks);
  return static_cast<size_t>((rows * (D + 1) + B + 1) * 4 + 15) / 16 * 16;
}

extern "C" kvq_status_t kvq_paged_decode_attention_fp4(const void* q, const void* k_cache, const void* v_cache,
                                                       const float* k_scale, const float* v_scale,
                                                       const int32_t* block_table, const int32_t* seq_lens, void* out,
                                                       int B, int Hq, int Hkv, int D, int P, int max_blocks,
                                                       int64_t num_blocks, float sm_scale, int window, void* workspace,
                                                       size_t workspace_bytes, int* dev_status, kvq_stream_t stream) {
  clear_error();
  if (B < 1 || Hq < 1 || Hkv < 1 || max_blocks < 1 || num_blocks < 1 || Hq % Hkv != 0)
    return fail(KVQ_ERR_INVALID_ARG, "paged_decode_fp4: bad sizes");
  if (window == 0 || window < -1) return fail(KVQ_ERR_INVALID_ARG, "paged_decode_fp4: window must be -1 or > 0");
  if (!(sm_scale > 0.f) || !(sm_scale < FLT_MAX)) return fail(KVQ_ERR_INVALID_ARG, "paged_decode_fp4: bad sm_scale");
  if (P != kPage) return fail(KVQ_ERR_UNSUPPORTED, "paged_decode_fp4: page size %d (only 16)", P);
  if (D != 64 && D != 128) return fail(KVQ_ERR_UNSUPPORTED, "paged_decode_fp4: head_dim %d (64 or 128)", D);
  if (Hq / Hkv > 8) return fail(KVQ_ERR_UNSUPPORTED, "paged_decode_fp4: GQA ratio %d > 8", Hq / Hkv);
  // positions in the stream of pages, and tokens, are 32-bit
  if (static_cast<int64_t>(max_blocks) * kPage > 0x7FFFFFFF - kPage || static_cast<int64_t>(B) * Hq > 0x7FFFFFFF ||
      static_cast<double>(B) * Hkv * max_blocks > 0x7FFFFFFF - 65536.0)
    return fail(KVQ_ERR_UNSUPPORTED, "paged_decode_fp4: problem too large");
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !out || !workspace)
    return fail(KVQ_ERR_INVALID_ARG, "paged_decode_fp4: null pointer");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(workspace, 16) || !aligned(out, 4) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return fail(KVQ_ERR_INVALID_ARG, "paged_decode_fp4: misaligned pointer");
  const size_t need = kvq_decode_fp4_workspace_size(B, Hq, Hkv, D, P, max_blocks);
  if (workspace_bytes < need)
    return fail(KVQ_ERR_INVALID_ARG, "paged_decode_fp4: workspace %zu bytes < %zu needed", workspace_bytes, need);
  const int64_t rows = fp4_rows(B, Hq, Hkv, max_blocks);
  Fp4Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  const PageStrides ps = page_strides(k_cache, v_cache, k_page_bytes(kFP4, D), v_page_bytes(kFP4, D));
  p.k_str = ps.k;
  p.v_str = ps.v;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.o_part = static_cast<float*>(workspace);
  p.lse_part = p.o_part + rows * D;
  p.prefix = reinterpret_cast<int32_t*>(p.lse_part + rows);
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.g = Hq / Hkv;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.sm_scale = sm_scale;
  p.window = window;
  p.dev_status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return D == 128 ? launch_fp4<128>(p, s) : launch_fp4<64>(p, s);
}
