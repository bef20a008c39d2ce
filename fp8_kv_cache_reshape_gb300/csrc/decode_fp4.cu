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
// Bound: memory in principle, 9/16 byte per element of K and V; in practice latency, with
// three warps a scheduler: no unit is full (issue slots 59%, ALU pipe 49%: half of it the
// conversions, an instruction for two codes; tensor pipe 22%).  Over longer contexts a call grows
// by 28 us per 128K tokens of 8 KV heads of 128, 5.5 TB/s; with the scores alone, or the
// outputs alone, it grows by 22, the copies' own time.  One request of 128K: 38.5 us, 3.9 TB/s with
// its fixed part of about 10; eight of 20K: 48.3 us, 4.0 TB/s; 64 of 500 to 1,000: 24 us for a
// floor of 8.
//
// Layout.  A warp takes two pages (32 tokens of a KV head) at a time from stages
// of its own in shared memory, filled by 16-byte asynchronous copies: no barrier,
// no producer warp, nothing between warps but the joining at the end.  The page
// format is the MMA operand order (m16n8k16, tokens as the rows of K Q^T, dims as the
// rows of V^T P^T), so that a lane reads its share of a page with wide loads: lane 4 r + c
// holds dims 32 c .. 32 c + 31 (at head dim 128) of tokens r and r + 8 of K, and
// tokens 2c, 2c + 1, 2c + 8, 2c + 9 of dims 2r, 2r + 1 of each 16 of V.
//
// The page stream.  All sequences' and KV heads' attended pages end to end, cut
// into one part per warp; a part's share of a (sequence, KV head) is a piece.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <type_traits>

#include "kvq_host.h"
#include "kvq_rows.cuh"

namespace kvq {

namespace {

constexpr int kWarps = kStreamWarps;  // warps per CTA, each with a ring of its own
constexpr int kCtasPerSm = 3;         // 168 registers a thread (four, with 128 and spills, at an earlier step: 128K 42.2 against 40.2 us)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLag = 3.f;           // by how much scores may pass the stabilizer
// Weights are 2^(s2 - M + base): below 2^16 / 2 ^ (exponent of V's largest block scale), so
// that their products with block scales stay within float16, and as large as that allows,
// so that they stay out of its subnormal numbers: 12 for scales below 2, 4 for those from 256 on.
constexpr float kBase = 12.f;
constexpr int kUnit = 7;  // exponent field of scales in [1, 2)
// The stabilizer before the first score: any score passes it, by an amount whose product
// with a coefficient of kLeast or more passes kLag.
constexpr float kNone = -FLT_MAX;
// Sums of code products are below 2^27, so a smaller coefficient gives scores of zero
// either way; one of zero would make a masked score, minus infinity, no number.
constexpr float kLeast = 1e-30f;
#define NEG_INF __int_as_float(0xff800000)

template <int D>
struct Fp4 {
  static constexpr int kCodes = kPage * D / 2;
  static constexpr int kScales = kPage * D / 16;
  static constexpr int kPageB = kCodes + kScales;
  static_assert(kPageB % 64 == 0, "pages lie at multiples of 64 bytes");
  static constexpr int kPairB = 2 * kPageB;            // K page, V page
  static constexpr int kStageB = 2 * kPairB;           // of two pages
  static constexpr int kStages = 3;                    // scores taken, outputs taken, in flight
  static constexpr int kHalfScales = 2 * kScales * 2;  // both pages' V scales as float16
  static constexpr int kRingB = kStages * kStageB + 2 * kHalfScales;
  static constexpr int kSmem = kWarps * kRingB;
  static constexpr int kTiles = D / 16;                // MMAs per page, of K and of V
  static constexpr int kRow = D + 8;                   // floats between the queries of a warp's output in shared memory
  static_assert(kRingB >= 8 * kRow * 4, "a warp's output takes its ring's place");
  static_assert(kCtasPerSm * (kSmem + 2048) <= 227 * 1024, "the CTAs of an SM");
};

struct Fp4Params {
  const __nv_bfloat16* q;
  const uint8_t *k_cache, *v_cache;
  int64_t str;  // bytes between pages, of both caches
  const float *k_scale, *v_scale;
  const int32_t *block_table, *seq_lens;
  __nv_bfloat16* out;
  float *o_part, *lse_part;
  int32_t* prefix;  // [B + 1]: attended pages of the sequences before b, for the combine
  int B, Hq, Hkv, g, max_blocks;
  int parts;  // of the page stream, a warp each
  int64_t num_blocks;
  float sm_scale;
  int window;
  int* dev_status;
};

// Attended tokens [lo, len) of a sequence, and their pages [first, first + n).
struct Span {
  int lo, len, first, n;
};
KVQ_DEVINL Span span_of(const Fp4Params& p, int b, bool report = false) {
  Span s;
  const int L = p.seq_lens[b];
  s.len = min(max(L, 0), p.max_blocks * kPage);
  if (report && s.len != L) set_status(p.dev_status, KVQ_DEV_BAD_SEQLEN);
  s.lo = p.window > 0 && s.len > p.window ? s.len - p.window : 0;
  s.first = s.lo / kPage;
  s.n = (s.len + kPage - 1) / kPage - s.first;
  return s;
}
// Where a warp's part [pos, end) of the page stream begins: in sequence b, `before`
// pages (of one KV head) after the stream's start.  Lengths that another stream
// changes while the call runs give wrong results, but every loop here ends, every
// address stays inside its table, and the warps of a CTA agree on who waits for whom.
struct Part {
  int pos, end, b, before;
  int chunk, total;  // pages of a part, of the stream
};
KVQ_DEVINL int scan_add(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
KVQ_DEVINL Part find_part(const Fp4Params& p, int index, int lane) {
  const int n0 = lane < p.B ? span_of(p, lane, index == 0).n : 0;  // of the first 32 sequences
  int sum = n0;
#pragma unroll 4
  for (int b = lane + 32; b < p.B; b += 32) sum += span_of(p, b, index == 0).n;
  Part r;
  r.total = __reduce_add_sync(0xffffffffu, sum) * p.Hkv;
  r.chunk = part_pages(r.total, p.parts);
  r.pos = index * r.chunk;
  r.end = min(r.total, r.pos + r.chunk);
  r.b = r.before = 0;
  if (r.pos >= r.end) return r;
  for (int b0 = 0, x = 0; b0 < p.B; b0 += 32) {  // 32 sequences at a time
    const int n = b0 == 0 ? n0 : b0 + lane < p.B ? span_of(p, b0 + lane).n : 0;
    const int incl = x + scan_add(n, lane);
    const unsigned past = __ballot_sync(0xffffffffu, r.pos < incl * p.Hkv);
    if (past) {
      const int who = __ffs(past) - 1;
      r.b = b0 + who;
      r.before = __shfl_sync(0xffffffffu, incl - n, who);
      return r;
    }
    x = __shfl_sync(0xffffffffu, incl, 31);
  }
  r.end = r.pos;  // not there: lengths that changed meanwhile
  return r;
}

KVQ_DEVINL void write_prefix(const Fp4Params& p, int lane) {
  int x = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int n = b0 + lane < p.B ? span_of(p, b0 + lane).n : 0;
    const int incl = scan_add(n, lane);
    if (b0 + lane < p.B) p.prefix[b0 + lane] = x + incl - n;
    x += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) p.prefix[p.B] = x;
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

// What a stage in flight holds.
struct Meta {
  int b, h, tok;  // sequence, KV head, first token
  int flags;      // bit i: page i is there; the piece's first and last stage; all of (b, h); 0: none
};
constexpr uint32_t kNowhere = 0xffffffffu;
constexpr int kFirst = 4, kLast = 8, kWhole = 16, kStage = 32;

// A warp's state for the queries of one KV head: lane 4 r + c holds the
// stabilizers and sums of queries 2c, 2c + 1 and, per 16 dims, the outputs
// O[.][0], O[.][1] of dim 2r and O[.][2], O[.][3] of dim 2r + 1.
template <int D>
struct Attend {
  using F = Fp4<D>;
  uint32_t q[D / 8];  // query r, dims (D / 4) c .. + D / 4 - 1
  float coef[2], vs;
  float m[2], l[2];  // the stabilizer is m * coef: differences of scores are taken before the product, which rounds them
  float O[F::kTiles][4];
  float base;
  uint32_t room;     // four bytes, each from the first code that base has no room for to its sign bit
  uint32_t p[2][2];  // weights of the stage whose outputs are due

  // The queries as they are, and (begin) as the products take them.
  struct Raw {
    uint4 q[D / 32];
    float ks, vs;
  };
  KVQ_DEVINL static Raw fetch(const Fp4Params& prm, int b, int h, int lane) {
    const int r = lane >> 2, c = lane & 3;
    const bool live = r < prm.g;
    const uint4* src = reinterpret_cast<const uint4*>(
        prm.q + (static_cast<int64_t>(b) * prm.Hq + h * prm.g + (live ? r : 0)) * D + c * (D / 4));
    Raw raw;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) raw.q[i] = live ? src[i] : make_uint4(0, 0, 0, 0);
    raw.ks = prm.k_scale[h];
    raw.vs = prm.v_scale[h];
    return raw;
  }
  KVQ_DEVINL void begin(const Fp4Params& prm, const Raw& raw, int lane) {
    const int c = lane & 3;
    float mx = 0.f;
    float2 x[D / 32][4];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      unpack8_bf16(raw.q[i], x[i]);
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
    vs = raw.vs;
    const float cf = __fmul_rn(__fmul_rn(raw.ks, prm.sm_scale), kLog2e);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      coef[i] = cf * __shfl_sync(0xffffffffu, inv_sigma, 8 * c + 4 * i);
      if (coef[i] < kLeast) coef[i] = kLeast;
      m[i] = kNone;
      l[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < F::kTiles; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) O[i][e] = 0.f;
    base = kBase;
    room = (0x78 - 8 * kUnit) * 0x01010101u;
  }

  // All sums times f.
  KVQ_DEVINL void scale_sums(float f) {
    l[0] *= f;
    l[1] *= f;
#pragma unroll
    for (int d = 0; d < F::kTiles; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) O[d][e] *= f;
  }

  KVQ_DEVINL float stabilizer(int i) const { return m[i] == kNone ? NEG_INF : m[i] * coef[i]; }

  // The piece's output, normalized: to the output where it is all of the sequence
  // and KV head, else to the workspace with its log-sum-exp, and without V's head scale: the
  // sum of partials has the values' range then, however large or small that is.
  KVQ_DEVINL void finish(const Fp4Params& prm, int index, const Meta& meta, int lane) {
    const int r = lane >> 2, c = lane & 3;
    const int64_t id = index + static_cast<int64_t>(meta.b) * prm.Hkv + meta.h;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = l[i];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const bool any = sum > 0.f || sum != sum;
      const float f = any ? 1.f / sum : 0.f;
      const int qh = 2 * c + i;
      if (qh >= prm.g) continue;
      if (meta.flags & kWhole) {
        __nv_bfloat16* out = prm.out + (static_cast<int64_t>(meta.b) * prm.Hq + meta.h * prm.g + qh) * D + 2 * r;
#pragma unroll
        for (int d = 0; d < F::kTiles; ++d) {
          const float2 y = fmul2(fmul2(make_float2(O[d][i], O[d][2 + i]), make_float2(f, f)), make_float2(vs, vs));
          *reinterpret_cast<uint32_t*>(out + 16 * d) = any ? pack_bf16x2(y.x, y.y) : 0;
        }
      } else {
        float* out = prm.o_part + (id * prm.g + qh) * D + 2 * r;
#pragma unroll
        for (int d = 0; d < F::kTiles; ++d)
          *reinterpret_cast<float2*>(out + 16 * d) = make_float2(any ? O[d][i] * f : 0.f, any ? O[d][2 + i] * f : 0.f);
        if (r == 0) prm.lse_part[id * prm.g + qh] = any ? stabilizer(i) + (log2f(sum) - base) : NEG_INF;
      }
    }
  }

  // The state to shared memory, for the CTA's warps to join.
  KVQ_DEVINL void show(float* o, float* sm, float* sl, int lane) {
    const int r = lane >> 2, c = lane & 3;
    scale_sums(ex2(-base));  // the warps' may differ
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = l[i];
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      if (r == 0) {
        sm[2 * c + i] = stabilizer(i);
        sl[2 * c + i] = sum;
      }
#pragma unroll
      for (int d = 0; d < F::kTiles; ++d)
        *reinterpret_cast<float2*>(o + (2 * c + i) * F::kRow + 16 * d + 2 * r) = make_float2(O[d][i], O[d][2 + i]);
    }
  }

  // The stage's K against the queries: t[i][0], [1] of token r of page i, queries 2c,
  // 2c + 1; [2], [3] of token r + 8.
  KVQ_DEVINL void scores(uint32_t stage, float (&t)[2][4], int lane) const {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int pg = 0; pg < 2; ++pg) {
      const uint32_t page = stage + pg * F::kPairB;
      // each lane's dims share two scales (one at D = 64) per token
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
#pragma unroll
      for (int e = 0; e < 4; ++e) t[pg][e] = s[0][e] + s[1][e];
    }
  }

  // The weights p against the stage's V, whose scales are at `half`: rows are 16
  // dims that share a token's scale, which multiplies the weights.
  KVQ_DEVINL void outputs(uint32_t stage, uint32_t half, int lane) {
    const int c = lane & 3;
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

  // The stage's weights from its scores, and its V scales, eight to a lane, as float16 at
  // `half`.  Tokens [lo[i], hi[i]) of page i are live (edge: not all are); the
  // scales of the others may be anything and become zero.
  KVQ_DEVINL void weigh(uint32_t stage, uint32_t half, float (&t)[2][4], bool edge, const int (&lo)[2], const int (&hi)[2],
                        int lane) {
    const int r = lane >> 2;
    constexpr int kLanes = F::kScales / 8;  // per page
    const int at = lane / kLanes;           // D = 64: the upper half of the lanes has none
    uint2 w = make_uint2(0, 0);
    if (at < 2) w = lds64(stage + at * F::kPairB + F::kPageB + F::kCodes + lane % kLanes * 8);
    if (edge) {
      uint32_t keep = 0xffffffffu;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = 2 * ((lane >> 1) & 3) + (e & 1) + 8 * (e >> 1);
        if (tok < (at ? lo[1] : lo[0]) || tok >= (at ? hi[1] : hi[0])) keep &= ~(0xffu << (8 * e));
      }
      w.x &= keep;
      w.y &= keep;
#pragma unroll
      for (int pg = 0; pg < 2; ++pg)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = r + 8 * (e >> 1);
          if (tok < lo[pg] || tok >= hi[pg]) t[pg][e] = NEG_INF;
        }
    }
    uint4 hs;
    e4m3x4_to_f16x2x2(w.x, hs.x, hs.y);
    e4m3x4_to_f16x2x2(w.y, hs.z, hs.w);
    if (at < 2) sts128(half + lane * 16, hs);
    constexpr uint32_t kSign = 0x80808080u;
    const bool larger = (((w.x & ~kSign) + room) | ((w.y & ~kSign) + room)) & kSign;
    // stabilizer: moved only when a score passes it by more than kLag
    float x[2][4];
    auto exponents = [&] {
      const float2 minus = make_float2(-m[0], -m[1]), by = make_float2(coef[0], coef[1]), plus = make_float2(base, base);
#pragma unroll
      for (int pg = 0; pg < 2; ++pg)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float2 y = ffma2(fadd2(make_float2(t[pg][e], t[pg][e + 1]), minus), by, plus);
          x[pg][e] = y.x;
          x[pg][e + 1] = y.y;
        }
    };
    exponents();
    const float top = fmax3(fmax3(x[0][0], x[0][2], fmaxf(x[1][0], x[1][2])), x[0][1], fmax3(x[0][3], x[1][1], x[1][3]));
    if (__any_sync(0xffffffffu, top > kLag + base || larger)) {
      const uint32_t most = __vmaxu4(w.x & ~kSign, w.y & ~kSign);
      const uint32_t byte = max(max(most & 0xFF, most >> 8 & 0xFF), max(most >> 16 & 0xFF, most >> 24));
      const int unit = static_cast<int>(__reduce_max_sync(0xffffffffu, byte) >> 3);
      const float lower = kBase + static_cast<float>(kUnit - unit);
      if (lower < base) {
        scale_sums(ex2(lower - base));
        base = lower;
        room = (0x78 - 8 * unit) * 0x01010101u;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float n = fmaxf(fmaxf(t[0][i], t[0][2 + i]), fmaxf(t[1][i], t[1][2 + i]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
        if (n > m[i]) {  // the same in every lane of the query
          const float alpha = ex2((m[i] - n) * coef[i]);
          l[i] *= alpha;
#pragma unroll
          for (int d = 0; d < F::kTiles; ++d) {
            O[d][i] *= alpha;
            O[d][2 + i] *= alpha;
          }
          m[i] = n;
        }
      }
      exponents();
    }
#pragma unroll
    for (int pg = 0; pg < 2; ++pg) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[pg][e] = ex2(x[pg][e]);
      l[0] += x[pg][0] + x[pg][2];
      l[1] += x[pg][1] + x[pg][3];
      p[pg][0] = movmatrix_t(pack_f16x2(x[pg][0], x[pg][1]));
      p[pg][1] = movmatrix_t(pack_f16x2(x[pg][2], x[pg][3]));
    }
  }
};

// Walks the stream's pieces ((sequence, KV head) parts) two pages at a time and
// issues their copies; every lane of the warp takes part.
template <int D>
struct Feeder {
  using F = Fp4<D>;
  int pos, end, b, before;  // as Part
  int h, pg, stop;          // the piece: pages [.., stop) of KV head h, pg next
  Span sp;
  int flags;                // of the next stage: kFirst, kWhole
  int base, ahead;          // a lane's page: base + lane of the sequence's attended ones; block id of the one 32 on
  uint32_t place;           // 64-byte units into the caches, or kNowhere

  KVQ_DEVINL void piece(const Fp4Params& p, int lane) {
    const int within = pos - before * p.Hkv;
    h = sp.n > 0 && within >= 0 ? within / sp.n : p.Hkv;
    if (h >= p.Hkv) {  // lengths that changed meanwhile
      pos = end;
      return;
    }
    pg = within - h * sp.n;
    stop = min(sp.n, pg + end - pos);
    flags = kFirst | (stop - pg == sp.n ? kWhole : 0);
    base = pg - 32;
    ahead = id_of(p, pg + lane);
    // the piece's queries, which its first stage's taker reads
    const int bytes = p.g * D * 2;
    if (lane * 128 < bytes)
      prefetch_l2(reinterpret_cast<const uint8_t*>(p.q + (static_cast<int64_t>(b) * p.Hq + h * p.g) * D) + lane * 128, 128);
  }
  KVQ_DEVINL int id_of(const Fp4Params& p, int page) const {
    return page < stop ? p.block_table[static_cast<int64_t>(b) * p.max_blocks + sp.first + page] : -1;
  }
  KVQ_DEVINL void start(const Fp4Params& p, const Part& part, int lane) {
    pos = part.pos;
    end = part.end;
    b = part.b;
    before = part.before;
    h = 0;
    sp = span_of(p, b);
    if (pos < end) piece(p, lane);
  }
  // The next stage's copies (none when the part is through), as one group.
  KVQ_DEVINL void feed(const Fp4Params& p, uint32_t stage, Meta* meta, int lane) {
    if (pos < end) {
      const int n = min(2, stop - pg);
      if (pg + n > base + 32) {  // the next 32 pages, whose ids have come meanwhile
        base = pg;
        place = static_cast<unsigned>(ahead) < static_cast<uint64_t>(p.num_blocks)
                    ? static_cast<uint32_t>((static_cast<int64_t>(ahead) * p.Hkv + h) * p.str >> 6)
                    : kNowhere;
        ahead = id_of(p, pg + 32 + lane);
      }
      int has = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i >= n) break;
        const uint32_t at = __shfl_sync(0xffffffffu, place, pg + i - base);
        if (at != kNowhere) {
          has |= 1 << i;
          const uint8_t* k = p.k_cache + (static_cast<uint64_t>(at) << 6) + lane * 16;
          const uint8_t* v = p.v_cache + (static_cast<uint64_t>(at) << 6) + lane * 16;
          const uint32_t to = stage + i * F::kPairB + lane * 16;
#pragma unroll
          for (int x = 0; x < F::kPageB; x += 512) {
            if (x + 512 <= F::kPageB || x + lane * 16 < F::kPageB) {
              copy16(to + x, k + x);
              copy16(to + F::kPageB + x, v + x);
            }
          }
        } else if (lane == 0) {
          set_status(p.dev_status, KVQ_DEV_BAD_BLOCK);
        }
      }
      if (lane == 0) *meta = Meta{b, h, (sp.first + pg) * kPage, has | flags | kStage | (pg + n == stop ? kLast : 0)};
      flags &= ~kFirst;
      pg += n;
      pos += n;
      if (pg == stop && pos < end) {  // the next piece
        if (h + 1 == p.Hkv) {         // of the next sequence with pages
          before += sp.n;
          sp.n = 0;
          for (++b; b < p.B; b += 32) {
            const unsigned some = __ballot_sync(0xffffffffu, b + lane < p.B && span_of(p, min(b + lane, p.B - 1)).n > 0);
            if (some) {
              b += __ffs(some) - 1;
              sp = span_of(p, b);
              break;
            }
          }
        }
        piece(p, lane);
      }
    } else if (lane == 0) {
      meta->flags = 0;
    }
    copy_commit();
  }
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) decode_fp4_kernel(const Fp4Params p) {
  using F = Fp4<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Meta s_meta[kWarps][F::kStages];
  __shared__ float s_m[kWarps][8], s_l[kWarps][8];
  __shared__ int s_view[kWarps];   // each warp's: no part, a part of its own, one of those that may be joined
  __shared__ int s_first[kWarps];  // the (sequence, KV head) that it begins with
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int index = blockIdx.x * kWarps + warp;
  grid_dependency_wait();
  grid_launch_dependents();
  if (index == 0) write_prefix(p, lane);
  const Part part = find_part(p, index, lane);

  const uint32_t ring = smem_u32(smem) + warp * F::kRingB;
  Meta* const meta = s_meta[warp];
  Feeder<D> feeder;
  feeder.start(p, part, lane);
  // Are all of the CTA's parts, more than one, of one (sequence, KV head)?  Then
  // their states meet at the end: one row of partials instead of four.  The warps
  // tell each other, so that all of them go by the same answer.
  const int x0 = feeder.before * p.Hkv + feeder.h * feeder.sp.n;
  const bool some = part.pos < part.end;
  if (lane == 0) s_view[warp] = !some ? 0 : parts_join((index - warp) * part.chunk, part.chunk, part.total, x0, feeder.sp.n) ? 2 : 1;
  __syncthreads();
  if (!some) return;
  bool joined = true;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) joined = joined && s_view[w] != 1;
  const int part_b = feeder.b, part_h = min(feeder.h, p.Hkv - 1);
  if (lane == 0) s_first[warp] = part_b * p.Hkv + part_h;
  Span sp = feeder.sp;
  const typename Attend<D>::Raw raw = Attend<D>::fetch(p, part_b, part_h, lane);  // ahead of the copies
  feeder.feed(p, ring, meta, lane);
  feeder.feed(p, ring + F::kStageB, meta + 1, lane);
  // Stage i's scores are taken together with stage i - 1's outputs: two independent
  // chains of conversions and MMAs for a warp to fill its issue slots with.
  Attend<D> at;
  at.begin(p, raw, lane);
  Meta before;  // of stage i - 1
  before.flags = 0;
  uint32_t here = ring, prev = ring + 2 * F::kStageB;  // the stages' places
  const uint32_t halves = ring + F::kStages * F::kStageB;
  for (int i = 0;; ++i) {
    copy_wait<1>();
    __syncwarp();  // every lane's copies are there, the meta word, and the scales of stage i - 1
    const int st = i % F::kStages;
    const Meta m = meta[st];
    const uint32_t half = halves + (i & 1) * F::kHalfScales, half_before = halves + (~i & 1) * F::kHalfScales;
    float t[2][4];
    if (before.flags != 0 && (m.flags == 0 || m.flags & kFirst)) {  // the piece before is through
      at.outputs(prev, half_before, lane);
      if (joined) break;
      at.finish(p, index, before, lane);
    }
    if (m.flags == 0) {
      if (joined) break;  // a part without a stage: lengths that changed meanwhile
      return;
    }
    if (m.flags & kFirst) {
      if (i > 0) {
        at.begin(p, Attend<D>::fetch(p, m.b, m.h, lane), lane);
        sp = span_of(p, m.b);
      }
      at.scores(here, t, lane);
    } else {
      at.scores(here, t, lane);
      at.outputs(prev, half_before, lane);
    }
    int lo[2], hi[2];
#pragma unroll
    for (int pg = 0; pg < 2; ++pg) {
      lo[pg] = sp.lo - m.tok - pg * kPage;
      hi[pg] = m.flags >> pg & 1 ? sp.len - m.tok - pg * kPage : 0;
    }
    const bool edge = lo[0] > 0 || lo[1] > 0 || hi[0] < kPage || hi[1] < kPage;
    at.weigh(here, half, t, edge, lo, hi, lane);
    __syncwarp();  // every lane is done with stage i - 1
    feeder.feed(p, prev, meta + (st + 2) % F::kStages, lane);
    before = m;
    const uint32_t next = 3 * ring + 3 * F::kStageB - here - prev;  // the three places add up to this
    prev = here;
    here = next;
  }
  {
    copy_wait<0>();
    __syncwarp();  // the stages are read, and no copies are left in flight
    at.show(reinterpret_cast<float*>(smem + warp * F::kRingB), s_m[warp], s_l[warp], lane);
    int warps = 0;  // with a part: the first ones
#pragma unroll
    for (int w = 0; w < kWarps; ++w) warps += s_view[w] != 0;
    named_bar_sync(1, warps * 32);
    const int64_t id = index - warp + static_cast<int64_t>(s_first[warp]);
    for (int x = threadIdx.x; x < p.g * (D / 2); x += warps * 32) {  // two dims
      const int qh = x / (D / 2), d = x % (D / 2) * 2;
      float mw[kWarps], lw[kWarps];
      float2 ow[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const bool is = w < warps;
        mw[w] = is ? s_m[w][qh] : NEG_INF;
        lw[w] = is ? s_l[w][qh] : 0.f;
        ow[w] = is ? *reinterpret_cast<const float2*>(smem + w * F::kRingB + (qh * F::kRow + d) * 4) : make_float2(0.f, 0.f);
      }
      float M = mw[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) M = fmaxf(M, mw[w]);
      const float base = M == NEG_INF ? 0.f : M;
      float l = 0.f;
      float2 o = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(mw[w] - base);
        l = fmaf(lw[w], f, l);
        o = ffma2(ow[w], make_float2(f, f), o);
      }
      const bool any = l > 0.f || l != l;
      const float f = any ? 1.f / l : 0.f;
      *reinterpret_cast<float2*>(p.o_part + (id * p.g + qh) * D + d) = any ? make_float2(o.x * f, o.y * f) : make_float2(0.f, 0.f);
      if (d == 0) p.lse_part[id * p.g + qh] = any ? M + log2f(l) : NEG_INF;
    }
  }
}

// Joins the pieces of a row: a CTA per (sequence, query head) and W dims.  A warp loads
// kAtOnce pieces' log-sum-exps and outputs together, so that a row of up to NW *
// kAtOnce pieces takes one round trip to L2, then joins them against their own
// maximum; the warps meet in shared memory.
constexpr int kAtOnce = 8;
template <int D, int W, int NW>
__global__ void __launch_bounds__(NW * 32) decode_fp4_combine_kernel(const Fp4Params p) {
  __shared__ float s_max[NW], s_l[NW];
  __shared__ __align__(16) float s_o[NW][W];
  constexpr int V = W / 32;
  using Vec = typename std::conditional<V == 4, float4, typename std::conditional<V == 2, float2, float>::type>::type;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.Hq, hq = blockIdx.x % p.Hq, d0 = blockIdx.y * W;
  const int h = hq / p.g, qh = hq % p.g;
  grid_dependency_wait();
  grid_launch_dependents();  // the next call's CTAs may come; they wait for this kernel's end
  const int total = p.prefix[p.B], before = p.prefix[b], n = p.prefix[b + 1] - before;
  __nv_bfloat16* out = p.out + (static_cast<int64_t>(b) * p.Hq + hq) * D + d0;
  if (n == 0) {
    for (int d = threadIdx.x; d < W; d += NW * 32) out[d] = __float2bfloat16(0.f);
    return;
  }
  const int chunk = part_pages(total * p.Hkv, p.parts);
  const int x = before * p.Hkv + h * n;
  const StreamRows rows(x, n, total * p.Hkv, chunk);
  if (rows.first == rows.last) return;  // written where it was computed
  const float vs = p.v_scale[h];
  const int count = rows.count;
  const int64_t pair = static_cast<int64_t>(b) * p.Hkv + h;
  auto row = [&](int i) -> int64_t { return (rows.part(i) + pair) * p.g + qh; };
  float m = NEG_INF, l = 0.f, acc[V] = {};
  for (int i0 = warp; i0 < count; i0 += NW * kAtOnce) {
    float e[kAtOnce];
    Vec o[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + k * NW;
      const int64_t at = row(min(i, count - 1));
      e[k] = i < count ? p.lse_part[at] : NEG_INF;
      o[k] = reinterpret_cast<const Vec*>(p.o_part + at * D + d0)[lane];
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
  for (int d = threadIdx.x; d < W; d += NW * 32) {
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
    out[d] = __float2bfloat16(sum > 0.f || sum != sum ? y / sum * vs : 0.f);
  }
}

// Parts of a call's page stream, a warp each: one wave of CTAs, and no more than pairs
// of pages.
int fp4_parts(int B, int Hkv, int max_blocks) {
  const int64_t most = (static_cast<int64_t>(B) * Hkv * max_blocks + kMinPart - 1) / kMinPart;
  return static_cast<int>(std::min<int64_t>(static_cast<int64_t>(kCtasPerSm) * sm_count() * kWarps, most));
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
  static std::atomic<uint64_t> configured{0};  // devices whose attribute is set
  int dev = 0;
  cudaGetDevice(&dev);
  if (!(configured.load() >> (dev & 63) & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem);
    if (e != cudaSuccess) return cuda_status(e, "paged_decode_fp4: set shared memory size");
    configured.fetch_or(uint64_t(1) << (dev & 63));
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.parts + kWarps - 1) / kWarps);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = F::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return cuda_status(e, "paged_decode_fp4 launch");
  cfg.dynamicSmemBytes = 0;
  const unsigned rows = static_cast<unsigned>(p.B) * p.Hq;
  // Few rows have many pieces (about four of which are one row of partials): more warps, 32 dims
  // to a CTA.  By the mean over the rows.  128K, us with 32, 8, 2 warps: one KV head 19.9, 23.6, 36.8,
  // two 22.1, 23.0, 31.5, eight 39.4, 38.5, 42.3; 16 x 4,000 tokens 57, 26.8, 25.9, 64 x 500 to
  // 1,000 149, 30.8, 24.2.
  const int64_t pieces = p.parts / (static_cast<int64_t>(p.B) * p.Hkv);
  if (pieces >= 512) {
    cfg.gridDim = dim3(rows, D / 32);
    cfg.blockDim = dim3(32 * 32);
    e = cudaLaunchKernelEx(&cfg, decode_fp4_combine_kernel<D, 32, 32>, p);
  } else if (pieces >= 8) {
    cfg.gridDim = dim3(rows);
    cfg.blockDim = dim3(8 * 32);
    e = cudaLaunchKernelEx(&cfg, decode_fp4_combine_kernel<D, D, 8>, p);
  } else {
    cfg.gridDim = dim3(rows);
    cfg.blockDim = dim3(2 * 32);
    e = cudaLaunchKernelEx(&cfg, decode_fp4_combine_kernel<D, D, 2>, p);
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
      static_cast<double>(B) * Hkv * max_blocks > 0x7F000000)
    return fail(KVQ_ERR_UNSUPPORTED, "paged_decode_fp4: problem too large");
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !out || !workspace)
    return fail(KVQ_ERR_INVALID_ARG, "paged_decode_fp4: null pointer");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(workspace, 16) || !aligned(out, 4) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return fail(KVQ_ERR_INVALID_ARG, "paged_decode_fp4: misaligned pointer");
  const size_t need = kvq_decode_fp4_workspace_size(B, Hq, Hkv, D, P, max_blocks);
  if (workspace_bytes < need)
    return fail(KVQ_ERR_INVALID_ARG, "paged_decode_fp4: workspace %zu bytes < %zu needed", workspace_bytes, need);
  const PageStrides ps = page_strides(k_cache, v_cache, k_page_bytes(kFP4, D), v_page_bytes(kFP4, D));
  if (static_cast<double>(num_blocks) * Hkv * ps.k >= 64.0 * 0xffffffffu)  // places are 32-bit, in 64-byte units
    return fail(KVQ_ERR_UNSUPPORTED, "paged_decode_fp4: cache larger than 256 GiB");
  const int64_t rows = fp4_rows(B, Hq, Hkv, max_blocks);
  Fp4Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.str = ps.k;  // K and V pages are of one size: ps.v is the same
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
  p.parts = fp4_parts(B, Hkv, max_blocks);
  p.num_blocks = num_blocks;
  p.sm_scale = sm_scale;
  p.window = window;
  p.dev_status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return D == 128 ? launch_fp4<128>(p, s) : launch_fp4<64>(p, s);
}
