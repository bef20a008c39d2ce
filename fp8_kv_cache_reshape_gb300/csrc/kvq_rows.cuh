// What the kernels that move tokens between rows and the paged cache share:
// eight dims of a token per lane, their quantization and the page formats
// (include/kvq.h).
#pragma once

#include <cuda_fp4.h>

#include "kvq_device.cuh"
#include "kvq_page_plan.h"

namespace kvq {

static_assert(kPlanPage == kPage, "one page size");

// Heads a CTA walks: as many, in halves from `most`, as leave `ctas` CTAs.
inline int heads_per_cta(int heads, int tiles, int most, int ctas) {
  int n = most;
  while (n > 1 && static_cast<int64_t>(tiles) * ((heads + n - 1) / n) < ctas) n /= 2;
  return n;
}

// The formats of a cache, one kernel instantiation each.
enum CacheFormat { kRowsOnly, kE4M3, kE5M2, kBF16, kFP4, kE4M3Token, kE5M2Token };

template <int FMT>
struct Format {
  static constexpr bool kFp8 = FMT == kE4M3 || FMT == kE5M2 || FMT == kE4M3Token || FMT == kE5M2Token;
  static constexpr bool kE5 = FMT == kE5M2 || FMT == kE5M2Token;
  static constexpr bool kToken = FMT == kE4M3Token || FMT == kE5M2Token;
  static constexpr bool kHeadScale = FMT == kE4M3 || FMT == kE5M2 || FMT == kFP4;
  static constexpr float kMax = kE5 ? 57344.f : 448.f;
};

// Bytes of a K page, and of a V page with its scale tail.
__host__ __device__ constexpr int64_t k_page_bytes(int fmt, int D) {
  return fmt == kFP4 ? kPage * (D / 2 + D / 16) : static_cast<int64_t>(kPage) * D * (fmt == kBF16 ? 2 : 1);
}
__host__ __device__ constexpr int64_t v_page_bytes(int fmt, int D) {
  return k_page_bytes(fmt, D) + (fmt == kE4M3Token || fmt == kE5M2Token ? kScaleTailBytes : 0);
}

// Byte of dims 2j and 2j + 1 of token t in an FP4 V page: the operand order of
// the decode's P.V (decode_fp4.cu).
KVQ_DEVINL int fp4_v_offset(int t, int j) {
  return (j >> 5) * 512 + (j & 7) * 64 + ((t & 7) >> 1) * 16 + ((j >> 3) & 3) * 4 + (t >> 3) * 2 + (t & 1);
}
// E4M3 scale of block i of token t, from the end of the page's codes.
KVQ_DEVINL int fp4_v_scale_offset(int t, int i) {
  return (i >> 2) * 64 + ((t & 7) >> 1) * 16 + (i & 3) * 4 + (t >> 3) * 2 + (t & 1);
}

// Eight dims as four pairs of neighbours, for the two-wide float32 instructions.
KVQ_DEVINL void unpack8_bf16(const uint4& a, float2 (&x)[4]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
KVQ_DEVINL uint4 pack8_bf16(const float2 (&x)[4]) {
  return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                    pack_bf16x2(x[3].x, x[3].y));
}
// A divisor of quotients that are about to be rounded to few bits.  The code of
// fl32(x / s) is that of x * lo and of x * hi where those two agree, for lo and hi
// that enclose 1 / s: rounding is monotone.  Two products per value instead of a
// division; where they disagree (x / s within 2^-20 of a midpoint between codes, one
// value in 10^5 unless the scale is a ratio of small numbers) the eight values
// are divided.  A power of two needs no enclosure: x * (1 / s) is x / s.  4,096
// tokens with 32 query heads quantized and 8 KV heads of 128 into an E4M3 cache:
// 39.6 us with divisions, 28.6 so.
struct Divisor {
  float s, lo, hi;
  KVQ_DEVINL Divisor(float divisor, float2 bounds) : s(divisor), lo(bounds.x), hi(bounds.y) {}
  // rcp.approx is off by at most 2^-23, lo and hi by 2^-24 more each and each
  // product by 2^-24: within 2^-22, so 2^-21 to either side encloses
  KVQ_DEVINL explicit Divisor(float divisor) : s(divisor) {
    const uint32_t u = __float_as_uint(s);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    const bool exact = (u & 0x7FFFFFu) == 0;
    if (exact) r = __uint_as_float(0x7F000000u - u);  // 2^-e of 2^e
    lo = exact ? r : r * (1.f - 0x1p-21f);
    hi = exact ? r : r * (1.f + 0x1p-21f);
    if (u - 0x04000000u >= 0x7A000000u - 0x04000000u) {
      // not 2^-119 <= s < 2^117: no normal 1 / s.  Products whose codes differ (0 and
      // NaN of 0, 0 and infinity of others), but for NaN and, in E2M1, where NaN is 6, for
      // infinity, whose quotients have those codes too
      lo = 0.f;
      hi = __uint_as_float(0x7F800000u);
    }
  }
};
// Four values' FP8 codes, eight values' E2M1 codes, nearest even, saturating.
template <bool E5>
KVQ_DEVINL uint32_t fp8x4(float2 a, float2 b) {
  uint32_t w;
  if constexpr (E5)
    asm("{\n\t.reg .b16 u, v;\n\tcvt.rn.satfinite.e5m2x2.f32 u, %2, %1;\n\tcvt.rn.satfinite.e5m2x2.f32 v, %4, %3;\n\t"
        "mov.b32 %0, {u, v};\n\t}" : "=r"(w) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  else
    asm("{\n\t.reg .b16 u, v;\n\tcvt.rn.satfinite.e4m3x2.f32 u, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 v, %4, %3;\n\t"
        "mov.b32 %0, {u, v};\n\t}" : "=r"(w) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return w;
}
KVQ_DEVINL uint32_t e2m1x8(const float2 (&x)[4]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y));
  return w;
}
KVQ_DEVINL void scale8(const float2 (&x)[4], float f, float2 (&y)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = fmul2(x[i], make_float2(f, f));
}
KVQ_DEVINL void divide8(const float2 (&x)[4], float s, float2 (&y)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = make_float2(__fdiv_rn(x[i].x, s), __fdiv_rn(x[i].y, s));
}
// fp8(fl32(x / s)) of eight values.
template <bool E5>
KVQ_DEVINL uint2 quant8_fp8(const float2 (&x)[4], const Divisor& d) {
  float2 lo[4], hi[4];
  scale8(x, d.lo, lo);
  scale8(x, d.hi, hi);
  uint2 w = make_uint2(fp8x4<E5>(lo[0], lo[1]), fp8x4<E5>(lo[2], lo[3]));
  if (w.x != fp8x4<E5>(hi[0], hi[1]) || w.y != fp8x4<E5>(hi[2], hi[3])) {
    divide8(x, d.s, lo);
    w = make_uint2(fp8x4<E5>(lo[0], lo[1]), fp8x4<E5>(lo[2], lo[3]));
  }
  return w;
}
// e2m1(fl32(x / s)) of eight values.
KVQ_DEVINL uint32_t quant8_e2m1(const float2 (&x)[4], const Divisor& d) {
  float2 lo[4], hi[4];
  scale8(x, d.lo, lo);
  scale8(x, d.hi, hi);
  uint32_t w = e2m1x8(lo);
  if (w != e2m1x8(hi)) {
    divide8(x, d.s, lo);
    w = e2m1x8(lo);
  }
  return w;
}
KVQ_DEVINL float e4m3_value(uint8_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}
// e4m3(fl32(x / s)) of one value.
KVQ_DEVINL uint32_t quant1_e4m3(float x, const Divisor& d) {
  const uint32_t w = __nv_cvt_float2_to_fp8x2(make_float2(x * d.lo, x * d.hi), __NV_SATFINITE, __NV_E4M3);
  const uint32_t lo = w & 0xFF;
  return lo == w >> 8 ? lo : f32_to_e4m3(__fdiv_rn(x, d.s));
}
KVQ_DEVINL float amax8(const float2 (&x)[4]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) a = fmax3(a, fabsf(x[i].x), fabsf(x[i].y));
  return a;
}
// The same, but NaN where one of them is: E2M1 has no code for it, the block's scale has.
KVQ_DEVINL float amax8_nan(const float2 (&x)[4]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(fabsf(x[i].x)), "f"(fabsf(x[i].y)));
  return a;
}
// The E4M3 scale of a block of 16 dims, of which two neighbouring lanes hold
// eight each, and their E2M1 codes.  s: the head's scale, six: Divisor(fl32(6 s)).
KVQ_DEVINL uint32_t quant8_fp4(const float2 (&x)[4], float s, const Divisor& six, uint8_t& block_scale) {
  float a = amax8_nan(x);
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(__shfl_xor_sync(0xffffffffu, a, 1)));
  block_scale = static_cast<uint8_t>(quant1_e4m3(a, six));
  const float step = __fmul_rn(e4m3_value(block_scale), s);
  if (!(step > 0.f)) return 0;
  return quant8_e2m1(x, Divisor(step));
}

// 4 x 4 bytes transposed: byte j of word i to byte i of word j.
KVQ_DEVINL void transpose4(const uint32_t (&w)[4], uint32_t (&o)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
  o[0] = __byte_perm(a, b, 0x5410);
  o[1] = __byte_perm(a, b, 0x7632);
  o[2] = __byte_perm(c, d, 0x5410);
  o[3] = __byte_perm(c, d, 0x7632);
}

// The tokens of a tile.  Plain tiles are 16 tokens in order.  Aligned ones
// follow the pages: the tokens whose page, if its tokens lie in order, began with
// one of the 16 tokens from 16 (tile - 1) on.  A run of tokens in order through
// whole pages then has each page in one tile, wherever in a page it starts; any
// other tokens fall to some tile too, each to one, at most 31 to a tile.  A page
// whose tile begins with other tokens is not taken as a whole.
struct TileTokens {
  int token[32];
  int64_t slot[32];
  int n;
  bool page;  // tokens 0 .. 15 fill one page in order (16 on never do: they are 15 at most)
};
// By warp 0, before a barrier of the CTA.
KVQ_DEVINL void find_tokens(TileTokens& s, const int64_t* slots, int T, int64_t num_slots, int tile, bool aligned, int* dev_status) {
  const int lane = threadIdx.x & 31;
  const int64_t token = static_cast<int64_t>(tile - (aligned ? 1 : 0)) * kPage + lane;
  int64_t slot = -1;
  if (token >= 0 && token < T && (aligned || lane < kPage)) slot = slots[token];
  if (slot >= num_slots) {
    set_status(dev_status, KVQ_DEV_BAD_SLOT);
    slot = -1;
  }
  bool mine = slot >= 0;
  if (aligned && mine) mine = tile_takes(lane, slot);
  const unsigned have = __ballot_sync(0xffffffffu, mine);
  if (mine) {
    const int at = __popc(have & ((1u << lane) - 1));
    s.token[at] = static_cast<int>(token);
    s.slot[at] = slot;
  }
  __syncwarp();
  const int n = __popc(have);
  const int64_t first = n ? s.slot[0] : 0;
  const bool run = lane < n && first % kPage == 0 && s.slot[lane] == first + lane;
  const unsigned runs = __ballot_sync(0xffffffffu, run);
  if (lane == 0) {
    s.n = n;
    s.page = (runs & 0xFFFFu) == 0xFFFFu;
  }
}

}  // namespace kvq
