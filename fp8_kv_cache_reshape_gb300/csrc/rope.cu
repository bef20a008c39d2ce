// kvq_qk_norm_rope, kvq_rope_and_cache, and the 4-bit form of
// kvq_reshape_and_cache: one kernel that takes tokens' q, k and v rows, norms
// and turns q and k, and writes rows or cache pages.
//
// Mathematics.  y = x * rsqrt(mean x^2 + eps) * w per head, then each pair is
// turned by a = position * inv_freq.  Norm weight and rotation fold into two
// factors per dim that do not depend on the head: with p(d) the pair's other
// dim, out_d = r x_d A_d + r x_p(d) B_d, A_d = w_d cos a, B_d = -+ w_p(d) sin a,
// r the head's norm factor (first, so that no product with a weight leaves float32
// whose result does not).  A lane holds eight dims of one token and walks
// heads, so angles, sines and weights are paid once per token and CTA.
//
// The angle is taken in turns in 64-bit fixed point: inv_freq / 2 pi as a
// 64-bit fraction times the position, whose overflow is the reduction by whole
// turns.  No float64 (two operations a clock per SM here) and no position too
// far for float32.
//
// Bound: memory in principle (every row is read once and written once).  16,383 tokens,
// 32 + 8 heads of 128, normed and turned along three axes: 58.5 us, 5.7 TB/s of the
// measured copy rate of 6.8, the issue slots 71% full.  4,096 tokens into an E4M3 cache,
// queries quantized: 19.5 us, 3.9 TB/s (normed: 24), where no unit is full (issue slots 65%, ALU pipe,
// which converts and selects bytes, 51%): a row's chain of dependent steps, with five of six
// warps a scheduler there on average, is what it waits for.  A step of 64 tokens: 5.5 us, latency.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "kvq_host.h"
#include "kvq_rows.cuh"

namespace kvq {

namespace {

// floor(2^66 / 2 pi)
constexpr uint64_t kInvTwoPi = 0xA2F9836E4E441529ull;

// inv_freq / 2 pi as a fraction of a turn in units of 2^-64 (whole turns drop out).
KVQ_DEVINL uint64_t turns_per_position(float inv_freq) {
  const uint32_t u = __float_as_uint(inv_freq);
  const int e = static_cast<int>((u >> 23) & 0xFF);
  const uint32_t m = e ? (u & 0x7FFFFFu) | 0x800000u : u & 0x7FFFFFu;
  // inv_freq = m 2^(e - 150) (e = 1 for subnormals), so the fraction is
  // (m kInvTwoPi / 2^24) 2^(e - 128)
  const uint64_t f = (static_cast<uint64_t>(m) * static_cast<uint32_t>(kInvTwoPi >> 32) << 8) +
                     (static_cast<uint64_t>(m) * static_cast<uint32_t>(kInvTwoPi) >> 24);
  const int shift = (e ? e : 1) - 128;
  const uint64_t x = shift <= -64 ? 0 : shift < 0 ? f >> -shift : shift < 64 ? f << shift : 0;
  return u >> 31 ? 0 - x : x;
}

// Sine and cosine of a fraction of a turn: to the nearest quarter, then the
// Taylor series of the rest, y up to pi / 4 either way.  The first terms left
// out are y^11 / 11! < 2^-29 and y^12 / 12! < 2^-32; y is rounded three times, 2^-22 of it,
// and cut to 55 bits of a turn, of which the lower 23 become a float32 as the
// mantissa of 2^23 + x.
KVQ_DEVINL void sincos_turns(uint64_t turns, float& s, float& c) {
  const uint32_t t = static_cast<uint32_t>(turns >> 32);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const int rest = static_cast<int>(t - (quarter << 30));  // within an eighth of a turn
  const float low = __uint_as_float(0x4B000000u | static_cast<uint32_t>(turns) >> 9) - 0x1p23f;
  const float turn = 6.283185307f;
  const float y = fmaf(static_cast<float>(rest), turn * 0x1p-32f, low * (turn * 0x1p-55f)), z = y * y;
  float s0 = fmaf(z, 1.f / 362880, -1.f / 5040), c0 = fmaf(z, -1.f / 3628800, 1.f / 40320);
  s0 = fmaf(z, s0, 1.f / 120);
  s0 = fmaf(z, s0, -1.f / 6);
  s0 = fmaf(y * z, s0, y);
  c0 = fmaf(z, c0, -1.f / 720);
  c0 = fmaf(z, c0, 1.f / 24);
  c0 = fmaf(z, c0, -0.5f);
  c0 = fmaf(z, c0, 1.f);
  s = quarter & 1 ? c0 : s0;
  c = quarter & 1 ? s0 : c0;
  if (quarter & 2) s = -s;
  if ((quarter + 1) & 2) c = -c;
}

struct TokenParams {
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const __nv_bfloat16 *q_weight, *k_weight;
  float eps;
  kvq_rotary_t rotary;  // rot_dim 0: no rotation
  const int64_t* slots;
  uint8_t *k_cache, *v_cache;
  int64_t k_str, v_str;  // bytes between pages
  const float *k_scale, *v_scale;
  int64_t num_slots;
  __nv_bfloat16 *q_out, *k_out;
  int64_t q_out_stride, k_out_stride;
  uint8_t* q8;
  const float* q_scale;
  int T, Hq, Hkv;
  // CTAs: kv_tiles x kv_chunks of k's (and v's) heads, then tiles x chunks of q's
  int kv_tiles, tiles, kv_chunk, q_chunk;
  unsigned kv_ctas;
  bool aligned;
  int* dev_status;
};

// The factors of a lane's eight dims (see the top of the file).
struct Turn {
  float2 a[4], b[4];
  int from;         // lane that holds the pairs' other dims (this one, interleaved)
  uint32_t px, py;  // which bytes of its words they are, as float32 (0x4444: none, zero)
};

template <int D>
KVQ_DEVINL Turn make_turn(const TokenParams& p, const __nv_bfloat16* weight, int token, int lane) {
  constexpr int LPT = D / 8;
  const int j = lane % LPT;
  Turn t;
  const int rot = p.rotary.rot_dim, half = rot / 2;
  const bool turned = 8 * j < rot;
  int partner = j;
  if (turned && !p.rotary.interleaved) partner = 8 * j < half ? j + half / 8 : j - half / 8;
  t.from = lane - j + partner;
  t.px = !turned ? 0x4444 : p.rotary.interleaved ? 0x3244 : 0x1044;
  t.py = !turned ? 0x4444 : p.rotary.interleaved ? 0x1044 : 0x3244;
  float2 w[4], wp[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = wp[i] = make_float2(1.f, 1.f);
  if (weight) {
    unpack8_bf16(__ldg(reinterpret_cast<const uint4*>(weight) + j), w);
    unpack8_bf16(__ldg(reinterpret_cast<const uint4*>(weight) + partner), wp);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t.a[i] = w[i];
    t.b[i] = make_float2(-0.f, -0.f);  // x * 1 + 0 * -0 is x, a negative zero too
  }
  auto angle = [&](int pair, float& s, float& c) {
    int axis = p.rotary.pair_axis ? __ldg(p.rotary.pair_axis + pair) : 0;
    if (static_cast<unsigned>(axis) >= static_cast<unsigned>(p.rotary.num_axes)) {
      set_status(p.dev_status, KVQ_DEV_BAD_AXIS);
      axis = 0;
    }
    const uint64_t pos = static_cast<uint64_t>(__ldg(p.rotary.positions + axis * p.rotary.positions_stride + token));
    sincos_turns(pos * turns_per_position(__ldg(p.rotary.inv_freq + pair)), s, c);
    s *= p.rotary.scale;
    c *= p.rotary.scale;
  };
  if (p.rotary.interleaved) {
    if (!turned) return t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float s, c;
      angle(4 * j + i, s, c);
      t.a[i] = make_float2(c * w[i].x, c * w[i].y);
      t.b[i] = make_float2(-s * w[i].y, s * w[i].x);
    }
  } else {
    // this lane and its partner turn the same eight pairs: four angles each
    const bool low = 8 * j < half;
    float2 sc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sc[i] = make_float2(0.f, 1.f);
      if (turned) angle(low ? 8 * j + i : 8 * j - half + 4 + i, sc[i].x, sc[i].y);
    }
    const float sign = low ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // dims 2i, 2i + 1: the lower lane has the angles of the first four
      float2 u[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 mine = sc[(2 * i + e) & 3];
        const float so = __shfl_sync(0xffffffffu, mine.x, t.from), co = __shfl_sync(0xffffffffu, mine.y, t.from);
        u[e] = low == (i < 2) ? mine : make_float2(so, co);
      }
      if (!turned) continue;
      t.a[i] = make_float2(w[i].x * u[0].y, w[i].y * u[1].y);
      t.b[i] = make_float2(wp[i].x * u[0].x * sign, wp[i].y * u[1].x * sign);
    }
  }
  return t;
}

// The norm's factor of a row whose squares float32 does not hold, x * y * z: the first two
// are a power of two that brings the row's maximum to [1, 2), but eps with it no further than
// 2^100, where it outweighs the rest; the third is the factor of that row.  Every lane of the
// warp takes part.  Not inlined: its code between the others' costs 2 to 4%.
template <int D>
__device__ __noinline__ float3 norm_factors(float eps, uint4 raw) {
  constexpr int LPT = D / 8;
  float2 x[4];
  unpack8_bf16(raw, x);
  float top = amax8(x);
#pragma unroll
  for (int off = 1; off < LPT; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  int k = 127 - static_cast<int>(__float_as_uint(top) >> 23);
  if (eps > 0.f) k = min(k, (227 - static_cast<int>(__float_as_uint(eps) >> 23)) >> 1);
  // 2^k in two steps: -128 to 127 is beyond one float32 factor
  const float f = __uint_as_float(static_cast<uint32_t>(127 + (k >> 1)) << 23);
  const float g = __uint_as_float(static_cast<uint32_t>(127 + k - (k >> 1)) << 23);
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = fmul2(fmul2(x[i], make_float2(f, f)), make_float2(g, g));
    sum = ffma2(x[i], x[i], sum);
  }
  float all = sum.x + sum.y;
#pragma unroll
  for (int off = 1; off < LPT; off <<= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
  return make_float3(f, g, rsqrtf(fmaf(all, 1.f / D, eps * f * f * g * g)));
}

// Norm and rotation of a lane's eight dims, `other` those of lane t.from; every
// lane of the warp takes part.
template <int D>
KVQ_DEVINL void turn_row(const Turn& t, bool norm, float eps, const uint4& raw, const uint4& other, float2 (&o)[4]) {
  constexpr int LPT = D / 8;
  const uint32_t w[4] = {other.x, other.y, other.z, other.w};
  float2 x[4], y[4];
  unpack8_bf16(raw, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = w[i];
    y[i] = make_float2(__uint_as_float(__byte_perm(u, 0, t.px)), __uint_as_float(__byte_perm(u, 0, t.py)));
  }
  if (norm) {
    float2 sum = fmul2(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) sum = ffma2(x[i], x[i], sum);
    float all = sum.x + sum.y;
#pragma unroll
    for (int off = 1; off < LPT; off <<= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
    const float mean = fmaf(all, 1.f / D, eps);
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(mean));
    // Squares that float32 does not hold: of a sum beyond it, or below 2^-149 beside a mean
    // that they would be part of.  Only such rows take the other factor; a warp without any
    // pays for a comparison and a vote.
    const bool plain = __float_as_uint(mean) - 0x13000000u < 0x7F800000u - 0x13000000u;  // 2^-89 <= mean < infinity
    if (__any_sync(0xffffffffu, !plain)) {
      const float3 f = norm_factors<D>(eps, raw);
      if (!plain) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = fmul2(fmul2(x[i], make_float2(f.x, f.x)), make_float2(f.y, f.y));
          y[i] = fmul2(fmul2(y[i], make_float2(f.x, f.x)), make_float2(f.y, f.y));
        }
        r = f.z;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = fmul2(x[i], make_float2(r, r));
      y[i] = fmul2(y[i], make_float2(r, r));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = ffma2(x[i], t.a[i], fmul2(y[i], t.b[i]));
}

// Rows of a warp's tokens on their way through shared memory: a stage is the 16
// bytes of each lane, of one row (or of a k and a v row).  The copies of all stages but one
// are in flight, which costs no registers, and a pair's other dims are a second read
// instead of four shuffles (at the step that brought it: 4,096 tokens into an E4M3 cache
// 22.8 -> 20.3 us, 16,383 tokens' rows 59.8 -> 58).
template <int D>
struct Ring {
  static constexpr int kBytes = D == 256 ? 2048 : 4096;  // of a warp (of 16 at D = 256)
  static constexpr int kRow = 512;
  static constexpr int kRows = kBytes / kRow, kPairs = kRows / 2;  // stages
};

// Rows in, rows (or E4M3 codes) out: 16 tokens, heads h0 .. h1 - 1.
template <int D>
KVQ_DEVINL void turn_rows(const TokenParams& p, uint32_t ring, bool is_q, int tile, int h0, int h1) {
  constexpr int LPT = D / 8;
  constexpr int kStages = Ring<D>::kRows, kStageB = Ring<D>::kRow;
  const int lane = threadIdx.x & 31, j = threadIdx.x % LPT;
  const int token = tile * kPage + threadIdx.x / LPT;
  const bool live = token < p.T;
  const int row = live ? token : p.T - 1;
  const uint8_t* src = reinterpret_cast<const uint8_t*>((is_q ? p.q : p.k) + row * (is_q ? p.q_stride : p.k_stride) + h0 * D + 8 * j);
  const int n = h1 - h0;
  auto issue = [&](int i) {
    if (i < n) copy16(ring + i % kStages * kStageB + lane * 16, src + i * (D * 2));
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  const __nv_bfloat16* weight = is_q ? p.q_weight : p.k_weight;
  const Turn turn = make_turn<D>(p, weight, row, lane);
  __nv_bfloat16* dst = is_q ? p.q_out : p.k_out;
  if (dst) dst += row * (is_q ? p.q_out_stride : p.k_out_stride) + h0 * D + 8 * j;
  uint8_t* codes = is_q && p.q8 ? p.q8 + (static_cast<int64_t>(row) * p.Hq + h0) * D + 8 * j : nullptr;
  const Divisor s(codes ? __ldg(p.q_scale) : 1.f);
  auto walk = [&](auto normed) {  // a loop each: without norms 3% less
    for (int i = 0; i < n; ++i) {
      copy_wait<kStages - 2>();
      __syncwarp();  // the other lanes' copies too, and they are done with the stage before
      issue(i + kStages - 1);
      const uint32_t at = ring + i % kStages * kStageB;
      float2 o[4];
      turn_row<D>(turn, normed.value, p.eps, lds128(at + lane * 16), lds128(at + turn.from * 16), o);
      if (!live) continue;
      if (dst) *reinterpret_cast<uint4*>(dst + i * D) = pack8_bf16(o);
      if (codes) *reinterpret_cast<uint2*>(codes + i * D) = quant8_fp8<false>(o, s);
    }
  };
  if (weight)
    walk(std::true_type{});
  else
    walk(std::false_type{});
}

// Bytes between tokens of a V page in shared memory, before its transposition:
// the four token rows that a page's word takes from fall into different banks.
template <int D, int FMT>
constexpr int kVStride = (FMT == kFP4 ? D / 2 : FMT == kBF16 ? 2 * D : D) + 16;

// A V page from its 16 token rows in shared memory.
template <int D, int FMT>
KVQ_DEVINL void write_v_page(const uint8_t* rows, uint8_t* vp) {
  constexpr int S = kVStride<D, FMT>;
  const int x = threadIdx.x;
  if constexpr (FMT == kBF16) {
    if (x >= D) return;
    const int half = x & 1, d = x & ~1;  // dims d, d + 1 of eight tokens
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint32_t*>(rows + (8 * half + i) * S + 2 * d);
    uint4 lo, hi;
    lo.x = __byte_perm(w[0], w[1], 0x5410);
    lo.y = __byte_perm(w[2], w[3], 0x5410);
    lo.z = __byte_perm(w[4], w[5], 0x5410);
    lo.w = __byte_perm(w[6], w[7], 0x5410);
    hi.x = __byte_perm(w[0], w[1], 0x7632);
    hi.y = __byte_perm(w[2], w[3], 0x7632);
    hi.z = __byte_perm(w[4], w[5], 0x7632);
    hi.w = __byte_perm(w[6], w[7], 0x7632);
    *reinterpret_cast<uint4*>(vp + bf16_v_offset(d, 8 * half)) = lo;
    *reinterpret_cast<uint4*>(vp + bf16_v_offset(d + 1, 8 * half)) = hi;
  } else {
    // a word is one byte of tokens 2c, 2c + 1, 2c + 8, 2c + 9, in the FP8 and the FP4 page
    int c, col, at, step;  // four columns from `col` on, whose words lie `step` apart from `at` on
    if constexpr (FMT == kFP4) {
      if (x >= D / 2) return;
      const int b = x & 3, half = (x >> 4) & 1, h = x >> 5;
      c = (x >> 2) & 3;
      col = 32 * h + 8 * b + 4 * half;
      at = h * 512 + half * 256 + c * 16 + b * 4;
      step = 64;
    } else {
      if (x >= D) return;
      c = x & 3;
      col = x & ~3;
      at = col * kPage + c * 4;
      step = kPage;
    }
    uint32_t w[4], o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(rows + (2 * c + (i & 1) + 8 * (i >> 1)) * S + col);
    transpose4(w, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(vp + at + i * step) = o[i];
  }
}

constexpr int kMaxKvChunk = 8;  // heads of a cache CTA

// k and v into the cache: a tile's tokens, heads h0 .. h1 - 1.
// TURN: k is normed or turned.
template <int D, int FMT, bool TURN>
KVQ_DEVINL void cache_rows(const TokenParams& p, uint32_t ring, int tile, int h0, int h1) {
  using F = Format<FMT>;
  constexpr int LPT = D / 8;
  constexpr int kStages = Ring<D>::kPairs, kStageB = Ring<D>::kRow;
  __shared__ TileTokens tt;
  __shared__ __align__(16) uint8_t rows[2][kPage * kVStride<D, FMT>];
  // lo and hi of the divisors of each head's k and v, once instead of in every lane
  // for every row (32,768 tokens into E4M3: 49.6 us without, 46.7 so)
  __shared__ float4 bounds[kMaxKvChunk];
  const int lane = threadIdx.x & 31, t = threadIdx.x / LPT, j = threadIdx.x % LPT;
  if (threadIdx.x < 32) find_tokens(tt, p.slots, p.T, p.num_slots, tile, p.aligned, p.dev_status);
  if constexpr (F::kHeadScale) {
    const int h = h0 + static_cast<int>(threadIdx.x) - 32;
    if (h >= h0 && h < h1) {
      constexpr float f = FMT == kFP4 ? 6.f : 1.f;
      const Divisor kd(__fmul_rn(f, __ldg(p.k_scale + h))), vd(__fmul_rn(f, __ldg(p.v_scale + h)));
      bounds[h - h0] = make_float4(kd.lo, kd.hi, vd.lo, vd.hi);
    }
  }
  __syncthreads();
  const int n = tt.n;
  for (int r = 0; r < n; r += kPage) {
    const bool valid = r + t < n, page_run = r == 0 && tt.page;
    const int row = tt.token[valid ? r + t : r];
    const int64_t slot = tt.slot[valid ? r + t : r];
    const int off = static_cast<int>(slot % kPage);
    const uint8_t* ksrc = reinterpret_cast<const uint8_t*>(p.k + row * p.k_stride + h0 * D + 8 * j);
    const uint8_t* vsrc = reinterpret_cast<const uint8_t*>(p.v + row * p.v_stride + h0 * D + 8 * j);
    auto issue = [&](int i) {
      if (i < h1 - h0) {
        const uint32_t at = ring + i % kStages * (2 * kStageB) + lane * 16;
        copy16(at, ksrc + i * (D * 2));
        copy16(at + kStageB, vsrc + i * (D * 2));
      }
      copy_commit();
    };
    __syncwarp();  // done with the stages of the 16 tokens before
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);
    const int64_t page = slot / kPage * p.Hkv + h0;
    uint8_t* kp = p.k_cache + page * p.k_str;
    uint8_t* vp = p.v_cache + page * p.v_str;
    Turn turn;
    if constexpr (TURN) turn = make_turn<D>(p, p.k_weight, row, lane);
    for (int h = h0; h < h1; ++h) {
      uint8_t* buf = rows[(h - h0) & 1];
      copy_wait<kStages - 2>();
      __syncwarp();  // the other lanes' copies too, and they are done with the stage before
      issue(h - h0 + kStages - 1);
      const uint32_t at = ring + (h - h0) % kStages * (2 * kStageB);
      const uint4 vraw = lds128(at + kStageB + lane * 16);
      float2 ko[4], vo[4];
      if constexpr (TURN)
        turn_row<D>(turn, p.k_weight != nullptr, p.eps, lds128(at + lane * 16), lds128(at + turn.from * 16), ko);
      else
        unpack8_bf16(lds128(at + lane * 16), ko);
      unpack8_bf16(vraw, vo);
      if constexpr (F::kFp8) {
        uint2 kq, vq;
        if constexpr (F::kToken) {
          float ka = amax8(ko), va = amax8(vo);
#pragma unroll
          for (int o = 1; o < LPT; o <<= 1) {
            ka = fmaxf(ka, __shfl_xor_sync(0xffffffffu, ka, o));
            va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, o));
          }
          const float ks = ka > 0.f ? __fdiv_rn(ka, F::kMax) : 1.f;  // an all-zero token keeps scale 1
          const float vs = va > 0.f ? __fdiv_rn(va, F::kMax) : 1.f;
          if (valid && j == 0) {
            float* tail = reinterpret_cast<float*>(vp + kPage * D);
            tail[off] = ks;
            tail[kPage + off] = vs;
          }
          kq = quant8_fp8<F::kE5>(ko, Divisor(ks));
          vq = quant8_fp8<F::kE5>(vo, Divisor(vs));
        } else {
          const float4 b = bounds[h - h0];
          kq = quant8_fp8<F::kE5>(ko, Divisor(__ldg(p.k_scale + h), make_float2(b.x, b.y)));
          vq = quant8_fp8<F::kE5>(vo, Divisor(__ldg(p.v_scale + h), make_float2(b.z, b.w)));
        }
        if (valid) {
          *reinterpret_cast<uint2*>(kp + fp8_k_offset(off, j >> 1, D) + (j & 1) * 8) = kq;
          if (page_run) {
            *reinterpret_cast<uint2*>(buf + off * kVStride<D, FMT> + 8 * j) = vq;
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              vp[(8 * j + i) * kPage + fp8_v_slot(off)] = static_cast<uint8_t>((i < 4 ? vq.x : vq.y) >> (8 * (i & 3)));
          }
        }
      } else if constexpr (FMT == kBF16) {
        if (valid) {
          *reinterpret_cast<uint4*>(kp + k_chunk_offset(off, j, 2 * D)) = pack8_bf16(ko);
          if (page_run) {
            *reinterpret_cast<uint4*>(buf + off * kVStride<D, FMT> + 16 * j) = vraw;
          } else {
            const uint32_t w[4] = {vraw.x, vraw.y, vraw.z, vraw.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint16_t*>(vp + bf16_v_offset(8 * j + i, off)) =
                  static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
          }
        }
      } else {
        uint8_t ks, vs;
        const float sk = __ldg(p.k_scale + h), sv = __ldg(p.v_scale + h);
        const float4 b = bounds[h - h0];
        const uint32_t kw = quant8_fp4(ko, sk, Divisor(__fmul_rn(6.f, sk), make_float2(b.x, b.y)), ks);
        const uint32_t vw = quant8_fp4(vo, sv, Divisor(__fmul_rn(6.f, sv), make_float2(b.z, b.w)), vs);
        if (valid) {
          *reinterpret_cast<uint32_t*>(kp + off * (D / 2) + 4 * j) = kw;
          if (page_run) {
            *reinterpret_cast<uint32_t*>(buf + off * kVStride<D, FMT> + 4 * j) = vw;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) vp[fp4_v_offset(off, 4 * j + i)] = static_cast<uint8_t>(vw >> (8 * i));
          }
          if ((j & 1) == 0) {
            kp[kPage * D / 2 + off * (D / 16) + j / 2] = ks;
            vp[kPage * D / 2 + fp4_v_scale_offset(off, j / 2)] = vs;
          }
        }
      }
      if (page_run) {
        // two buffers: the next head's rows go to the other one, and the one after
        // comes behind the next barrier, which nobody passes before reading this one
        __syncthreads();
        write_v_page<D, FMT>(buf, vp);
      }
      kp += p.k_str;
      vp += p.v_str;
    }
  }
}

// Three CTAs of 256 threads an SM (80 registers) where there is a cache to write, four (64)
// for rows alone (16,000 tokens normed: 56.9 us, with three 58.0; 8,000 of head dim 256: 35.7 and 45.1).
template <int D, int FMT, bool TURN = true>
__global__ void __launch_bounds__(kPage * D / 8, (FMT == kRowsOnly ? 1024 : 768) / (2 * D)) token_kernel(const TokenParams p) {
  __shared__ __align__(16) uint8_t ring_mem[D / 16 * Ring<D>::kBytes];
  const uint32_t ring = smem_u32(ring_mem) + threadIdx.x / 32 * Ring<D>::kBytes;
  if (blockIdx.x >= p.kv_ctas) {
    const unsigned x = blockIdx.x - p.kv_ctas;
    const int h = static_cast<int>(x / p.tiles) * p.q_chunk;
    turn_rows<D>(p, ring, true, x % p.tiles, h, min(p.Hq, h + p.q_chunk));
  } else {
    const int h = static_cast<int>(blockIdx.x / p.kv_tiles) * p.kv_chunk, tile = blockIdx.x % p.kv_tiles;
    if constexpr (FMT == kRowsOnly)
      turn_rows<D>(p, ring, false, tile, h, min(p.Hkv, h + p.kv_chunk));
    else
      cache_rows<D, FMT, TURN>(p, ring, tile, h, min(p.Hkv, h + p.kv_chunk));
  }
}

// Heads to a CTA: angles and weights are paid once per CTA (16,383 tokens: 66.4 us
// with 8 query heads, 57.9 with 16, 58.5 with 32), but the SMs want filling: about a
// CTA of the cache's rows for each, and two of the queries' (4,096 tokens: 19.4 us;
// 21.2 with twice as many of the first, 20.2 and 20.8 with half and twice as many of the second;
// 1,777 tokens of head dim 64: 10.1 us, 12.6 and 11.7 with half and twice the first).
// Without queries as many of the cache's CTAs as run at once, three to an SM (3,500
// tokens, 4 bits: 7.9 us; 11.1 and 9.0 with half and twice as many).
// Aligned tiles pay from a few hundred tokens in order on (256 tokens of one
// prompt 6.4 us against 8.0, 1,024: 9.2 against 14.7) and cost steps of many sequences a
// little (256: 10.3 against 8.3, 1,024: 21.4 against 20.0).
template <int FMT, bool TURN = true>
kvq_status_t launch_tokens(TokenParams& p, int D, cudaStream_t s, const char* where) {
  p.tiles = (p.T - 1) / kPage + 1;
  p.aligned = FMT != kRowsOnly && p.T >= 256;
  p.kv_tiles = p.tiles + (p.aligned ? 1 : 0);
  p.kv_chunk = heads_per_cta(p.Hkv, p.kv_tiles, kMaxKvChunk, p.Hq ? 128 * sm_count() / D : 192 * sm_count() / D + 1);
  p.q_chunk = heads_per_cta(p.Hq, p.tiles, 32, 2 * sm_count());
  const int64_t kv_ctas = static_cast<int64_t>(p.kv_tiles) * ((p.Hkv + static_cast<int64_t>(p.kv_chunk) - 1) / p.kv_chunk);
  const int64_t ctas = kv_ctas + static_cast<int64_t>(p.tiles) * ((p.Hq + static_cast<int64_t>(p.q_chunk) - 1) / p.q_chunk);
  if (ctas > 0x7FFFFFFF) return fail(KVQ_ERR_UNSUPPORTED, "%s: problem too large", where);
  p.kv_ctas = static_cast<unsigned>(kv_ctas);
  const unsigned grid = static_cast<unsigned>(ctas);
  if (D == 64) {
    token_kernel<64, FMT, TURN><<<grid, 128, 0, s>>>(p);
  } else if (D == 128) {
    token_kernel<128, FMT, TURN><<<grid, 256, 0, s>>>(p);
  } else if constexpr (FMT == kRowsOnly || FMT == kE4M3 || FMT == kE5M2) {
    token_kernel<256, FMT><<<grid, 512, 0, s>>>(p);
  }
  return cuda_status(cudaGetLastError(), where);
}

bool rows_ok(const void* x, int64_t stride, int heads, int D) {
  return aligned(x, 16) && stride % 8 == 0 && stride >= static_cast<int64_t>(heads) * D;
}

// Rows in place go by one stride: with another, a token's output is one that is still to be read.
bool in_place_ok(const void* x, int64_t stride, const void* out, int64_t out_stride, int T) {
  return out != x || out_stride == stride || T <= 1;
}

// Checks of the norm and the rotation; fills them in.
kvq_status_t take_turn(TokenParams& p, const kvq_head_norm_t* norm, const kvq_rotary_t* rotary, int D, const char* where) {
  p.eps = 0.f;
  p.q_weight = p.k_weight = nullptr;
  if (norm) {
    if (!(norm->eps >= 0.f) || !(norm->eps <= FLT_MAX)) return fail(KVQ_ERR_INVALID_ARG, "%s: bad eps", where);
    if (!aligned(norm->q_weight, 16) || !aligned(norm->k_weight, 16))
      return fail(KVQ_ERR_INVALID_ARG, "%s: norm weights must be 16-byte aligned", where);
    p.eps = norm->eps;
    p.q_weight = static_cast<const __nv_bfloat16*>(norm->q_weight);
    p.k_weight = static_cast<const __nv_bfloat16*>(norm->k_weight);
  }
  p.rotary = kvq_rotary_t{};
  if (rotary) {
    if (rotary->rot_dim < 16 || rotary->rot_dim > D || rotary->rot_dim % 16 != 0)
      return fail(KVQ_ERR_UNSUPPORTED, "%s: rot_dim %d (a multiple of 16 up to the head dim)", where, rotary->rot_dim);
    if (rotary->num_axes < 1 || rotary->num_axes > 4)
      return fail(KVQ_ERR_UNSUPPORTED, "%s: %d position axes (1 to 4)", where, rotary->num_axes);
    if ((p.T && !rotary->positions) || !rotary->inv_freq || !aligned(rotary->positions, 8) || !aligned(rotary->inv_freq, 4) ||
        !aligned(rotary->pair_axis, 4))
      return fail(KVQ_ERR_INVALID_ARG, "%s: rotary tables null or misaligned", where);
    if (!(std::fabs(rotary->scale) <= FLT_MAX)) return fail(KVQ_ERR_INVALID_ARG, "%s: bad rotary scale", where);
    if (rotary->num_axes > 1 && rotary->positions_stride != 0 && rotary->positions_stride < p.T)
      return fail(KVQ_ERR_INVALID_ARG, "%s: positions_stride must be 0 or at least T", where);
    p.rotary = *rotary;
  }
  return KVQ_OK;
}

// Checks of the cache arguments; fills them in.
kvq_status_t take_cache(TokenParams& p, const int64_t* slot_mapping, void* k_cache, void* v_cache, const float* k_scale,
                        const float* v_scale, int fmt, int D, int64_t num_blocks, int* dev_status, const char* where) {
  if (!slot_mapping || !k_cache || !v_cache) return fail(KVQ_ERR_INVALID_ARG, "%s: null pointer", where);
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slot_mapping, 8))
    return fail(KVQ_ERR_INVALID_ARG, "%s: misaligned pointer", where);
  const bool per_head = fmt == kE4M3 || fmt == kE5M2 || fmt == kFP4;
  if (per_head && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4)))
    return fail(KVQ_ERR_INVALID_ARG, "%s: this cache needs k_scale and v_scale", where);
  const PageStrides ps = page_strides(k_cache, v_cache, k_page_bytes(fmt, D), v_page_bytes(fmt, D));
  p.slots = slot_mapping;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.k_str = ps.k;
  p.v_str = ps.v;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.num_slots = num_blocks * kPage;
  p.dev_status = dev_status;
  return KVQ_OK;
}

}  // namespace

kvq_status_t write_fp4(const void* k, const void* v, const int64_t* slot_mapping, void* k_cache, void* v_cache,
                       const float* k_scale, const float* v_scale, int T, int Hkv, int D, int64_t num_blocks,
                       int* dev_status, cudaStream_t s) {
  TokenParams p = {};
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_stride = p.v_stride = static_cast<int64_t>(Hkv) * D;
  p.T = T;
  p.Hkv = Hkv;
  const kvq_status_t st =
      take_cache(p, slot_mapping, k_cache, v_cache, k_scale, v_scale, kFP4, D, num_blocks, dev_status, "reshape_and_cache");
  return st != KVQ_OK ? st : launch_tokens<kFP4, false>(p, D, s, "reshape_and_cache");
}

}  // namespace kvq

using namespace kvq;

extern "C" kvq_status_t kvq_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                         const kvq_head_norm_t* norm, const kvq_rotary_t* rotary, void* q_out,
                                         int64_t q_out_stride, void* k_out, int64_t k_out_stride, int T, int Hq, int Hkv,
                                         int D, int* dev_status, kvq_stream_t stream) {
  clear_error();
  if (T < 0 || Hq < 0 || Hkv < 0 || Hq + static_cast<int64_t>(Hkv) < 1)
    return fail(KVQ_ERR_INVALID_ARG, "qk_norm_rope: bad sizes");
  if (D != 64 && D != 128 && D != 256) return fail(KVQ_ERR_UNSUPPORTED, "qk_norm_rope: head_dim %d (64, 128 or 256)", D);
  TokenParams p = {};
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.dev_status = dev_status;
  const kvq_status_t st = take_turn(p, norm, rotary, D, "qk_norm_rope");
  if (st != KVQ_OK || T == 0) return st;
  if ((Hq && (!q || !q_out)) || (Hkv && (!k || !k_out))) return fail(KVQ_ERR_INVALID_ARG, "qk_norm_rope: null pointer");
  if ((Hq && (!rows_ok(q, q_stride, Hq, D) || !rows_ok(q_out, q_out_stride, Hq, D))) ||
      (Hkv && (!rows_ok(k, k_stride, Hkv, D) || !rows_ok(k_out, k_out_stride, Hkv, D))))
    return fail(KVQ_ERR_INVALID_ARG, "qk_norm_rope: rows must be 16-byte aligned, heads * D or more apart");
  if ((Hq && !in_place_ok(q, q_stride, q_out, q_out_stride, T)) || (Hkv && !in_place_ok(k, k_stride, k_out, k_out_stride, T)))
    return fail(KVQ_ERR_INVALID_ARG, "qk_norm_rope: in place, the strides must be the same");
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  return launch_tokens<kRowsOnly>(p, D, static_cast<cudaStream_t>(stream), "qk_norm_rope");
}

extern "C" kvq_status_t kvq_rope_and_cache(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                           const void* v, int64_t v_stride, const kvq_head_norm_t* norm,
                                           const kvq_rotary_t* rotary, const int64_t* slot_mapping, void* k_cache,
                                           void* v_cache, const float* k_scale, const float* v_scale, void* q_out,
                                           int64_t q_out_stride, uint8_t* q8, const float* q_scale, int T, int Hq,
                                           int Hkv, int D, int P, int64_t num_blocks, kvq_dtype_t cache_dtype,
                                           int per_token, int* dev_status, kvq_stream_t stream) {
  clear_error();
  if (T < 0 || Hq < 0 || Hkv < 1 || num_blocks < 1) return fail(KVQ_ERR_INVALID_ARG, "rope_and_cache: bad sizes");
  if (P != kPage) return fail(KVQ_ERR_UNSUPPORTED, "rope_and_cache: page size %d (only 16)", P);
  int fmt;
  if (!cache_format(cache_dtype, per_token != 0, &fmt))
    return fail(KVQ_ERR_INVALID_ARG, "rope_and_cache: bad cache dtype (per-token scales need FP8)");
  if (D != 64 && D != 128 && !(D == 256 && (fmt == kE4M3 || fmt == kE5M2)))
    return fail(KVQ_ERR_UNSUPPORTED, "rope_and_cache: head_dim %d (64 or 128; 256 for FP8 with per-head scales)", D);
  TokenParams p = {};
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  kvq_status_t st = take_turn(p, norm, rotary, D, "rope_and_cache");
  if (st != KVQ_OK || T == 0) return st;
  if (!k || !v || (Hq && (!q || (!q_out && !q8)))) return fail(KVQ_ERR_INVALID_ARG, "rope_and_cache: null pointer");
  if (Hq && q8 && (!q_scale || !aligned(q_scale, 4) || !aligned(q8, 16)))
    return fail(KVQ_ERR_INVALID_ARG, "rope_and_cache: q8 needs q_scale and 16-byte alignment");
  if (!rows_ok(k, k_stride, Hkv, D) || !rows_ok(v, v_stride, Hkv, D) || (Hq && !rows_ok(q, q_stride, Hq, D)) ||
      (Hq && q_out && !rows_ok(q_out, q_out_stride, Hq, D)))
    return fail(KVQ_ERR_INVALID_ARG, "rope_and_cache: rows must be 16-byte aligned, heads * D or more apart");
  if (Hq && !in_place_ok(q, q_stride, q_out, q_out_stride, T))
    return fail(KVQ_ERR_INVALID_ARG, "rope_and_cache: in place, the strides must be the same");
  st = take_cache(p, slot_mapping, k_cache, v_cache, k_scale, v_scale, fmt, D, num_blocks, dev_status, "rope_and_cache");
  if (st != KVQ_OK) return st;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.q_out_stride = q_out_stride;
  p.q8 = q8;
  p.q_scale = q_scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (fmt) {
    case kE4M3: return launch_tokens<kE4M3>(p, D, s, "rope_and_cache");
    case kE5M2: return launch_tokens<kE5M2>(p, D, s, "rope_and_cache");
    case kBF16: return launch_tokens<kBF16>(p, D, s, "rope_and_cache");
    case kFP4: return launch_tokens<kFP4>(p, D, s, "rope_and_cache");
    case kE4M3Token: return launch_tokens<kE4M3Token>(p, D, s, "rope_and_cache");
    default: return launch_tokens<kE5M2Token>(p, D, s, "rope_and_cache");
  }
}
