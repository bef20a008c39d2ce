// kvq_qk_norm_rope, kvq_rope_and_cache, and the 4-bit form of
// kvq_reshape_and_cache: one kernel that takes tokens' q, k and v rows, norms
// and turns q and k, and writes rows or cache pages.
//
// Mathematics.  y = x * rsqrt(mean x^2 + eps) * w per head, then each pair is
// turned by a = position * inv_freq.  Norm weight and rotation fold into two
// factors per dim that do not depend on the head: with p(d) the pair's other
// dim, out_d = r * (x_d A_d + x_p(d) B_d), A_d = w_d cos a, B_d = -+ w_p(d) sin a,
// r the head's norm factor.  A lane holds eight dims of one token and walks
// heads, so angles, sines and weights are paid once per token and CTA.
//
// The angle is taken in turns in 64-bit fixed point: inv_freq / 2 pi as a
// 64-bit fraction times the position, whose overflow is the reduction by whole
// turns.  No float64 (two operations a clock per SM here) and no position too
// far for float32.
//
// Bound: memory.  Every row is read once and written once.
#include <cfloat>
#include <cmath>

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
  const uint64_t m = e ? (u & 0x7FFFFFu) | 0x800000u : u & 0x7FFFFFu;
  // inv_freq = m 2^(e - 150) (e = 1 for subnormals), so the fraction is
  // (m kInvTwoPi / 2^24) 2^(e - 128)
  const uint64_t f = __umul64hi(m << 40, kInvTwoPi);
  const int shift = (e ? e : 1) - 128;
  const uint64_t x = shift <= -64 ? 0 : shift < 0 ? f >> -shift : shift < 64 ? f << shift : 0;
  return u >> 31 ? 0 - x : x;
}

// Sine and cosine of a fraction of a turn: to the nearest quarter, then the rest.
KVQ_DEVINL void sincos_turns(uint64_t turns, float& s, float& c) {
  const uint32_t t = static_cast<uint32_t>(turns >> 32);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const int rest = static_cast<int>(t - (quarter << 30));  // within an eighth of a turn
  float s0, c0;
  sincospif(static_cast<float>(rest) * 0x1p-31f, &s0, &c0);
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
  int tiles, q_chunk, kv_chunk, kv_chunks;  // CTAs: tiles x (kv_chunks, then chunks of q heads)
  int* dev_status;
};

// The factors of a lane's eight dims (see the top of the file).
struct Turn {
  float a[8], b[8];
  int from;     // lane that holds the pairs' other dims
  bool swap;    // they are the neighbours instead
  bool turned;  // false: b is zero, and so is what it multiplies
};

template <int D>
KVQ_DEVINL Turn make_turn(const TokenParams& p, const __nv_bfloat16* weight, int token, int lane) {
  constexpr int LPT = D / 8;
  const int j = lane % LPT;
  Turn t;
  t.from = lane;
  t.swap = false;
  const int rot = p.rotary.rot_dim, half = rot / 2;
  const bool turned = t.turned = 8 * j < rot;
  int partner = j;
  if (p.rotary.interleaved)
    t.swap = true;
  else if (turned)
    partner = 8 * j < half ? j + half / 8 : j - half / 8;
  t.from = lane - j + partner;
  float w[8], wp[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = wp[i] = 1.f;
  if (weight) {
    unpack8_bf16(__ldg(reinterpret_cast<const uint4*>(weight) + j), w);
    unpack8_bf16(__ldg(reinterpret_cast<const uint4*>(weight) + partner), wp);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.a[i] = w[i];
    t.b[i] = 0.f;
  }
  if (!turned) return t;
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
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float s, c;
      angle(4 * j + i, s, c);
      t.a[2 * i] = c * w[2 * i];
      t.b[2 * i] = -s * w[2 * i + 1];
      t.a[2 * i + 1] = c * w[2 * i + 1];
      t.b[2 * i + 1] = s * w[2 * i];
    }
  } else {
    const bool low = 8 * j < half;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s, c;
      angle((low ? 8 * j : 8 * j - half) + i, s, c);
      t.a[i] = c * w[i];
      t.b[i] = (low ? -s : s) * wp[i];
    }
  }
  return t;
}

// Norm and rotation of a lane's eight dims; every lane of the warp takes part.
template <int D>
KVQ_DEVINL void turn_row(const Turn& t, bool norm, float eps, const uint4& raw, float (&o)[8]) {
  constexpr int LPT = D / 8;
  float x[8], y[8];
  unpack8_bf16(raw, x);
  uint4 other;
  other.x = __shfl_sync(0xffffffffu, raw.x, t.from);
  other.y = __shfl_sync(0xffffffffu, raw.y, t.from);
  other.z = __shfl_sync(0xffffffffu, raw.z, t.from);
  other.w = __shfl_sync(0xffffffffu, raw.w, t.from);
  unpack8_bf16(other, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (t.swap) y[i] = x[i ^ 1];
    if (!t.turned) y[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = fmaf(x[i], t.a[i], y[i] * t.b[i]);
  if (norm) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
    for (int off = 1; off < LPT; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const float r = rsqrtf(fmaf(sum, 1.f / D, eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= r;
  }
}

// One tile of 16 tokens: a thread holds dims 8 j .. 8 j + 7 of token tid / LPT.
template <int D, int FMT>
__global__ void __launch_bounds__(kPage * D / 8) token_kernel(const TokenParams p) {
  using F = Format<FMT>;
  constexpr int LPT = D / 8;
  const int tid = threadIdx.x, lane = tid & 31;
  const int t = tid / LPT, j = tid % LPT;
  const int tile = blockIdx.x % p.tiles, chunk = blockIdx.x / p.tiles;
  const int token = tile * kPage + t;
  const bool live = token < p.T;
  const int row = live ? token : p.T - 1;  // a token to take angles of

  if (chunk >= p.kv_chunks || FMT == kRowsOnly) {
    // rows in, rows out
    const bool is_q = chunk >= p.kv_chunks;
    const __nv_bfloat16* weight = is_q ? p.q_weight : p.k_weight;
    const Turn turn = make_turn<D>(p, weight, row, lane);
    const int per = is_q ? p.q_chunk : p.kv_chunk, heads = is_q ? p.Hq : p.Hkv;
    const int h0 = (is_q ? chunk - p.kv_chunks : chunk) * per, h1 = min(heads, h0 + per);
    const __nv_bfloat16* src = (is_q ? p.q : p.k) + row * (is_q ? p.q_stride : p.k_stride) + 8 * j;
    __nv_bfloat16* dst = is_q ? p.q_out : p.k_out;
    if (dst) dst += row * (is_q ? p.q_out_stride : p.k_out_stride) + 8 * j;
    uint8_t* codes = is_q && p.q8 ? p.q8 + static_cast<int64_t>(row) * p.Hq * D + 8 * j : nullptr;
    const float s = codes ? __ldg(p.q_scale) : 1.f;
    for (int h = h0; h < h1; ++h) {
      float o[8];
      turn_row<D>(turn, weight != nullptr, p.eps, *reinterpret_cast<const uint4*>(src + h * D), o);
      if (!live) continue;
      if (dst) *reinterpret_cast<uint4*>(dst + h * D) = pack8_bf16(o);
      if (codes) *reinterpret_cast<uint2*>(codes + h * D) = quant8_fp8<false>(o, s);
    }
    return;
  }

  if constexpr (FMT != kRowsOnly) {
    const Turn turn = make_turn<D>(p, p.k_weight, row, lane);
    const int64_t slot = live ? p.slots[token] : -1;
    if (slot >= p.num_slots && j == 0) set_status(p.dev_status, KVQ_DEV_BAD_SLOT);
    const bool valid = slot >= 0 && slot < p.num_slots;
    const int off = static_cast<int>(slot % kPage);
    const int h0 = chunk * p.kv_chunk, h1 = min(p.Hkv, h0 + p.kv_chunk);
    for (int h = h0; h < h1; ++h) {
      const uint4 kr = *reinterpret_cast<const uint4*>(p.k + row * p.k_stride + h * D + 8 * j);
      const uint4 vr = *reinterpret_cast<const uint4*>(p.v + row * p.v_stride + h * D + 8 * j);
      float ko[8], vo[8];
      turn_row<D>(turn, p.k_weight != nullptr, p.eps, kr, ko);
      unpack8_bf16(vr, vo);
      const int64_t page = valid ? slot / kPage * p.Hkv + h : 0;
      uint8_t* kp = p.k_cache + page * p.k_str;
      uint8_t* vp = p.v_cache + page * p.v_str;
      if constexpr (F::kFp8) {
        float ks, vs;
        if constexpr (F::kToken) {
          float ka = amax8(ko), va = amax8(vo);
#pragma unroll
          for (int o = 1; o < LPT; o <<= 1) {
            ka = fmaxf(ka, __shfl_xor_sync(0xffffffffu, ka, o));
            va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, o));
          }
          ks = ka > 0.f ? __fdiv_rn(ka, F::kMax) : 1.f;  // an all-zero token keeps scale 1
          vs = va > 0.f ? __fdiv_rn(va, F::kMax) : 1.f;
          if (valid && j == 0) {
            float* tail = reinterpret_cast<float*>(vp + kPage * D);
            tail[off] = ks;
            tail[kPage + off] = vs;
          }
        } else {
          ks = __ldg(p.k_scale + h);
          vs = __ldg(p.v_scale + h);
        }
        if (!valid) continue;
        *reinterpret_cast<uint2*>(kp + fp8_k_offset(off, j >> 1, D) + (j & 1) * 8) = quant8_fp8<F::kE5>(ko, ks);
        const uint2 codes = quant8_fp8<F::kE5>(vo, vs);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          vp[(8 * j + i) * kPage + fp8_v_slot(off)] = static_cast<uint8_t>((i < 4 ? codes.x : codes.y) >> (8 * (i & 3)));
      } else if constexpr (FMT == kBF16) {
        if (!valid) continue;
        *reinterpret_cast<uint4*>(kp + k_chunk_offset(off, j, 2 * D)) = pack8_bf16(ko);
        const uint32_t w[4] = {vr.x, vr.y, vr.z, vr.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint16_t*>(vp + bf16_v_offset(8 * j + i, off)) = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
      } else {
        uint8_t ks, vs;
        const uint32_t kw = quant8_fp4(ko, __ldg(p.k_scale + h), ks);
        const uint32_t vw = quant8_fp4(vo, __ldg(p.v_scale + h), vs);
        if (!valid) continue;
        *reinterpret_cast<uint32_t*>(kp + off * (D / 2) + 4 * j) = kw;
#pragma unroll
        for (int i = 0; i < 4; ++i) vp[fp4_v_offset(off, 4 * j + i)] = static_cast<uint8_t>(vw >> (8 * i));
        if ((j & 1) == 0) {
          kp[kPage * D / 2 + off * (D / 16) + j / 2] = ks;
          vp[kPage * D / 2 + fp4_v_scale_offset(off, j / 2)] = vs;
        }
      }
    }
  }
}

template <int FMT>
kvq_status_t launch_tokens(TokenParams& p, int D, cudaStream_t s, const char* where) {
  p.tiles = (p.T - 1) / kPage + 1;
  p.kv_chunk = 1;
  p.q_chunk = 4;
  p.kv_chunks = (p.Hkv + p.kv_chunk - 1) / p.kv_chunk;
  const int64_t ctas = static_cast<int64_t>(p.tiles) * (p.kv_chunks + (p.Hq + p.q_chunk - 1) / p.q_chunk);
  if (ctas > 0x7FFFFFFF) return fail(KVQ_ERR_UNSUPPORTED, "%s: problem too large", where);
  const unsigned grid = static_cast<unsigned>(ctas);
  if (D == 64) {
    token_kernel<64, FMT><<<grid, 128, 0, s>>>(p);
  } else if (D == 128) {
    token_kernel<128, FMT><<<grid, 256, 0, s>>>(p);
  } else if constexpr (FMT == kRowsOnly || FMT == kE4M3 || FMT == kE5M2) {
    token_kernel<256, FMT><<<grid, 512, 0, s>>>(p);
  }
  return cuda_status(cudaGetLastError(), where);
}

bool rows_ok(const void* x, int64_t stride, int heads, int D) {
  return aligned(x, 16) && stride % 8 == 0 && stride >= static_cast<int64_t>(heads) * D;
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
    if (rotary->num_axes > 1 && rotary->positions_stride < p.T)
      return fail(KVQ_ERR_INVALID_ARG, "%s: positions_stride < T", where);
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
  return st != KVQ_OK ? st : launch_tokens<kFP4>(p, D, s, "reshape_and_cache");
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
