// kvq_gather_cache: cached tokens back as bf16 rows.
//
// value = bf16(fl32(code * scale)).  Bound: memory (codes in, two bytes per
// element out): 32,763 tokens of 8 KV heads of 128 from an E4M3 cache in 34 us,
// 5.9 TB/s of the measured copy rate of 6.8 (66 us with each token's V bytes read one by
// one, 51 us as whole words with the next head's in registers); 16,000 from a 4-bit
// cache in 18.3 us, 4.6 TB/s, where no unit is full (issue slots 58%, ALU pipe 45%).
// 32,763 tokens from BF16 43.5 us, 6.2 TB/s, with scales per token 36.
#include "kvq_host.h"
#include "kvq_rows.cuh"

namespace kvq {

namespace {

struct GatherParams {
  const int64_t* slots;
  const uint8_t *k_cache, *v_cache;
  int64_t k_str, v_str;
  const float *k_scale, *v_scale;
  int64_t num_slots;
  __nv_bfloat16 *k_out, *v_out;
  int T, Hkv;
  int tiles, chunk;  // CTAs: tiles x chunks of heads
  bool aligned;
  int* dev_status;
};

// Eight codes, a byte each, as values times s.
template <bool E5>
KVQ_DEVINL void value8_fp8(const uint2& c, float s, float2 (&x)[4]) {
  const float2 ss = make_float2(s, s);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    fp8x4_to_f16x2x2<E5>(i ? c.y : c.x, lo, hi);
    x[2 * i] = fmul2(__half22float2(*reinterpret_cast<__half2*>(&lo)), ss);
    x[2 * i + 1] = fmul2(__half22float2(*reinterpret_cast<__half2*>(&hi)), ss);
  }
}
// Eight E2M1 codes times the block's scale (exact) times s.
KVQ_DEVINL void value8_fp4(uint32_t c, uint8_t block, float s, float2 (&x)[4]) {
  const float b = e4m3_value(block);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __half2(__nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(c >> (8 * i)), __NV_E2M1));
    x[i] = fmul2(fmul2(__half22float2(h), make_float2(b, b)), make_float2(s, s));
  }
}

// One thread's eight dims of a token, from the pages themselves.
template <int D, int FMT>
KVQ_DEVINL void one_token(const GatherParams& p, const uint8_t* kp, const uint8_t* vp, int off, int j, int h, uint4& k, uint4& v) {
  using F = Format<FMT>;
  if constexpr (FMT == kBF16) {
    k = *reinterpret_cast<const uint4*>(kp + k_chunk_offset(off, j, 2 * D));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i >> 1] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(vp + bf16_v_offset(8 * j + i, off))) << (16 * (i & 1));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float2 kf[4], vf[4];
    if constexpr (FMT == kFP4) {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) w |= static_cast<uint32_t>(vp[fp4_v_offset(off, 4 * j + i)]) << (8 * i);
      value8_fp4(*reinterpret_cast<const uint32_t*>(kp + off * (D / 2) + 4 * j), kp[kPage * D / 2 + off * (D / 16) + j / 2],
                 __ldg(p.k_scale + h), kf);
      value8_fp4(w, vp[kPage * D / 2 + fp4_v_scale_offset(off, j / 2)], __ldg(p.v_scale + h), vf);
    } else {
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i >> 2] |= static_cast<uint32_t>(vp[(8 * j + i) * kPage + fp8_v_slot(off)]) << (8 * (i & 3));
      const float* tail = reinterpret_cast<const float*>(vp + kPage * D);
      value8_fp8<F::kE5>(*reinterpret_cast<const uint2*>(kp + fp8_k_offset(off, j >> 1, D) + (j & 1) * 8),
                         F::kToken ? tail[off] : __ldg(p.k_scale + h), kf);
      value8_fp8<F::kE5>(make_uint2(w[0], w[1]), F::kToken ? tail[kPage + off] : __ldg(p.v_scale + h), vf);
    }
    k = pack8_bf16(kf);
    v = pack8_bf16(vf);
  }
}

// Whole pages pass through shared memory, their V part turned by transposing
// matrix loads: a matrix's rows are eight 16-byte chunks of the page, and a lane
// gets two rows' values of the same two (FP8, FP4) or one (BF16) tokens.  Rows
// are chosen so that a lane's four matrices hold neighbouring dims, and chunks
// placed so that a matrix's rows lie in different banks.
template <int D, int FMT>
struct Staged {
  using F = Format<FMT>;
  static constexpr int kKPage = static_cast<int>(k_page_bytes(FMT, D)), kVPage = static_cast<int>(v_page_bytes(FMT, D));
  static constexpr int kStageB = kKPage + kVPage;
  static constexpr int kStages = 4;
  static constexpr int kThreads = kPage * D / 8;
  static constexpr int kCodes = FMT == kFP4 ? kPage * D / 2 : kPage * D * (FMT == kBF16 ? 2 : 1);
  static_assert(kCodes % 512 == 0 && kStageB % 16 == 0, "whole 16-byte chunks, and whole groups of those that change places");

  // Where the V page's 16-byte chunk x goes.
  static KVQ_DEVINL int place(int x) {
    if constexpr (F::kFp8) {
      return x < kCodes / 16 ? x ^ (((x >> 3) & 3) << 1) : x;  // row x is dim x
    } else if constexpr (FMT == kBF16) {
      return x ^ ((x >> 4) & 1) ^ (((x >> 5) & 1) << 2);  // row x / 2
    } else {
      return x;
    }
  }
  static KVQ_DEVINL void copy(uint32_t stage, const uint8_t* kp, const uint8_t* vp) {
#pragma unroll
    for (int x = threadIdx.x; x < kStageB / 16; x += kThreads) {
      if (x < kKPage / 16)
        copy16(stage + x * 16, kp + x * 16);
      else
        copy16(stage + kKPage + place(x - kKPage / 16) * 16, vp + (x - kKPage / 16) * 16);
    }
  }

  // This thread's part of a head's rows: put(token of the tile, dim, is_v, eight dims).
  template <typename Put>
  static KVQ_DEVINL void rows(uint32_t stage, float ks, float vs, Put put) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i = lane & 7, m = lane >> 3, u = lane >> 2, c = lane & 3;
    const uint32_t v = stage + kKPage;
    uint32_t w[4];
    if constexpr (FMT == kBF16) {
      const int t = threadIdx.x / (D / 8), j = threadIdx.x % (D / 8);
      put(t, 8 * j, false, lds128(stage + k_chunk_offset(t, j, 2 * D)));
      const int base = 32 * (warp >> 1), half = warp & 1;
      const int d = base + 8 * (i >> 1) + 2 * m + (i & 1);
      ldsm_x4_t(v + place(2 * d + (half ^ ((d >> 2) & 1))) * 16, w);
      put(8 * half + u, base + 8 * c, true, make_uint4(w[0], w[1], w[2], w[3]));
    } else if constexpr (F::kFp8) {
      constexpr int kVWarps = D / 32;  // the others take K
      if (warp < kVWarps) {
        const int d = 32 * warp + 8 * (i >> 1) + 2 * m + (i & 1);
        ldsm_x4_t(v + place(d) * 16, w);
        const int t = u & 1 ? 7 + u : u;  // slots 2u, 2u + 1 hold tokens t, t + 1
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t pick = e ? 0x7531 : 0x6420;
          float2 x[4];
          value8_fp8<F::kE5>(make_uint2(__byte_perm(w[0], w[1], pick), __byte_perm(w[2], w[3], pick)),
                             F::kToken ? lds_f32(v + kCodes + (kPage + t + e) * 4) : vs, x);
          put(t + e, 32 * warp + 8 * c, true, pack8_bf16(x));
        }
      } else {
        const int y = threadIdx.x - 32 * kVWarps, j = y % (D / 8);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = y / (D / 8) + 8 * e;
          float2 x[4];
          value8_fp8<F::kE5>(lds64(stage + fp8_k_offset(t, j >> 1, D) + (j & 1) * 8), F::kToken ? lds_f32(v + kCodes + t * 4) : ks, x);
          put(t, 8 * j, false, pack8_bf16(x));
        }
      }
    } else {
      constexpr int kVWarps = D / 64;
      if (warp < kVWarps) {
        ldsm_x4_t(v + (warp * 32 + (2 * m + (i & 1)) * 4 + (i >> 1)) * 16, w);
        // the lane has 16 dims of tokens 2c + 8 hi, + 1; with its neighbour in hi it
        // changes halves, so that they write 32 bytes of a row between them
        const int b = u >> 1, hi = u & 1;
        uint32_t code[4];  // tokens 2c, 2c + 1, 2c + 8, 2c + 9; dims 8 hi .. + 7 of the block
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t pick = e ? 0x7531 : 0x6420;
          const uint32_t q0 = __byte_perm(w[0], w[1], pick), q1 = __byte_perm(w[2], w[3], pick);
          const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? q0 : q1, 4);
          code[e] = hi ? got : q0;
          code[2 + e] = hi ? q1 : got;
        }
        const uint32_t scales = lds32(v + kCodes + warp * 64 + c * 16 + b * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 x[4];
          value8_fp4(code[e], static_cast<uint8_t>(scales >> (8 * e)), vs, x);
          put(2 * c + (e & 1) + 8 * (e >> 1), 64 * warp + 16 * b + 8 * hi, true, pack8_bf16(x));
        }
      } else if (warp < kVWarps + D / 32) {
        const int y = threadIdx.x - 32 * kVWarps, j = y % (D / 8);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = y / (D / 8) + 8 * e;
          float2 x[4];
          value8_fp4(lds32(stage + t * (D / 2) + 4 * j), static_cast<uint8_t>(lds8(stage + kCodes + t * (D / 16) + j / 2)), ks, x);
          put(t, 8 * j, false, pack8_bf16(x));
        }
      }
    }
  }
};

// A tile's tokens, a chunk of heads.  Six CTAs of 256 threads an SM (40
// registers; E4M3 and E5M2 without a spill, with scales per token 4 bytes, 4 bits 24): with five
// 35.5 us for the 32,763 tokens from E4M3, with eight, spilling, 41.
template <int D, int FMT>
__global__ void __launch_bounds__(kPage * D / 8, 1536 / (2 * D)) gather_kernel(const GatherParams p) {
  using S = Staged<D, FMT>;
  constexpr int LPT = D / 8;
  __shared__ TileTokens tt;
  __shared__ __align__(128) uint8_t stages[S::kStages * S::kStageB];
  const uint32_t ring = smem_u32(stages);
  const int x = threadIdx.x, t = x / LPT, j = x % LPT;
  const int tile = blockIdx.x % p.tiles;
  const int h0 = blockIdx.x / p.tiles * p.chunk, n = min(p.Hkv - h0, p.chunk);
  if (x < 32) find_tokens(tt, p.slots, p.T, p.num_slots, tile, p.aligned, p.dev_status);
  __syncthreads();
  const int tokens = tt.n;
  for (int r = 0; r < tokens; r += kPage) {
    if (r == 0 && tt.page) {
      const int64_t page = tt.slot[0] / kPage * p.Hkv + h0;
      const uint8_t* kp = p.k_cache + page * p.k_str;
      const uint8_t* vp = p.v_cache + page * p.v_str;
      auto issue = [&](int i) {
        if (i < n) S::copy(ring + i % S::kStages * S::kStageB, kp + i * p.k_str, vp + i * p.v_str);
        copy_commit();
      };
#pragma unroll
      for (int i = 0; i < S::kStages - 1; ++i) issue(i);
      for (int i = 0; i < n; ++i) {
        copy_wait<S::kStages - 2>();
        __syncthreads();  // everybody's copies are there, and the stage before is read
        issue(i + S::kStages - 1);
        float ks = 1.f, vs = 1.f;
        if (FMT != kBF16 && !Format<FMT>::kToken) {
          ks = __ldg(p.k_scale + h0 + i);
          vs = __ldg(p.v_scale + h0 + i);
        }
        S::rows(ring + i % S::kStages * S::kStageB, ks, vs, [&](int token, int d, bool is_v, const uint4& o) {
          const int64_t at = (static_cast<int64_t>(tt.token[token]) * p.Hkv + h0 + i) * D + d;
          *reinterpret_cast<uint4*>((is_v ? p.v_out : p.k_out) + at) = o;
        });
      }
    } else if (r + t < tokens) {
      const int64_t slot = tt.slot[r + t];
      const int64_t page = slot / kPage * p.Hkv + h0;
      for (int i = 0; i < n; ++i) {
        uint4 k, v;
        one_token<D, FMT>(p, p.k_cache + (page + i) * p.k_str, p.v_cache + (page + i) * p.v_str,
                          static_cast<int>(slot % kPage), j, h0 + i, k, v);
        const int64_t at = (static_cast<int64_t>(tt.token[r + t]) * p.Hkv + h0 + i) * D + 8 * j;
        *reinterpret_cast<uint4*>(p.k_out + at) = k;
        *reinterpret_cast<uint4*>(p.v_out + at) = v;
      }
    }
  }
}

template <int FMT>
kvq_status_t launch_gather(GatherParams& p, int D, cudaStream_t s) {
  p.aligned = p.T >= 64;  // no difference below, nor for tokens each of another page
  p.tiles = (p.T - 1) / kPage + 1 + (p.aligned ? 1 : 0);
  // heads to a CTA: 4 where that leaves work for every SM (8 of them: 35.8 us for the 32,763 tokens)
  p.chunk = heads_per_cta(p.Hkv, p.tiles, 4, 4 * sm_count());
  const int64_t ctas = static_cast<int64_t>(p.tiles) * ((p.Hkv + static_cast<int64_t>(p.chunk) - 1) / p.chunk);
  if (ctas > 0x7FFFFFFF) return fail(KVQ_ERR_UNSUPPORTED, "gather_cache: problem too large");
  const unsigned grid = static_cast<unsigned>(ctas);
  if (D == 64) {
    gather_kernel<64, FMT><<<grid, 128, 0, s>>>(p);
  } else if (D == 128) {
    gather_kernel<128, FMT><<<grid, 256, 0, s>>>(p);
  } else if constexpr (FMT == kE4M3 || FMT == kE5M2) {
    gather_kernel<256, FMT><<<grid, 512, 0, s>>>(p);
  }
  return cuda_status(cudaGetLastError(), "gather_cache launch");
}

}  // namespace

bool cache_format(kvq_dtype_t dtype, bool per_token, int* fmt) {
  switch (dtype) {
    case KVQ_DTYPE_FP8_E4M3: *fmt = per_token ? kE4M3Token : kE4M3; return true;
    case KVQ_DTYPE_FP8_E5M2: *fmt = per_token ? kE5M2Token : kE5M2; return true;
    case KVQ_DTYPE_BF16: *fmt = kBF16; return !per_token;
    case KVQ_DTYPE_FP4_E2M1: *fmt = kFP4; return !per_token;
  }
  return false;
}

}  // namespace kvq

using namespace kvq;

extern "C" kvq_status_t kvq_gather_cache(const int64_t* slot_mapping, const void* k_cache, const void* v_cache,
                                         const float* k_scale, const float* v_scale, void* k_out, void* v_out, int T,
                                         int Hkv, int D, int P, int64_t num_blocks, kvq_dtype_t cache_dtype,
                                         int per_token, int* dev_status, kvq_stream_t stream) {
  clear_error();
  if (T < 0 || Hkv < 1 || num_blocks < 1) return fail(KVQ_ERR_INVALID_ARG, "gather_cache: bad sizes");
  if (P != kPage) return fail(KVQ_ERR_UNSUPPORTED, "gather_cache: page size %d (only 16)", P);
  int fmt;
  if (!cache_format(cache_dtype, per_token != 0, &fmt))
    return fail(KVQ_ERR_INVALID_ARG, "gather_cache: bad cache dtype (per-token scales need FP8)");
  if (D != 64 && D != 128 && !(D == 256 && (fmt == kE4M3 || fmt == kE5M2)))
    return fail(KVQ_ERR_UNSUPPORTED, "gather_cache: head_dim %d (64 or 128; 256 for FP8 with per-head scales)", D);
  if (T == 0) return KVQ_OK;
  if (!slot_mapping || !k_cache || !v_cache || !k_out || !v_out)
    return fail(KVQ_ERR_INVALID_ARG, "gather_cache: null pointer");
  const bool per_head = fmt == kE4M3 || fmt == kE5M2 || fmt == kFP4;
  if (per_head && (!k_scale || !v_scale)) return fail(KVQ_ERR_INVALID_ARG, "gather_cache: this cache needs k_scale and v_scale");
  if (!aligned(slot_mapping, 8) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_out, 16) ||
      !aligned(v_out, 16) || (per_head && (!aligned(k_scale, 4) || !aligned(v_scale, 4))))
    return fail(KVQ_ERR_INVALID_ARG, "gather_cache: misaligned pointer");
  const PageStrides ps = page_strides(k_cache, v_cache, k_page_bytes(fmt, D), v_page_bytes(fmt, D));
  GatherParams p;
  p.slots = slot_mapping;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_str = ps.k;
  p.v_str = ps.v;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.num_slots = num_blocks * kPage;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.T = T;
  p.Hkv = Hkv;
  p.dev_status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (fmt) {
    case kE4M3: return launch_gather<kE4M3>(p, D, s);
    case kE5M2: return launch_gather<kE5M2>(p, D, s);
    case kBF16: return launch_gather<kBF16>(p, D, s);
    case kFP4: return launch_gather<kFP4>(p, D, s);
    case kE4M3Token: return launch_gather<kE4M3Token>(p, D, s);
    default: return launch_gather<kE5M2Token>(p, D, s);
  }
}
