// kvq_gather_cache: cached tokens back as bf16 rows.
//
// value = bf16(fl32(code * scale)).  Bound: memory (codes in, two bytes per
// element out).
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
  int* dev_status;
};

// Eight codes, a byte each, as values times s.
template <bool E5>
KVQ_DEVINL void value8_fp8(const uint2& c, float s, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    fp8x4_to_f16x2x2<E5>(i ? c.y : c.x, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    x[4 * i] = __fmul_rn(a.x, s);
    x[4 * i + 1] = __fmul_rn(a.y, s);
    x[4 * i + 2] = __fmul_rn(b.x, s);
    x[4 * i + 3] = __fmul_rn(b.y, s);
  }
}
// Eight E2M1 codes times the block's scale (exact) times s.
KVQ_DEVINL void value8_fp4(uint32_t c, uint8_t block, float s, float (&x)[8]) {
  const float b = e4m3_value(block);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __half2(__nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(c >> (8 * i)), __NV_E2M1));
    const float2 f = __half22float2(h);
    x[2 * i] = __fmul_rn(f.x * b, s);
    x[2 * i + 1] = __fmul_rn(f.y * b, s);
  }
}

// A tile of 16 tokens; a thread holds dims 8 j .. 8 j + 7 of one.
template <int D, int FMT>
__global__ void __launch_bounds__(kPage * D / 8) gather_kernel(const GatherParams p) {
  using F = Format<FMT>;
  constexpr int LPT = D / 8;
  const int t = threadIdx.x / LPT, j = threadIdx.x % LPT;
  const int token = blockIdx.x % p.tiles * kPage + t;
  if (token >= p.T) return;
  const int64_t slot = p.slots[token];
  if (slot >= p.num_slots && j == 0) set_status(p.dev_status, KVQ_DEV_BAD_SLOT);
  if (slot < 0 || slot >= p.num_slots) return;
  const int off = static_cast<int>(slot % kPage);
  const int h0 = blockIdx.x / p.tiles * p.chunk, h1 = min(p.Hkv, h0 + p.chunk);
  for (int h = h0; h < h1; ++h) {
    const int64_t page = slot / kPage * p.Hkv + h;
    const uint8_t* kp = p.k_cache + page * p.k_str;
    const uint8_t* vp = p.v_cache + page * p.v_str;
    uint4 k, v;
    if constexpr (FMT == kBF16) {
      k = *reinterpret_cast<const uint4*>(kp + k_chunk_offset(off, j, 2 * D));
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = *reinterpret_cast<const uint16_t*>(vp + bf16_v_offset(8 * j + 2 * i, off)) |
               static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(vp + bf16_v_offset(8 * j + 2 * i + 1, off))) << 16;
      v = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float ko[8], vo[8];
      if constexpr (F::kFp8) {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w[i >> 2] |= static_cast<uint32_t>(vp[(8 * j + i) * kPage + fp8_v_slot(off)]) << (8 * (i & 3));
        float ks, vs;
        if constexpr (F::kToken) {
          const float* tail = reinterpret_cast<const float*>(vp + kPage * D);
          ks = tail[off];
          vs = tail[kPage + off];
        } else {
          ks = __ldg(p.k_scale + h);
          vs = __ldg(p.v_scale + h);
        }
        value8_fp8<F::kE5>(*reinterpret_cast<const uint2*>(kp + fp8_k_offset(off, j >> 1, D) + (j & 1) * 8), ks, ko);
        value8_fp8<F::kE5>(make_uint2(w[0], w[1]), vs, vo);
      } else {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= static_cast<uint32_t>(vp[fp4_v_offset(off, 4 * j + i)]) << (8 * i);
        value8_fp4(*reinterpret_cast<const uint32_t*>(kp + off * (D / 2) + 4 * j),
                   kp[kPage * D / 2 + off * (D / 16) + j / 2], __ldg(p.k_scale + h), ko);
        value8_fp4(w, vp[kPage * D / 2 + fp4_v_scale_offset(off, j / 2)], __ldg(p.v_scale + h), vo);
      }
      k = pack8_bf16(ko);
      v = pack8_bf16(vo);
    }
    const int64_t at = (static_cast<int64_t>(token) * p.Hkv + h) * D + 8 * j;
    *reinterpret_cast<uint4*>(p.k_out + at) = k;
    *reinterpret_cast<uint4*>(p.v_out + at) = v;
  }
}

template <int FMT>
kvq_status_t launch_gather(GatherParams& p, int D, cudaStream_t s) {
  p.tiles = (p.T - 1) / kPage + 1;
  p.chunk = 1;
  const int64_t ctas = static_cast<int64_t>(p.tiles) * ((p.Hkv + p.chunk - 1) / p.chunk);
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
