// What the kernels that move tokens between rows and the paged cache share:
// eight dims of a token per lane, their quantization and the page formats
// (include/kvq.h).
#pragma once

#include <cuda_fp4.h>

#include "kvq_device.cuh"

namespace kvq {

// The formats of a cache, one kernel instantiation each.
enum CacheFormat { kRowsOnly, kE4M3, kE5M2, kBF16, kFP4, kE4M3Token, kE5M2Token };

template <int FMT>
struct Format {
  static constexpr bool kFp8 = FMT == kE4M3 || FMT == kE5M2 || FMT == kE4M3Token || FMT == kE5M2Token;
  static constexpr bool kE5 = FMT == kE5M2 || FMT == kE5M2Token;
  static constexpr bool kToken = FMT == kE4M3Token || FMT == kE5M2Token;
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

KVQ_DEVINL void unpack8_bf16(const uint4& a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
KVQ_DEVINL uint4 pack8_bf16(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
// fp8(fl32(x / s)) of eight values.
template <bool E5>
KVQ_DEVINL uint2 quant8_fp8(const float (&x)[8], float s) {
  constexpr auto kind = E5 ? __NV_E5M2 : __NV_E4M3;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s)), __NV_SATFINITE, kind);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}
KVQ_DEVINL float amax8(const float (&x)[8]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
  return a;
}
KVQ_DEVINL float e4m3_value(uint8_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}
// The E4M3 scale of a block of 16 dims, of which two neighbouring lanes hold
// eight each, and their E2M1 codes.  s: the head's scale.
KVQ_DEVINL uint32_t quant8_fp4(const float (&x)[8], float s, uint8_t& block_scale) {
  float a = amax8(x);
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
  block_scale = f32_to_e4m3(__fdiv_rn(a, __fmul_rn(6.f, s)));
  const float step = __fmul_rn(e4m3_value(block_scale), s);
  uint32_t w = 0;
  if (step > 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(__fdiv_rn(x[2 * i], step), __fdiv_rn(x[2 * i + 1], step)),
                                                          __NV_E2M1, cudaRoundNearest)) << (8 * i);
  }
  return w;
}

}  // namespace kvq
