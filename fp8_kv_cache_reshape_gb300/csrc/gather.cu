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

// Bytes between the token rows of a page in shared memory: those that a thread
// writes together, and the two halves of a BF16 page, fall into different banks.
template <int D, int FMT>
constexpr int kRowStride = FMT == kBF16 ? 2 * D + 8 : (FMT == kFP4 ? D / 2 : D) + 16;

// What a thread brings of a V page: four words of four (FP8, FP4) or eight
// tokens (BF16: two 16-byte rows), and where they go.
template <int D, int FMT>
struct VPart {
  static constexpr int kThreads = FMT == kFP4 ? D / 2 : D;  // that take part
  uint32_t w[FMT == kBF16 ? 8 : 4];

  KVQ_DEVINL void load(const uint8_t* vp, int x) {
    if (x >= kThreads) return;
    if constexpr (FMT == kBF16) {
      const int half = x & 1, d = x & ~1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 u = *reinterpret_cast<const uint4*>(vp + bf16_v_offset(d + i, 8 * half));
        w[4 * i] = u.x;
        w[4 * i + 1] = u.y;
        w[4 * i + 2] = u.z;
        w[4 * i + 3] = u.w;
      }
    } else {
      int at, step;
      if constexpr (FMT == kFP4) {
        at = (x >> 5) * 512 + ((x >> 4) & 1) * 256 + ((x >> 2) & 3) * 16 + (x & 3) * 4;
        step = 64;
      } else {
        at = (x & ~3) * kPage + (x & 3) * 4;
        step = kPage;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(vp + at + i * step);
    }
  }
  KVQ_DEVINL void store(uint8_t* rows, int x) const {
    constexpr int S = kRowStride<D, FMT>;
    if (x >= kThreads) return;
    if constexpr (FMT == kBF16) {
      const int half = x & 1, d = x & ~1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // tokens 8 half + 2i, + 1: dims d, d + 1
        *reinterpret_cast<uint32_t*>(rows + (8 * half + 2 * i) * S + 2 * d) = __byte_perm(w[i], w[4 + i], 0x5410);
        *reinterpret_cast<uint32_t*>(rows + (8 * half + 2 * i + 1) * S + 2 * d) = __byte_perm(w[i], w[4 + i], 0x7632);
      }
    } else {
      const int c = FMT == kFP4 ? (x >> 2) & 3 : x & 3;
      const int col = FMT == kFP4 ? 32 * (x >> 5) + 8 * (x & 3) + 4 * ((x >> 4) & 1) : x & ~3;
      uint32_t o[4];
      transpose4(w, o);  // a word's bytes are tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(rows + (2 * c + (i & 1) + 8 * (i >> 1)) * S + col) = o[i];
    }
  }
};

// What a thread brings of its own token: eight dims of K and their scales.
template <int D, int FMT>
struct KPart {
  uint4 k;
  float ks, vs;

  KVQ_DEVINL void load(const GatherParams& p, const uint8_t* kp, const uint8_t* vp, int off, int j, int h) {
    if constexpr (FMT == kBF16) {
      k = *reinterpret_cast<const uint4*>(kp + k_chunk_offset(off, j, 2 * D));
    } else if constexpr (FMT == kFP4) {
      k.x = *reinterpret_cast<const uint32_t*>(kp + off * (D / 2) + 4 * j);
      k.y = kp[kPage * D / 2 + off * (D / 16) + j / 2];
      k.z = vp[kPage * D / 2 + fp4_v_scale_offset(off, j / 2)];
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(kp + fp8_k_offset(off, j >> 1, D) + (j & 1) * 8);
      k.x = u.x;
      k.y = u.y;
    }
    if constexpr (Format<FMT>::kToken) {
      const float* tail = reinterpret_cast<const float*>(vp + kPage * D);
      ks = tail[off];
      vs = tail[kPage + off];
    } else if constexpr (FMT != kBF16) {
      ks = __ldg(p.k_scale + h);
      vs = __ldg(p.v_scale + h);
    }
  }
};

// One thread's eight dims of V of a token, from the page itself.
template <int D, int FMT>
KVQ_DEVINL uint4 v_of_page(const uint8_t* vp, int off, int j) {
  uint32_t w[4] = {0, 0, 0, 0};
  if constexpr (FMT == kBF16) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i >> 1] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(vp + bf16_v_offset(8 * j + i, off))) << (16 * (i & 1));
  } else if constexpr (FMT == kFP4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[0] |= static_cast<uint32_t>(vp[fp4_v_offset(off, 4 * j + i)]) << (8 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i >> 2] |= static_cast<uint32_t>(vp[(8 * j + i) * kPage + fp8_v_slot(off)]) << (8 * (i & 3));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// ... and from the page's token rows in shared memory.
template <int D, int FMT>
KVQ_DEVINL uint4 v_of_rows(const uint8_t* rows, int off, int j) {
  const uint8_t* at = rows + off * kRowStride<D, FMT>;
  uint4 v = make_uint4(0, 0, 0, 0);
  if constexpr (FMT == kFP4) {
    v.x = *reinterpret_cast<const uint32_t*>(at + 4 * j);
  } else {
    const uint2* u = reinterpret_cast<const uint2*>(at + (FMT == kBF16 ? 16 : 8) * j);
    v.x = u[0].x;
    v.y = u[0].y;
    if constexpr (FMT == kBF16) {
      v.z = u[1].x;
      v.w = u[1].y;
    }
  }
  return v;
}

// A tile's tokens, a chunk of heads; a thread holds dims 8 j .. 8 j + 7 of a
// token.  Where the tokens fill a page in order, its V part comes in whole words that are
// transposed in registers and meet in shared memory; the next head's loads are
// in flight meanwhile.
template <int D, int FMT>
__global__ void __launch_bounds__(kPage * D / 8) gather_kernel(const GatherParams p) {
  using F = Format<FMT>;
  constexpr int LPT = D / 8;
  __shared__ TileTokens tt;
  __shared__ __align__(16) uint8_t rows[2][kPage * kRowStride<D, FMT>];
  const int x = threadIdx.x, t = x / LPT, j = x % LPT;
  const int tile = blockIdx.x % p.tiles;
  const int h0 = blockIdx.x / p.tiles * p.chunk, h1 = min(p.Hkv, h0 + p.chunk);
  if (x < 32) find_tokens(tt, p.slots, p.T, p.num_slots, tile, p.aligned, p.dev_status);
  __syncthreads();
  const int n = tt.n;
  for (int r = 0; r < n; r += kPage) {
    const bool valid = r + t < n, page_run = tt.page[r / kPage];
    const int token = tt.token[valid ? r + t : r];
    const int64_t slot = tt.slot[valid ? r + t : r];
    const int off = static_cast<int>(slot % kPage);
    const int64_t page = slot / kPage * p.Hkv + h0;
    const uint8_t* kp = p.k_cache + page * p.k_str;
    const uint8_t* vp = p.v_cache + page * p.v_str;
    KPart<D, FMT> k;
    VPart<D, FMT> part;
    k.load(p, kp, vp, off, j, h0);
    if (page_run) part.load(vp, x);
    for (int h = h0; h < h1; ++h) {
      const KPart<D, FMT> now = k;
      uint4 v;
      if (page_run) {
        uint8_t* buf = rows[(h - h0) & 1];  // the other one is read no longer when it is written again, a barrier later
        part.store(buf, x);
        if (h + 1 < h1) part.load(vp + p.v_str, x);
      } else {
        v = v_of_page<D, FMT>(vp, off, j);
      }
      kp += p.k_str;
      vp += p.v_str;
      if (h + 1 < h1) k.load(p, kp, vp, off, j, h + 1);
      if (page_run) {
        __syncthreads();
        v = v_of_rows<D, FMT>(rows[(h - h0) & 1], off, j);
      }
      if (!valid) continue;
      uint4 ko = now.k;
      if constexpr (FMT != kBF16) {
        float2 kf[4], vf[4];
        if constexpr (FMT == kFP4) {
          value8_fp4(now.k.x, static_cast<uint8_t>(now.k.y), now.ks, kf);
          value8_fp4(v.x, static_cast<uint8_t>(now.k.z), now.vs, vf);
        } else {
          value8_fp8<F::kE5>(make_uint2(now.k.x, now.k.y), now.ks, kf);
          value8_fp8<F::kE5>(make_uint2(v.x, v.y), now.vs, vf);
        }
        ko = pack8_bf16(kf);
        v = pack8_bf16(vf);
      }
      const int64_t at = (static_cast<int64_t>(token) * p.Hkv + h) * D + 8 * j;
      *reinterpret_cast<uint4*>(p.k_out + at) = ko;
      *reinterpret_cast<uint4*>(p.v_out + at) = v;
    }
    if (page_run) __syncthreads();  // the next 16 tokens start with the first buffer again
  }
}

template <int FMT>
kvq_status_t launch_gather(GatherParams& p, int D, cudaStream_t s) {
  p.aligned = p.T >= KVQ_TUNE(galign, 64);
  p.tiles = (p.T - 1) / kPage + 1 + (p.aligned ? 1 : 0);
  p.chunk = heads_per_cta(p.Hkv, p.tiles, KVQ_TUNE(gmost, 8), KVQ_TUNE(gctas, 8) * sm_count());
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
