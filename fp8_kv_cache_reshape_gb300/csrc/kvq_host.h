// Host-side helpers shared by the libkvq entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kvq.h"

namespace kvq {

// Record an error message for kvq_last_error_string() and return `st`.
kvq_status_t fail(kvq_status_t st, const char* fmt, ...);
// Clear the calling thread's last error.
void clear_error();
// Map a CUDA error (from a launch) to a status, recording its text.
kvq_status_t cuda_status(cudaError_t e, const char* where);
// Streaming multiprocessors of the current device (cached per device).
int sm_count();
inline bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// The failure-path test hook of kvq_debug_set_stall_ns (0 = off).
uint64_t stall_ns();

// Bytes between the pages of consecutive (block, KV head) pairs in the K and
// the V cache.  Separate caches: a K page and a V page (k_page, v_page bytes).
// Paired layout (v_cache == k_cache + k_page: each pair's K page followed by
// its V page in one allocation): both advance by k_page + v_page.
struct PageStrides {
  int64_t k, v;
  bool paired;
};
inline PageStrides page_strides(const void* k_cache, const void* v_cache, int64_t k_page, int64_t v_page) {
  const bool paired = static_cast<const uint8_t*>(v_cache) == static_cast<const uint8_t*>(k_cache) + k_page;
  return paired ? PageStrides{k_page + v_page, k_page + v_page, true} : PageStrides{k_page, v_page, false};
}

// The split-KV partials of an FP8 decode (per-head scales, no window) without
// their combine: float32 outputs [rows][D] and base-2 log-sum-exps [rows].
// slots > 0: the wide balanced plan (kvq_plan.cuh), a segment (slot, sequence)
// of query head h at ((h * (slots + B - 1) + slot + b) * 4 + warp); slots 0:
// (b * Hq + h) * splits * 4 + i.
struct DecodePartialPlan {
  int slots, splits;
  size_t rows;
  int64_t items;
};
DecodePartialPlan decode_partial_plan(int B, int Hq, int Hkv, int D, int max_blocks);
struct DecodePartialArgs {
  const void* q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t *block_table, *seq_lens;
  float *o_part, *lse_part;
  int B, Hq, Hkv, D, max_blocks;
  int64_t num_blocks;
  float sm_scale;
  bool e5m2;
  bool late;  // launched beside the preceding kernel (programmatic), which it only outlasts (wide plan)
  int* dev_status;
};
kvq_status_t decode_partials(const DecodePartialArgs& a, const DecodePartialPlan& plan, cudaStream_t s);

}  // namespace kvq
