// Shared by the decode-step kernels (kv_plan.cu, kv_append.cu,
// kv_attention.cu, logprobs.cu): argument checks and small device helpers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "sm103.cuh"
#include "twell_internal.h"

namespace twell {

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A required device array of n-byte aligned elements.
inline int check_array(const void* p, size_t n) {
  if (!p) return TWELL_ERR_INVALID_ARG;
  return aligned_to(p, n) ? TWELL_OK : TWELL_ERR_MISALIGNED;
}

#define KV_TRY(expr)                 \
  do {                               \
    const int rc_ = (expr);          \
    if (rc_ != TWELL_OK) return rc_; \
  } while (0)

inline bool valid_page_size(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }

// The cache's fields (no device query).
inline int check_kv(const twell_kv_t* c) {
  if (!c) return TWELL_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->n_heads < 1 || c->head_dim < 1 || c->reserved != 0) return TWELL_ERR_INVALID_ARG;
  if (c->format != TWELL_KV_E4M3 && c->format != TWELL_KV_INT8) return TWELL_ERR_INVALID_ARG;
  if (!valid_page_size(c->page_size)) return TWELL_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return TWELL_ERR_UNSUPPORTED;
  KV_TRY(check_array(c->k, 16));
  KV_TRY(check_array(c->v, 16));
  KV_TRY(check_array(c->k_scale, 4));
  KV_TRY(check_array(c->v_scale, 4));
  return check_array(c->status, 4);
}

// A bf16 token matrix [n_tokens][heads][dim] with ld elements between tokens.
inline int check_rows(const void* p, int64_t ld, int heads, int dim) {
  KV_TRY(check_array(p, 16));
  return ld >= static_cast<int64_t>(heads) * dim && ld % 8 == 0 ? TWELL_OK : TWELL_ERR_INVALID_ARG;
}

// The largest i in [0, n) with f(i) <= x, for a non-decreasing f with f(0) <=
// x, found by a whole warp: 32 probes a round, so that a table of 1024 costs
// two dependent loads instead of ten.
template <typename F>
__device__ __forceinline__ int warp_upper(int n, int64_t x, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < len && f(i) <= x;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int last = m ? 31 - __clz(m) : 0;
    lo += last * step;
    len = min(step, len - last * step);
  }
  return lo;
}

}  // namespace twell
