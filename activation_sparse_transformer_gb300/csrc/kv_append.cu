// Keys and values of a step into the 8-bit paged cache (twell_kv_append).
//
// A run is the tokens of one request that fall into one page.  One CTA takes
// one run and some heads of K or of V, one head after the other: it reads the
// run's 2-byte values of a head once into registers (while the head before is being
// encoded), takes their largest magnitude, sets the scale 2^e from its bits and
// writes the codes.  Reads 2 bytes and writes 1 byte per value, so HBM bounds
// long runs; the launch and three dependent latencies (request, slot, values)
// bound single tokens (16 of them 2.8 us), which get a CTA for each head.  The tokens of a run lie ld
// apart, each with 2 D bytes in one piece: 16-byte loads, D / 8 lanes a token.
#include <cuda_bf16.h>

#include "kv_internal.h"

namespace twell {
namespace {

// Threads for a full page's run: four 16-byte loads each, which leaves the registers for
// several CTAs on an SM (pages of 128 tokens: 55.3 us; with 128 threads, eight loads each, 57.5).
constexpr int append_threads(int page, int dim) { return page * dim / 32 < 128 ? 128 : page * dim / 32; }
constexpr int kMinExponent = -100;

struct AppendArgs {
  const uint16_t *k, *v;
  int64_t ldk, ldv;
  uint8_t *k_codes, *v_codes;
  float *k_scale, *v_scale;
  const int32_t* cu_q;
  const int64_t* slots;
  int32_t* status;
  int n_tokens, n_requests, n_pages, heads;
  int heads_per_cta;
};

// Least e with amax <= q 2^e (q = 448 = 1.75 * 2^8 or 127 = 1.984375 * 2^6),
// from the bits of a finite amax >= 0.
template <int FMT>
__device__ __forceinline__ int scale_exponent(float amax) {
  const int bits = __float_as_int(amax);
  const int k = (bits >> 23) - 127, frac = bits & 0x7FFFFF;
  const int e = FMT == TWELL_KV_E4M3 ? k - 8 + (frac > 0x600000) : k - 6 + (frac > 0x7E0000);
  return max(e, kMinExponent);
}

__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }

// Two codes (low byte first) of two values that are already divided by the scale.
template <int FMT>
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  if (FMT == TWELL_KV_E4M3) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
  }
  // 1.5 * 2^23 + x has x rounded to the nearest integer in its low bits
  const uint32_t l = __float_as_uint(lo + 12582912.0f), h = __float_as_uint(hi + 12582912.0f);
  return __byte_perm(l, h, 0x7740) & 0xFFFFu;
}

// Four codes of two words of bf16 pairs times inv, a power of two: the products are
// exact, so that the fused addition rounds to the integer as the separate one does.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(uint32_t w0, uint32_t w1, float inv) {
  const auto fma2 = [](uint32_t w, float m, float c) {  // both halves of a word by one instruction
    uint2 r;
    asm("{\n\t.reg .b64 v, m, c;\n\tmov.b64 v, {%2, %3};\n\tmov.b64 m, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
        "fma.rn.f32x2 v, v, m, c;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(w << 16), "r"(w & 0xFFFF0000u), "f"(m), "f"(c));
    return r;
  };
  if (FMT == TWELL_KV_E4M3) {
    const uint2 a = fma2(w0, inv, -0.0f), b = fma2(w1, inv, -0.0f);
    return encode2<FMT>(__uint_as_float(a.x), __uint_as_float(a.y)) |
           (encode2<FMT>(__uint_as_float(b.x), __uint_as_float(b.y)) << 16);
  }
  const uint2 a = fma2(w0, inv, 12582912.0f), b = fma2(w1, inv, 12582912.0f);
  return __byte_perm(__byte_perm(a.x, a.y, 0x0040), __byte_perm(b.x, b.y, 0x0040), 0x5410);
}

template <int FMT>
__device__ __forceinline__ float2 decode2(uint32_t codes) {
  if (FMT == TWELL_KV_E4M3) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
    float2 f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
  }
  return make_float2(static_cast<float>(static_cast<int8_t>(codes & 0xFF)),
                     static_cast<float>(static_cast<int8_t>((codes >> 8) & 0xFF)));
}

// bf16 bits with an infinity made the largest finite value and a NaN made 0;
// *bad is set when there was one.
__device__ __forceinline__ uint32_t finite2(uint32_t w, bool* bad) {
  const uint32_t lo = w & 0xFFFFu, hi = w >> 16;
  const bool bl = (lo & 0x7F80u) == 0x7F80u, bh = (hi & 0x7F80u) == 0x7F80u;
  if (!(bl || bh)) return w;
  *bad = true;
  const uint32_t l = !bl ? lo : (lo & 0x7Fu) ? 0u : (lo & 0x8000u) | 0x7F7Fu;
  const uint32_t h = !bh ? hi : (hi & 0x7Fu) ? 0u : (hi & 0x8000u) | 0x7F7Fu;
  return l | (h << 16);
}

template <int FMT, int D, int P>
__global__ void __launch_bounds__(append_threads(P, D)) append_kernel(const AppendArgs a) {
  constexpr int kThreads = append_threads(P, D);
  constexpr int kLanes = D / 8;                       // lanes of one token, 8 values each
  constexpr int kRows = kThreads / kLanes;      // tokens of one pass
  constexpr int kPasses = (P + kRows - 1) / kRows;
  __shared__ uint32_t warp_max[2][kThreads / 32];
  grid_dependency_wait();
  const int tid = threadIdx.x;
  // run x of the grid: request r has room for floor(cu[r + 1] / P) -
  // floor(cu[r] / P) + 2 runs, at least as many as its tokens can touch pages
  const int64_t x = blockIdx.x;
  const int r = warp_upper(a.n_requests, x, [&](int i) {
    return static_cast<int64_t>(min(max(a.cu_q[i], 0), a.n_tokens) / P) + 2 * i;
  });
  const int t0 = min(max(a.cu_q[r], 0), a.n_tokens), t1 = min(a.cu_q[r + 1], a.n_tokens);
  const int k = static_cast<int>(x - (t0 / P + 2 * r));
  if (t1 <= t0) return;
  const int64_t slot0 = a.slots[t0];
  if (slot0 < 0) return;
  const int o = static_cast<int>(slot0 % P);
  const int beg = max(t0, t0 + k * P - o), end = min(t1, t0 + (k + 1) * P - o);
  if (beg >= end) return;
  const int64_t slot = a.slots[beg];
  const int64_t page = slot / P;
  const int first = static_cast<int>(slot % P);
  if (slot < 0 || page >= a.n_pages || first + (end - beg) > P) {
    if (tid == 0) report_error(a.status, TWELL_ERR_BAD_FORMAT);
    return;
  }
  const bool is_v = blockIdx.z != 0;
  const int head0 = blockIdx.y * a.heads_per_cta, head1 = min(a.heads, head0 + a.heads_per_cta);
  const int lane_col = (tid % kLanes) * 8, row0 = tid / kLanes;
  const int64_t ld = is_v ? a.ldv : a.ldk;
  const uint16_t* const src = (is_v ? a.v : a.k) + beg * ld + lane_col;
  float* const scales = (is_v ? a.v_scale : a.k_scale) + page * a.heads;
  uint8_t* const codes = (is_v ? a.v_codes : a.k_codes) + page * a.heads * (P * D);
  const int n = end - beg;
  const auto load = [&](int head, uint4 (&w)[kPasses]) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int t = row0 + i * kRows;
      w[i] = t < n ? __ldg(reinterpret_cast<const uint4*>(src + t * ld + static_cast<int64_t>(head) * D))
                   : make_uint4(0, 0, 0, 0);
    }
  };
  uint4 next[kPasses];
  load(head0, next);
  float next_was = first > 0 ? scales[head0] : 0.0f;
  for (int head = head0; head < head1; ++head) {
    uint4 w[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) w[i] = next[i];
    const float was = next_was;
    if (head + 1 < head1) {
      load(head + 1, next);
      if (first > 0) next_was = scales[head + 1];
    }
    // the largest magnitude by the bits, which order as the magnitudes do, two at a time
    uint32_t both = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t* q = &w[i].x;
#pragma unroll
      for (int j = 0; j < 4; ++j) both = __vmaxu2(both, q[j] & 0x7FFF7FFFu);
    }
    if (max(both & 0xFFFFu, both >> 16) >= 0x7F80u) {  // an infinity or a NaN: rare
      bool bad = false;
      both = 0;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        uint32_t* q = &w[i].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          q[j] = finite2(q[j], &bad);
          both = __vmaxu2(both, q[j] & 0x7FFF7FFFu);
        }
      }
      report_error(a.status, TWELL_ERR_NOT_FINITE);
    }
    uint32_t most = __reduce_max_sync(0xffffffffu, max(both & 0xFFFFu, both >> 16));
    uint32_t* const maxima = warp_max[(head - head0) & 1];  // two, so that one barrier a head is enough
    if ((tid & 31) == 0) maxima[tid / 32] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) most = max(most, maxima[i]);
    const float amax = __uint_as_float(most << 16);
    const float scale = fmaxf(two_to(scale_exponent<FMT>(amax)), was);
    uint8_t* const dst = codes + static_cast<int64_t>(head) * (P * D);
    // earlier tokens of the page move to the larger scale
    if (first > 0 && scale > was) {
      const float ratio = was / scale;
      for (int t = row0; t < first; t += kRows) {
        uint2* at = reinterpret_cast<uint2*>(dst + t * D + lane_col);
        uint2 c = *at;
        uint32_t* q = &c.x;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 lo = decode2<FMT>(q[j] & 0xFFFFu), hi = decode2<FMT>(q[j] >> 16);
          q[j] = encode2<FMT>(lo.x * ratio, lo.y * ratio) | (encode2<FMT>(hi.x * ratio, hi.y * ratio) << 16);
        }
        *at = c;
      }
    }
    // 1 / scale is exact for a power of two; another scale (a cache written by
    // someone else) divides
    const bool pow2 = (__float_as_uint(scale) & 0x7FFFFFu) == 0;
    const float inv = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int t = row0 + i * kRows;
      if (t >= n) continue;
      const uint32_t* q = &w[i].x;
      uint2 c;
      if (pow2) {
        c = make_uint2(encode4<FMT>(q[0], q[1], inv), encode4<FMT>(q[2], q[3], inv));
      } else {
        const auto divided = [&](uint32_t v) { return encode2<FMT>(bf16_lo(v) / scale, bf16_hi(v) / scale); };
        c = make_uint2(divided(q[0]) | (divided(q[1]) << 16), divided(q[2]) | (divided(q[3]) << 16));
      }
      *reinterpret_cast<uint2*>(dst + (first + t) * D + lane_col) = c;
    }
    if (tid == 0 && scale != was) scales[head] = scale;
  }
}

template <int FMT, int D>
int launch_append(AppendArgs a, int page, cudaStream_t s) {
  // heads one after the other, a head's loads under the encoding of the one before, once every SM has CTAs enough:
  // 24 prompts of up to 4000 tokens, 8 heads of 128, int8: 55.4 us (6.1 TB/s); with a
  // CTA for each head 70, with twice as many CTAs 55.7 (pages of 64: 56.7 and 59.6)
  const int64_t runs = a.n_tokens / page + 2 * static_cast<int64_t>(a.n_requests);
  while (a.heads_per_cta < a.heads && runs * 2 * (a.heads / (2 * a.heads_per_cta)) >= 6 * sm_count())
    a.heads_per_cta *= 2;
  const dim3 grid(static_cast<unsigned>(runs),
                  static_cast<unsigned>((a.heads + a.heads_per_cta - 1) / a.heads_per_cta), 2);
  LaunchScope scope(TWELL_KERNEL_KV_APPEND, s);
  cudaError_t e = cudaErrorInvalidValue;
  switch (page) {
    case 16: e = launch_pdl(append_kernel<FMT, D, 16>, grid, dim3(append_threads(16, D)), 0, s, a); break;
    case 32: e = launch_pdl(append_kernel<FMT, D, 32>, grid, dim3(append_threads(32, D)), 0, s, a); break;
    case 64: e = launch_pdl(append_kernel<FMT, D, 64>, grid, dim3(append_threads(64, D)), 0, s, a); break;
    case 128: e = launch_pdl(append_kernel<FMT, D, 128>, grid, dim3(append_threads(128, D)), 0, s, a); break;
  }
  return e == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

}  // namespace
}  // namespace twell

using namespace twell;

extern "C" TWELL_API int twell_kv_append(const uint16_t* K, int64_t ldk, const uint16_t* V, int64_t ldv,
                                         const int32_t* cu_q, const int64_t* slots, int32_t n_tokens,
                                         int32_t n_requests, const twell_kv_t* cache, twell_stream_t stream) {
  KV_TRY(check_kv(cache));
  if (n_tokens < 0 || n_requests < 0) return TWELL_ERR_INVALID_ARG;
  if (n_tokens > 0 && n_requests > 0) {
    KV_TRY(check_rows(K, ldk, cache->n_heads, cache->head_dim));
    KV_TRY(check_rows(V, ldv, cache->n_heads, cache->head_dim));
    KV_TRY(check_array(cu_q, 4));
    KV_TRY(check_array(slots, 8));
    if (cache->n_heads > 65535) return TWELL_ERR_UNSUPPORTED;
    // the grid's runs: 2 a request and one more for every page of tokens
    if (n_tokens / cache->page_size + 2 * static_cast<int64_t>(n_requests) > INT32_MAX) return TWELL_ERR_UNSUPPORTED;
  }
  if (!device_is_sm103()) return TWELL_ERR_NO_DEVICE;
  if (n_tokens == 0 || n_requests == 0) return TWELL_OK;
  const AppendArgs a{K, V, ldk, ldv, cache->k, cache->v, cache->k_scale, cache->v_scale, cu_q, slots,
                     cache->status, n_tokens, n_requests, cache->n_pages, cache->n_heads, 1};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cache->format == TWELL_KV_E4M3)
    return cache->head_dim == 64 ? launch_append<TWELL_KV_E4M3, 64>(a, cache->page_size, s)
                                 : launch_append<TWELL_KV_E4M3, 128>(a, cache->page_size, s);
  return cache->head_dim == 64 ? launch_append<TWELL_KV_INT8, 64>(a, cache->page_size, s)
                               : launch_append<TWELL_KV_INT8, 128>(a, cache->page_size, s);
}

extern "C" TWELL_API int twell_kv_read_status(const twell_kv_t* cache, twell_stream_t stream) {
  if (!cache || !cache->status) return TWELL_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return TWELL_ERR_CUDA;
  int32_t st = 0;
  if (cudaMemcpy(&st, cache->status, sizeof st, cudaMemcpyDeviceToHost) != cudaSuccess) return TWELL_ERR_CUDA;
  return st;
}
