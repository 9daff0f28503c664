// Shared by the two kernels of the attention over the 8-bit cache
// (kv_attention.cu: few rows a request; kv_chunk.cu: many).
#pragma once

#include "kv_internal.h"

namespace twell {

struct AttArgs {
  const uint16_t* q;
  int64_t ldq;
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  const int32_t *block_table, *cu_q, *positions, *kv_lens;
  uint16_t* o;
  int64_t ldo;
  float* lse;
  int32_t* status;
  int max_blocks, n_tokens, n_requests, q_heads, heads, group, page_shift, n_pages;
  float scale_log2;  // softmax_scale * log2(e)
  int chunk_rows;    // requests of more rows than this go to chunk_attention
  int stall;         // self-test: arrivals that a barrier of each CTA's copies waits for in vain (else 0)
  uint64_t wait_ns;  // limit of each wait
};

// Requests of more than this many rows (tokens times query heads of a key head)
// fill tcgen05's 128 rows well enough to pay for the fp16 copy of the cache
// that its operands need; a.chunk_rows is this, or INT32_MAX when no request is that large.
constexpr int kChunkRows = 64;
// After an expired wait: how long a CTA waits for its own copies in flight before it leaves.
constexpr uint64_t kDrainNs = 10000000ull;
int launch_chunk_attention(const AttArgs& a, int format, int dim, int max_kv_len, void* workspace, cudaStream_t s);
size_t chunk_workspace_bytes(int64_t rows, int dim);  // for so many rows in all

// Weights are 2^(l - n) in fp16.  A row's reference n stands kRoom below the largest l that it was
// set by, and moves when an l passes that one by kLazy: the largest weights lie between 2^kRoom and
// 2^(kRoom + kLazy) = 2^15, below fp16's 65504, and a weight is off by 2^-32 of the largest at most where fp16
// cannot hold it to 2^-11 of itself (below 2^-21 of the largest; with n at the largest l 2^-25, which over
// 131072 tokens came to 2^-8 of the result).  The sums of weights are taken without the factor 2^kRoom.
constexpr float kLazy = 8.0f, kRoom = 7.0f, kUnroom = 1.0f / 128;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four codes of one word to two fp16 pairs: (byte 0, byte 1) and (byte 2, byte 3).
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& p01, uint32_t& p23) {
  if (FMT == TWELL_KV_E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(p01), "=r"(p23)
        : "r"(w));
  } else {
    // 0x6400 | u is the fp16 number 1024 + u: with u = code + 128, minus 1152
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p01) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p23) : "r"(b), "r"(0x64806480u));
  }
}

// Bits where a byte of w is e4m3's NaN, 0x7F or 0xFF.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// log2 of a value scale.  Always a number: a page that a row does not see may have any
// scale, and a masked -inf has to stay so when it is added.
__device__ __forceinline__ float log2_scale(float vs) { return fminf(fmaxf(log2_fast(vs), -200.0f), 200.0f); }

__device__ __forceinline__ int visible_len(const AttArgs& a, int r) {
  const int64_t room = static_cast<int64_t>(a.max_blocks) << a.page_shift;
  return static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(a.kv_lens[r]), room)));
}

struct Request {
  int t0, n_rows, len;
};

__device__ __forceinline__ Request request(const AttArgs& a, int r) {
  const int t0 = min(max(a.cu_q[r], 0), a.n_tokens), t1 = min(max(a.cu_q[r + 1], t0), a.n_tokens);
  return {t0, (t1 - t0) * a.group, visible_len(a, r)};
}

// Eight dims of one finished row: o / sum, rounded once, and the row's lse.  o has the
// weights' factor 2^kRoom, sum has not.  n = -inf: the row has seen nothing.
template <int D>
__device__ __forceinline__ void store_row(const AttArgs& a, int t0, int row, int head, int d0, float n, float sum,
                                          const float (&o)[8]) {
  const bool seen = n > -INFINITY;
  const float f = seen ? kUnroom / sum : 0.0f;
  const int64_t token = t0 + row / a.group;
  const int h = head * a.group + row % a.group;
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = static_cast<uint32_t>(float_to_bf16_bits(o[2 * i] * f)) |
             (static_cast<uint32_t>(float_to_bf16_bits(o[2 * i + 1] * f)) << 16);
  *reinterpret_cast<uint4*>(a.o + token * a.ldo + static_cast<int64_t>(h) * D + d0) =
      make_uint4(out[0], out[1], out[2], out[3]);
  if (a.lse && d0 == 0) a.lse[token * a.q_heads + h] = seen ? (n + kRoom + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace twell
