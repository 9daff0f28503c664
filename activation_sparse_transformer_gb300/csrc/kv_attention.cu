// Attention over the 8-bit paged cache (twell_kv_attention).
//
// For token t of request r and query head h (key / value head h / G):
//   x_j = c q . k_j,  o = sum_j exp(x_j) v_j / sum_j exp(x_j),  j < L
// with k_j = s_k code, v_j = s_v code, one scale per page and head.  The rows
// (token, query head) of one request that share a key / value head form the
// 16 rows of an mma tile, so each cached byte is read once for all of them.
// Per 16 cached tokens a warp computes
//   S = Q K^T                 fp16 x fp16 -> fp32, codes exact in fp16
//   l = S (c log2(e) 2^k s_k) (2^k: the row's own factor, see load_q)
//   p = 2^(l - m),  w = p s_v 2^-n  ->  fp16,  O += w V
// in one pass with running references: m follows the largest l and n the
// largest l + log2 s_v, both per row, so that neither the sum of p nor the
// fp16 weights leave their range whatever the pages' scales are.
//
// The reduction index of an mma may be permuted as long as both operands
// agree, and so may the columns of its result.  K's lanes therefore take 16
// consecutive bytes of one token (two loads for D = 128) and Q is gathered to
// match; V's lanes take the same 16 (D = 128) or 8 bytes of four tokens, whose
// bytes are paired to fp16 registers, and the output columns come out in runs.
// No transposition and no shared memory lies between the cache and the mma.
#include "kv_internal.h"

namespace twell {
namespace {

constexpr int kAttWarps = 4;
constexpr int kAttThreads = 32 * kAttWarps;
constexpr int kAttRows = 16;    // rows of a tile
constexpr int kAttGroup = 16;   // cached tokens of one warp step, all of one page
constexpr int kAttMaxRequests = 4096;
// The references m and n are moved only when a new value passes them by this
// much (as powers of two): weights up to 2^8 stay well inside fp16.
constexpr float kLazy = 8.0f;

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
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

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

// One tile's running state in a warp: rows g = lane / 4 and g + 8.
template <int D>
struct TileState {
  float acc[D / 8][4];   // n-tile i: dims (D / 8) * 2q + i and (D / 8) * (2q + 1) + i of both rows
  float m[2], n[2], sum[2];
};

template <int D>
__device__ __forceinline__ void reset(TileState<D>& s) {
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s.acc[i][j] = 0.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s.m[i] = s.n[i] = -INFINITY;
    s.sum[i] = 0.0f;
  }
}

// Rows of the tile as fp16 fragments.  A row enters as q 2^-k with its largest
// magnitude in [1, 2): exact in fp16 for components above 2^-14 and off by at
// most 2^-25 below, which is less than the fp32 sum's own rounding.  factor
// returns c log2(e) 2^k.
template <int D>
__device__ __forceinline__ void load_q(const AttArgs& a, int64_t t0, int n_rows, int row0, int head,
                                       uint32_t (&qa)[D / 16][4], float (&factor)[2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = row0 + g + 8 * half;
    const bool on = row < n_rows;
    const int token = row / a.group;
    const uint16_t* src = a.q + (t0 + token) * a.ldq + (static_cast<int64_t>(head) * a.group + row % a.group) * D;
    uint4 w[D / 32];  // 16 dims each D / 64: two uint4
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[2 * i + j] = on ? __ldg(reinterpret_cast<const uint4*>(src + 64 * i + 16 * quad + 8 * j))
                          : make_uint4(0, 0, 0, 0);
    const uint32_t* u = &w[0].x;
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(u[i])), fabsf(bf16_hi(u[i]))));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int k = min(max((__float_as_int(amax) >> 23) - 127, -126), 126);
    const float inv = __int_as_float((127 - k) << 23);
    factor[half] = a.scale_log2 * __int_as_float((127 + k) << 23);
    // word i of the 16-byte code vector holds dims 4 i .. 4 i + 3 = u[2 i], u[2 i + 1]
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        qa[j][half + 2 * p] = pack_f16(bf16_lo(u[2 * j + p]) * inv, bf16_hi(u[2 * j + p]) * inv);
  }
}

// One warp step: 16 cached tokens [j0, j0 + 16) whose codes are in kw and vw.
// limit: tokens each row sees; mask: some row sees not all of the 16.
template <int FMT, int D>
__device__ __forceinline__ void step16(TileState<D>& s, const uint32_t (&qa)[D / 16][4], const float (&factor)[2],
                                       const uint32_t (&kw)[2][D / 16], const uint32_t (&vw)[4][D / 32], float ks,
                                       float vs, int j0, const int (&limit)[2], bool mask) {
  const int quad = threadIdx.x & 3;
  float x[2][4] = {};
#pragma unroll
  for (int j = 0; j < D / 16; ++j)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      uint32_t b0, b1;
      codes_to_f16<FMT>(kw[nt][j], b0, b1);
      mma_f16(x[nt], qa[j], b0, b1);
    }
  const float lvs = fmaxf(log2_fast(vs), -200.0f);  // a scale of zero stands for zeros
  float top[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float f = factor[half] * ks;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float& v = x[nt][2 * half + c];
        v *= f;
        if (mask && j0 + nt * 8 + 2 * quad + c >= limit[half]) v = -INFINITY;
      }
    top[half] = fmaxf(fmaxf(x[0][2 * half], x[0][2 * half + 1]), fmaxf(x[1][2 * half], x[1][2 * half + 1]));
    top[half] = fmaxf(top[half], __shfl_xor_sync(0xffffffffu, top[half], 1));
    top[half] = fmaxf(top[half], __shfl_xor_sync(0xffffffffu, top[half], 2));
  }
  const bool move = top[0] > s.m[0] + kLazy || top[1] > s.m[1] + kLazy || top[0] + lvs > s.n[0] + kLazy ||
                    top[1] + lvs > s.n[1] + kLazy;
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float m = fmaxf(s.m[half], top[half]), n = fmaxf(s.n[half], top[half] + lvs);
      // a row that has seen nothing yet keeps sums of zero: no factor of inf - inf
      if (m > -INFINITY) s.sum[half] *= exp2_fast(s.m[half] - m);
      const float f = n > -INFINITY ? exp2_fast(s.n[half] - n) : 1.0f;
      s.m[half] = m;
      s.n[half] = n;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        s.acc[i][2 * half] *= f;
        s.acc[i][2 * half + 1] *= f;
      }
    }
  }
  uint32_t pa[4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float m = s.m[half] > -INFINITY ? s.m[half] : 0.0f;
    const float n = s.n[half] > -INFINITY ? s.n[half] : 0.0f;
    const float c = exp2_fast(fminf(m + lvs - n, 100.0f));
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const float p0 = exp2_fast(x[nt][2 * half] - m), p1 = exp2_fast(x[nt][2 * half + 1] - m);
      s.sum[half] += p0 + p1;
      pa[half + 2 * nt] = pack_f16(p0 * c, p1 * c);
    }
  }
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    // bytes of two neighbouring tokens side by side, then to fp16 pairs
    uint32_t b0[4], b1[4];
    codes_to_f16<FMT>(__byte_perm(vw[0][w], vw[1][w], 0x5140), b0[0], b0[1]);
    codes_to_f16<FMT>(__byte_perm(vw[0][w], vw[1][w], 0x7362), b0[2], b0[3]);
    codes_to_f16<FMT>(__byte_perm(vw[2][w], vw[3][w], 0x5140), b1[0], b1[1]);
    codes_to_f16<FMT>(__byte_perm(vw[2][w], vw[3][w], 0x7362), b1[2], b1[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) mma_f16(s.acc[4 * w + i], pa, b0[i], b1[i]);
  }
}

template <int D>
__device__ __forceinline__ void zero_row(const AttArgs& a, int64_t t, int tid, int n_threads) {
  for (int i = tid; i < a.q_heads * (D / 8); i += n_threads)
    *reinterpret_cast<uint4*>(a.o + t * a.ldo + i * 8) = make_uint4(0, 0, 0, 0);
  if (a.lse)
    for (int i = tid; i < a.q_heads; i += n_threads) a.lse[t * a.q_heads + i] = -INFINITY;
}

template <int FMT, int D>
__global__ void __launch_bounds__(kAttThreads) attention_kernel(const AttArgs a) {
  __shared__ float sh_o[kAttWarps][kAttRows][D + 4];
  __shared__ float sh_m[kAttWarps][kAttRows], sh_n[kAttWarps][kAttRows], sh_sum[kAttWarps][kAttRows];
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, quad = lane & 3;
  const int head = blockIdx.y;
  // row blocks: request r has room for floor(cu[r + 1] G / 16) - floor(cu[r] G / 16) + 1
  const int64_t x = blockIdx.x;
  const auto first_block = [&](int i) {
    return static_cast<int64_t>(min(max(a.cu_q[i], 0), a.n_tokens)) * a.group / kAttRows + i;
  };
  const int r = warp_upper(a.n_requests, x, first_block);
  const int t0 = min(max(a.cu_q[r], 0), a.n_tokens), t1 = min(max(a.cu_q[r + 1], t0), a.n_tokens);
  const int n_rows = (t1 - t0) * a.group, row0 = static_cast<int>(x - first_block(r)) * kAttRows;
  if (row0 >= n_rows) return;
  const int len = min(a.kv_lens[r], static_cast<int>(min(static_cast<int64_t>(a.max_blocks) << a.page_shift,
                                                         static_cast<int64_t>(INT32_MAX))));
  // what each row sees; rows past the last see everything and are not stored
  int limit[2], most = 0, least = INT32_MAX;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = row0 + g + 8 * half;
    limit[half] = INT32_MAX;
    if (row < n_rows) {
      const int pos = a.positions[t0 + row / a.group];
      limit[half] = max(0, min(pos < INT32_MAX ? pos + 1 : pos, len));
      most = max(most, limit[half]);
      least = min(least, limit[half]);
    }
  }
#pragma unroll
  for (int d = 16; d >= 4; d /= 2) {
    most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
    least = min(least, __shfl_xor_sync(0xffffffffu, least, d));
  }
  uint32_t qa[D / 16][4];
  float factor[2];
  load_q<D>(a, t0, n_rows, row0, head, qa, factor);
  TileState<D> s;
  reset(s);
  const int page_mask = (1 << a.page_shift) - 1;
  for (int j0 = warp * kAttGroup; j0 < most; j0 += kAttWarps * kAttGroup) {
    int page = a.block_table[static_cast<int64_t>(r) * a.max_blocks + (j0 >> a.page_shift)];
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.n_pages)) {
      if (lane == 0) report_error(a.status, TWELL_ERR_BAD_FORMAT);
      page = 0;
    }
    const int64_t cell = static_cast<int64_t>(page) * a.heads + head;
    const int64_t at = ((cell << a.page_shift) + (j0 & page_mask)) * D;
    const float ks = a.k_scale[cell], vs = a.v_scale[cell];
    uint32_t kw[2][D / 16], vw[4][D / 32];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        *reinterpret_cast<uint4*>(&kw[nt][4 * i]) =
            __ldg(reinterpret_cast<const uint4*>(a.k + at + (nt * 8 + g) * D + 64 * i + 16 * quad));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int token = (i >> 1) * 8 + 2 * quad + (i & 1);
      const uint8_t* src = a.v + at + token * D + (D / 8) * g;
      // a token nobody sees may hold anything, and 0 * NaN is not 0
      const bool seen = j0 + token < most;
      if constexpr (D == 128) {
        *reinterpret_cast<uint4*>(vw[i]) =
            seen ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
      } else {
        *reinterpret_cast<uint2*>(vw[i]) = seen ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0, 0);
      }
    }
    step16<FMT, D>(s, qa, factor, kw, vw, ks, vs, j0, limit, j0 + kAttGroup > least);
  }
  // the four warps' results of the tile, joined in warp order
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    s.sum[half] += __shfl_xor_sync(0xffffffffu, s.sum[half], 1);
    s.sum[half] += __shfl_xor_sync(0xffffffffu, s.sum[half], 2);
    const int row = g + 8 * half;
    if (quad == 0) {
      sh_m[warp][row] = s.m[half];
      sh_n[warp][row] = s.n[half];
      sh_sum[warp][row] = s.sum[half];
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      sh_o[warp][row][(D / 8) * (2 * quad) + i] = s.acc[i][2 * half];
      sh_o[warp][row][(D / 8) * (2 * quad + 1) + i] = s.acc[i][2 * half + 1];
    }
  }
  __syncthreads();
  constexpr int kLanes = D / 8;
  for (int row = tid / kLanes; row < min(kAttRows, n_rows - row0); row += kAttThreads / kLanes) {
    const int d0 = (tid % kLanes) * 8;
    float m = -INFINITY, n = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) {
      m = fmaxf(m, sh_m[w][row]);
      n = fmaxf(n, sh_n[w][row]);
    }
    float sum = 0.0f, o[8] = {};
    if (m > -INFINITY) {
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) {
        sum += sh_sum[w][row] * exp2_fast(sh_m[w][row] - m);
        const float f = exp2_fast(sh_n[w][row] - n);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += sh_o[w][row][d0 + i] * f;
      }
    }
    const float f = m > -INFINITY ? exp2_fast(n - m) / sum : 0.0f;
    const int grow = row0 + row, token = grow / a.group, h = head * a.group + grow % a.group;
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      out[i] = static_cast<uint32_t>(float_to_bf16_bits(o[2 * i] * f)) |
               (static_cast<uint32_t>(float_to_bf16_bits(o[2 * i + 1] * f)) << 16);
    *reinterpret_cast<uint4*>(a.o + (t0 + token) * a.ldo + static_cast<int64_t>(h) * D + d0) =
        make_uint4(out[0], out[1], out[2], out[3]);
    if (a.lse && d0 == 0)
      a.lse[static_cast<int64_t>(t0 + token) * a.q_heads + h] =
          m > -INFINITY ? (m + log2f(sum)) * 0.69314718055994531f : -INFINITY;
  }
}

template <int D>
__global__ void __launch_bounds__(kAttThreads) attention_rest_kernel(const AttArgs a) {
  grid_dependency_wait();
  // tokens of no request
  const int beg = min(max(a.cu_q[a.n_requests], 0), a.n_tokens);
  for (int t = beg + blockIdx.x; t < a.n_tokens; t += gridDim.x) zero_row<D>(a, t, threadIdx.x, kAttThreads);
}

template <int FMT, int D>
int launch_attention(const AttArgs& a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.n_tokens) * a.group / kAttRows + a.n_requests),
                  static_cast<unsigned>(a.heads));
  if (a.n_requests > 0) {
    LaunchScope scope(TWELL_KERNEL_KV_ATTENTION, s);
    if (launch_pdl(attention_kernel<FMT, D>, grid, dim3(kAttThreads), 0, s, a) != cudaSuccess) return TWELL_ERR_CUDA;
  }
  LaunchScope scope(TWELL_KERNEL_KV_ATTENTION, s);
  return launch_pdl(attention_rest_kernel<D>, dim3(16), dim3(kAttThreads), 0, s, a) == cudaSuccess ? TWELL_OK
                                                                                                   : TWELL_ERR_CUDA;
}

}  // namespace
}  // namespace twell

using namespace twell;

extern "C" TWELL_API size_t twell_kv_attention_workspace_bytes(int32_t n_tokens, int32_t n_requests,
                                                               int32_t n_q_heads, int32_t n_kv_heads,
                                                               int32_t head_dim) {
  if (n_tokens < 0 || n_requests < 0 || n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return 256;
}

extern "C" TWELL_API int twell_kv_attention(const uint16_t* Q, int64_t ldq, const twell_kv_t* cache,
                                            const int32_t* block_table, int32_t max_blocks, const int32_t* cu_q,
                                            const int32_t* positions, const int32_t* kv_lens, int32_t n_tokens,
                                            int32_t n_requests, int32_t n_q_heads, int32_t max_kv_len,
                                            int32_t max_q_len, float softmax_scale, uint16_t* O, int64_t ldo,
                                            float* lse, void* workspace, size_t workspace_bytes,
                                            twell_stream_t stream) {
  KV_TRY(check_kv(cache));
  if (n_tokens < 0 || n_requests < 0 || max_blocks < 0 || max_kv_len < 0 || max_q_len < 0)
    return TWELL_ERR_INVALID_ARG;
  if (n_q_heads < 1 || n_q_heads % cache->n_heads != 0) return TWELL_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.0f) || softmax_scale > 3.0e38f) return TWELL_ERR_INVALID_ARG;
  if (n_requests > kAttMaxRequests || cache->n_heads > 65535) return TWELL_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(n_tokens) * n_q_heads > INT32_MAX) return TWELL_ERR_UNSUPPORTED;
  if (n_tokens > 0) {
    KV_TRY(check_rows(Q, ldq, n_q_heads, cache->head_dim));
    KV_TRY(check_rows(O, ldo, n_q_heads, cache->head_dim));
    KV_TRY(check_array(positions, 4));
    KV_TRY(check_array(cu_q, 4));
    if (lse && !aligned_to(lse, 4)) return TWELL_ERR_MISALIGNED;
    if (n_requests > 0) {
      KV_TRY(check_array(kv_lens, 4));
      if (max_blocks > 0) KV_TRY(check_array(block_table, 4));
    }
  }
  const size_t need =
      twell_kv_attention_workspace_bytes(n_tokens, n_requests, n_q_heads, cache->n_heads, cache->head_dim);
  if (!workspace || workspace_bytes < need) return TWELL_ERR_WORKSPACE;
  if (!aligned_to(workspace, 256)) return TWELL_ERR_MISALIGNED;
  if (!device_is_sm103()) return TWELL_ERR_NO_DEVICE;
  if (n_tokens == 0) return TWELL_OK;
  AttArgs a{};
  a.q = Q;
  a.ldq = ldq;
  a.k = cache->k;
  a.v = cache->v;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.block_table = block_table;
  a.cu_q = cu_q;
  a.positions = positions;
  a.kv_lens = kv_lens;
  a.o = O;
  a.ldo = ldo;
  a.lse = lse;
  a.status = cache->status;
  a.max_blocks = max_blocks;
  a.n_tokens = n_tokens;
  a.n_requests = n_requests;
  a.q_heads = n_q_heads;
  a.heads = cache->n_heads;
  a.group = n_q_heads / cache->n_heads;
  a.page_shift = __builtin_ctz(cache->page_size);
  a.n_pages = cache->n_pages;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cache->format == TWELL_KV_E4M3)
    return cache->head_dim == 64 ? launch_attention<TWELL_KV_E4M3, 64>(a, s)
                                 : launch_attention<TWELL_KV_E4M3, 128>(a, s);
  return cache->head_dim == 64 ? launch_attention<TWELL_KV_INT8, 64>(a, s) : launch_attention<TWELL_KV_INT8, 128>(a, s);
}
