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
#include <algorithm>

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

// Eight dims of one finished row: o 2^(n - m) / sum, rounded once, and the row's lse.
template <int D>
__device__ __forceinline__ void store_row(const AttArgs& a, int t0, int row, int head, int d0, float m, float n,
                                          float sum, const float (&o)[8]) {
  const float f = m > -INFINITY ? exp2_fast(n - m) / sum : 0.0f;
  const int64_t token = t0 + row / a.group;
  const int h = head * a.group + row % a.group;
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = static_cast<uint32_t>(float_to_bf16_bits(o[2 * i] * f)) |
             (static_cast<uint32_t>(float_to_bf16_bits(o[2 * i + 1] * f)) << 16);
  *reinterpret_cast<uint4*>(a.o + token * a.ldo + static_cast<int64_t>(h) * D + d0) =
      make_uint4(out[0], out[1], out[2], out[3]);
  if (a.lse && d0 == 0)
    a.lse[token * a.q_heads + h] = m > -INFINITY ? (m + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

template <int D>
__device__ __forceinline__ void zero_row(const AttArgs& a, int64_t t, int tid, int n_threads) {
  for (int i = tid; i < a.q_heads * (D / 8); i += n_threads)
    *reinterpret_cast<uint4*>(a.o + t * a.ldo + i * 8) = make_uint4(0, 0, 0, 0);
  if (a.lse)
    for (int i = tid; i < a.q_heads; i += n_threads) a.lse[t * a.q_heads + i] = -INFINITY;
}

// ------------------------------------------------------------ work split
// A segment is one tile of 16 rows of one key head with all its cached tokens,
// in units of 64 of them.  The segments of all requests, laid end to end, are
// cut into as many equal pieces as CTAs run, so the lengths of the requests
// do not matter for the balance.  A piece's cut segments leave partial results in the
// workspace (two a CTA: of the segment it starts in the middle of, and of the
// one it ends in the middle of), which join_kernel adds in order.
constexpr int kUnit = kAttGroup * kAttWarps;  // cached tokens of a unit: 16 a warp
constexpr int kMaxCtas = 608;
// Segments of up to this many units are never cut: their join would cost more
// than the imbalance of leaving them whole.
constexpr int kWholeUnits = 4;
// Whole segments of up to this many units (512 tokens) go to single warps.
constexpr int kWarpUnits = 8;

struct Piece {   // of a segment that goes on in the next CTA, for join_kernel
  int32_t t0, n_rows, row0, head, last_cta, pad[3];
};

template <int D>
constexpr size_t partial_floats() { return static_cast<size_t>(kAttRows) * (D + 4); }

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

__device__ __forceinline__ int units_of(const Request& q) { return (q.len + kUnit - 1) / kUnit; }
__device__ __forceinline__ int row_blocks_of(const Request& q) { return (q.n_rows + kAttRows - 1) / kAttRows; }

// start[r] = units of the requests before r, start[n_requests] = all; by the whole CTA.
__device__ __forceinline__ void scan_requests(const AttArgs& a, int64_t* start, int64_t* warp_sum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_requests + kAttThreads - 1) / kAttThreads;
  const int r0 = min(a.n_requests, tid * per), r1 = min(a.n_requests, r0 + per);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) {
    const Request q = request(a, r);
    const int64_t w = static_cast<int64_t>(units_of(q)) * row_blocks_of(q) * a.heads;
    start[r] = w;
    mine += w;
  }
  int64_t inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int64_t run = inc - mine, all = 0;
#pragma unroll
  for (int w = 0; w < kAttWarps; ++w) {
    if (w < warp) run += warp_sum[w];
    all += warp_sum[w];
  }
  for (int r = r0; r < r1; ++r) {
    const int64_t w = start[r];
    start[r] = run;
    run += w;
  }
  if (tid == 0) start[a.n_requests] = all;
  __syncthreads();
}

// The last request that starts at or before unit u and has units.
__device__ __forceinline__ int request_at(const int64_t* start, int n, int64_t u) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (start[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Cut b of n_cuts over all units: moved to its segment's start where the segment stays whole.
__device__ __forceinline__ int64_t cut_at(const AttArgs& a, const int64_t* start, int64_t b, int64_t n_cuts,
                                          bool whole) {
  const int64_t all = start[a.n_requests];
  const int64_t u = b * all / n_cuts;
  if (b == 0 || u >= all) return b == 0 ? 0 : all;
  const int r = request_at(start, a.n_requests, u);
  const int units = units_of(request(a, r));
  const int64_t in = (u - start[r]) % units;
  return whole || units <= kWholeUnits ? u - in : u;
}

template <int D>
struct Ring {
  static constexpr int kStages = 4;
  static constexpr int kK = kAttGroup * D, kStage = 2 * kK + 16;  // bytes: keys, values, two scales
  static constexpr int kWarp = kStages * kStage;
  static_assert(kWarp >= static_cast<int>(partial_floats<D>() * 4), "a warp's results take the ring's place");
};

template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool on) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(kBytes),
                 "r"(on ? kBytes : 0)
                 : "memory");
}

// One warp's way through the segments seg, seg + 4, ... < seg_end of a request
// (row blocks of a head, then the next head): n_steps steps of 16 cached
// tokens each, j_stride tokens apart from j_first on.
struct Stream {
  const int32_t* table;
  int len, j_first, j_stride, n_steps, seg, seg_end, blocks;
};

// The copies run kStages - 1 steps ahead of the arithmetic, over the ends of
// segments too.  Several segments need n_steps <= 32 (their page numbers stay
// in one register a lane).
template <int FMT, int D, typename Emit>
__device__ __forceinline__ void run_stream(const AttArgs& a, const Stream& st, const Request& q, uint8_t* ring,
                                           Emit emit) {
  using R = Ring<D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
  const int page_mask = (1 << a.page_shift) - 1;
  // page numbers of 32 steps at a time, one a lane, and the next 32 behind them
  const auto pages_from = [&](int step) {
    int page = 0;
    if (step + lane < st.n_steps) {
      page = st.table[(st.j_first + (step + lane) * st.j_stride) >> a.page_shift];
      if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.n_pages)) {
        report_error(a.status, TWELL_ERR_BAD_FORMAT);
        page = 0;
      }
    }
    return page;
  };
  int pages = 0, pages_next = 0;
  if (st.seg < st.seg_end) {
    pages = pages_from(0);
    if (st.n_steps > 32) pages_next = pages_from(32);
  }
  int f_seg = st.seg, f_step = 0, f_slot = 0;  // the next copy
  const auto fetch = [&]() {
    if (f_seg < st.seg_end && st.n_steps > 0) {
      if (f_step > 0 && (f_step & 31) == 0) {
        pages = pages_next;
        if (f_step + 32 < st.n_steps) pages_next = pages_from(f_step + 32);
      }
      const int page = __shfl_sync(0xffffffffu, pages, f_step & 31);
      uint8_t* const stage = ring + f_slot * R::kStage;
      const int j0 = st.j_first + f_step * st.j_stride;
      const int64_t cell = static_cast<int64_t>(page) * a.heads + f_seg / st.blocks;
      const int64_t at = ((cell << a.page_shift) + (j0 & page_mask)) * D;
      // lane l's bytes of each load lie together: it reads back what it copied
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          copy_async<16>(stage + ((nt * (D / 64) + i) * 32 + lane) * 16,
                         a.k + at + (nt * 8 + g) * D + 64 * i + 16 * quad, true);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int token = (i >> 1) * 8 + 2 * quad + (i & 1);
        // past the request's tokens the page may hold anything, and 0 * NaN is
        // not 0: zeros in its place
        copy_async<D / 8>(stage + R::kK + (i * 32 + lane) * (D / 8), a.v + at + token * D + (D / 8) * g,
                          j0 + token < st.len);
      }
      if (lane < 2) copy_async<4>(stage + 2 * R::kK + 4 * lane, (lane == 0 ? a.k_scale : a.v_scale) + cell, true);
      if (++f_step == st.n_steps) f_step = 0, f_seg += kAttWarps;
    }
    f_slot = f_slot + 1 == R::kStages ? 0 : f_slot + 1;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < R::kStages - 1; ++i) fetch();
  int slot = 0;
  for (int seg = st.seg; seg < st.seg_end; seg += kAttWarps) {
    const int head = seg / st.blocks, row0 = seg % st.blocks * kAttRows;
    // what each row sees; rows past the last see everything and are not stored
    int limit[2], least = INT32_MAX;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = row0 + g + 8 * half;
      limit[half] = INT32_MAX;
      if (row < q.n_rows) {
        const int p = a.positions[q.t0 + row / a.group];
        limit[half] = max(0, min(p < INT32_MAX ? p + 1 : p, q.len));
        least = min(least, limit[half]);
      }
    }
#pragma unroll
    for (int d = 16; d >= 4; d /= 2) least = min(least, __shfl_xor_sync(0xffffffffu, least, d));
    least = min(least, st.len);
    uint32_t qa[D / 16][4];
    float factor[2];
    load_q<D>(a, q.t0, q.n_rows, row0, head, qa, factor);
    TileState<D> s;
    reset(s);
    for (int step = 0; step < st.n_steps; ++step) {
      __syncwarp();  // the scales that fetch replaces have been read by all lanes
      fetch();
      asm volatile("cp.async.wait_group %0;" ::"n"(R::kStages - 1) : "memory");
      __syncwarp();  // the scales came in by two lanes
      const uint8_t* const stage = ring + slot * R::kStage;
      slot = slot + 1 == R::kStages ? 0 : slot + 1;
      const int j0 = st.j_first + step * st.j_stride;
      uint32_t kw[2][D / 16], vw[4][D / 32];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          *reinterpret_cast<uint4*>(&kw[nt][4 * i]) =
              *reinterpret_cast<const uint4*>(stage + ((nt * (D / 64) + i) * 32 + lane) * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* src = stage + R::kK + (i * 32 + lane) * (D / 8);
        if constexpr (D == 128)
          *reinterpret_cast<uint4*>(vw[i]) = *reinterpret_cast<const uint4*>(src);
        else
          *reinterpret_cast<uint2*>(vw[i]) = *reinterpret_cast<const uint2*>(src);
      }
      const float2 scales = *reinterpret_cast<const float2*>(stage + 2 * R::kK);
      step16<FMT, D>(s, qa, factor, kw, vw, scales.x, scales.y, j0, limit, j0 + kAttGroup > least);
    }
    if (seg + kAttWarps >= st.seg_end) asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      s.sum[half] += __shfl_xor_sync(0xffffffffu, s.sum[half], 1);
      s.sum[half] += __shfl_xor_sync(0xffffffffu, s.sum[half], 2);
    }
    emit(s, head, row0);
  }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kAttThreads, 3)
    attention_kernel(const AttArgs a, float* partial, Piece* pieces, int whole) {
  using R = Ring<D>;
  extern __shared__ __align__(16) uint8_t dyn[];
  uint8_t* const ring_all = dyn;
  int64_t* const start = reinterpret_cast<int64_t*>(dyn + kAttWarps * R::kWarp);
  __shared__ int64_t warp_sum[kAttWarps];
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, quad = lane & 3;
  uint8_t* const ring = ring_all + warp * R::kWarp;
  scan_requests(a, start, warp_sum);
  // at least a unit for each CTA that works, so that every CTA between a cut
  // segment's first and last has a part of it
  const int64_t cta = blockIdx.x, n_ctas = min(static_cast<int64_t>(gridDim.x), start[a.n_requests]);
  const int64_t end = cta < n_ctas ? cut_at(a, start, cta + 1, n_ctas, whole) : 0;
  int64_t pos = cta < n_ctas ? cut_at(a, start, cta, n_ctas, whole) : 0;
  if (tid == 0) pieces[cta].last_cta = -1;
  // requests without cached tokens, and tokens of no request
  for (int r = blockIdx.x; r < a.n_requests; r += gridDim.x) {
    const Request q = request(a, r);
    if (q.len == 0)
      for (int t = 0; t < q.n_rows / a.group; ++t) zero_row<D>(a, q.t0 + t, tid, kAttThreads);
  }
  for (int t = min(max(a.cu_q[a.n_requests], 0), a.n_tokens) + blockIdx.x; t < a.n_tokens; t += gridDim.x)
    zero_row<D>(a, t, tid, kAttThreads);

  int turn = 0;  // of the warps at whole segments
  while (pos < end) {
    const int r = request_at(start, a.n_requests, pos);
    const Request q = request(a, r);
    const int units = units_of(q), blocks = row_blocks_of(q);
    const int64_t seg0 = (pos - start[r]) / units;
    const int unit0 = static_cast<int>((pos - start[r]) % units);
    Stream st;
    st.table = a.block_table + static_cast<int64_t>(r) * a.max_blocks;
    st.len = q.len;
    if (unit0 == 0 && units <= kWarpUnits && end - pos >= units) {
      // short segments that lie whole in this piece: each warp takes every fourth
      const int64_t left = static_cast<int64_t>(blocks) * a.heads - seg0;
      const int count = static_cast<int>(min(left, (end - pos) / units));
      st.j_first = 0;
      st.j_stride = kAttGroup;
      st.n_steps = (q.len + kAttGroup - 1) / kAttGroup;
      st.seg = static_cast<int>(seg0) + ((warp - turn) & (kAttWarps - 1));
      st.seg_end = static_cast<int>(seg0) + count;
      st.blocks = blocks;
      turn += count;
      pos += static_cast<int64_t>(count) * units;
      run_stream<FMT, D>(a, st, q, ring, [&](TileState<D>& s, int head, int row0) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = row0 + g + 8 * half;
          if (row >= q.n_rows) continue;
#pragma unroll
          for (int i0 = 0; i0 < 2 * (D / 8); i0 += 8) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = s.acc[(i0 + i) % (D / 8)][2 * half + (i0 + i) / (D / 8)];
            store_row<D>(a, q.t0, row, head, (D / 8) * 2 * quad + i0, s.m[half], s.n[half], s.sum[half], o);
          }
        }
      });
      continue;
    }
    const int n_units = static_cast<int>(min(static_cast<int64_t>(units - unit0), end - pos));
    pos += n_units;
    st.j_first = unit0 * kUnit + warp * kAttGroup;
    st.j_stride = kUnit;
    const int seen = min(n_units * kUnit, q.len - unit0 * kUnit) - warp * kAttGroup;
    st.n_steps = seen > 0 ? (seen + kUnit - 1) / kUnit : 0;
    st.seg = static_cast<int>(seg0);
    st.seg_end = st.seg + 1;
    st.blocks = blocks;
    // the four warps' results of the tile, joined in warp order; they take the ring's place
    run_stream<FMT, D>(a, st, q, ring, [&](TileState<D>& s, int, int row0) {
      float* const mine = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = g + 8 * half;
        if (row0 + row < q.n_rows) {
          float* const at = mine + row * (D + 4);
          if (quad == 0) at[D] = s.m[half], at[D + 1] = s.n[half], at[D + 2] = s.sum[half];
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            at[(D / 8) * (2 * quad) + i] = s.acc[i][2 * half];
            at[(D / 8) * (2 * quad + 1) + i] = s.acc[i][2 * half + 1];
          }
        }
      }
    });
    __syncthreads();
    const int head = st.seg / blocks, row0 = st.seg % blocks * kAttRows;
    constexpr int kLanes = D / 8;
    const bool complete = n_units == units, goes_on = unit0 + n_units < units;
    // a cut segment's part: slot 1 where it starts here, slot 0 where it came from the CTA before
    float* const out = partial + (2 * cta + (unit0 == 0 ? 1 : 0)) * partial_floats<D>();
    if (unit0 == 0 && goes_on && tid == 0) {
      // cuts inside a segment that may be cut are where the even split puts
      // them, so the CTA of its last unit follows from the split alone
      const int64_t seg_end = pos + (units - n_units);
      pieces[cta] = {q.t0, q.n_rows, row0, head,
                     static_cast<int32_t>((seg_end * n_ctas - 1) / start[a.n_requests]), {0, 0, 0}};
    }
    for (int row = tid / kLanes; row < min(kAttRows, q.n_rows - row0); row += kAttThreads / kLanes) {
      const int d0 = (tid % kLanes) * 8;
      float m = -INFINITY, n = -INFINITY, sum = 0.0f, o[8] = {};
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) {
        const float* at = reinterpret_cast<const float*>(ring_all + w * R::kWarp) + row * (D + 4);
        m = fmaxf(m, at[D]);
        n = fmaxf(n, at[D + 1]);
      }
      if (m > -INFINITY) {
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) {
          const float* at = reinterpret_cast<const float*>(ring_all + w * R::kWarp) + row * (D + 4);
          sum += at[D + 2] * exp2_fast(at[D] - m);
          const float f = exp2_fast(at[D + 1] - n);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += at[d0 + i] * f;
        }
      }
      if (complete) {
        store_row<D>(a, q.t0, row0 + row, head, d0, m, n, sum, o);
      } else {
        float* const to = out + row * (D + 4);
        *reinterpret_cast<float4*>(to + d0) = make_float4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<float4*>(to + d0 + 4) = make_float4(o[4], o[5], o[6], o[7]);
        if (d0 == 0) *reinterpret_cast<float4*>(to + D) = make_float4(m, n, sum, 0.0f);
      }
    }
    __syncthreads();  // the ring is free again
  }
}

// Adds a cut segment's parts in the order of its units: one CTA for each CTA
// of attention_kernel, idle unless a segment starts there and goes on.
template <int D>
__global__ void __launch_bounds__(kAttThreads) join_kernel(const AttArgs a, const float* partial, const Piece* pieces) {
  grid_dependency_wait();
  const int cta = blockIdx.x, tid = threadIdx.x;
  const Piece p = pieces[cta];
  if (p.last_cta <= cta) return;
  constexpr int kLanes = D / 8;
  const int d0 = (tid % kLanes) * 8;
  const auto part = [&](int c, int row) {
    return partial + (2 * static_cast<int64_t>(c) + (c == cta ? 1 : 0)) * partial_floats<D>() + row * (D + 4);
  };
  for (int row = tid / kLanes; row < min(kAttRows, p.n_rows - p.row0); row += kAttThreads / kLanes) {
    float m = -INFINITY, n = -INFINITY, sum = 0.0f, o[8] = {};
#pragma unroll 4
    for (int c = cta; c <= p.last_cta; ++c) {
      const float* const at = part(c, row);
      m = fmaxf(m, at[D]);
      n = fmaxf(n, at[D + 1]);
    }
    if (m > -INFINITY) {
#pragma unroll 4
      for (int c = cta; c <= p.last_cta; ++c) {
        const float* const at = part(c, row);
        const float4 st = *reinterpret_cast<const float4*>(at + D), lo = *reinterpret_cast<const float4*>(at + d0),
                     hi = *reinterpret_cast<const float4*>(at + d0 + 4);
        sum += st.z * exp2_fast(st.x - m);
        const float f = exp2_fast(st.y - n);
        o[0] += lo.x * f, o[1] += lo.y * f, o[2] += lo.z * f, o[3] += lo.w * f;
        o[4] += hi.x * f, o[5] += hi.y * f, o[6] += hi.z * f, o[7] += hi.w * f;
      }
    }
    store_row<D>(a, p.t0, p.row0 + row, p.head, d0, m, n, sum, o);
  }
}

template <int FMT, int D>
int launch_attention(const AttArgs& a, int max_kv_len, int max_q_len, void* workspace, cudaStream_t s) {
  float* const partial = static_cast<float*>(workspace);
  Piece* const pieces = reinterpret_cast<Piece*>(partial + 2 * kMaxCtas * partial_floats<D>());
  const size_t smem = kAttWarps * Ring<D>::kWarp + sizeof(int64_t) * (static_cast<size_t>(a.n_requests) + 1);
  const void* fn = reinterpret_cast<const void*>(attention_kernel<FMT, D>);
  KV_TRY(set_max_dynamic_smem(fn, static_cast<int>(kAttWarps * Ring<D>::kWarp + 8 * (kAttMaxRequests + 1))));
  const int resident = resident_ctas_per_sm(fn, kAttThreads, smem);
  if (resident < 1) return TWELL_ERR_CUDA;
  // no more CTAs than the units that the caller's bounds allow
  const int64_t blocks = (static_cast<int64_t>(max_q_len) * a.group + kAttRows - 1) / kAttRows;
  const int64_t units = (static_cast<int64_t>(max_kv_len) + kUnit - 1) / kUnit;
  const int64_t most = std::max<int64_t>(1, a.n_requests * a.heads * std::max<int64_t>(1, blocks * units));
  const int ctas = static_cast<int>(
      std::min<int64_t>(most, std::min(kMaxCtas, sm_count() * resident)));
  const bool whole = units <= kWholeUnits;
  {
    LaunchScope scope(TWELL_KERNEL_KV_ATTENTION, s);
    if (launch_pdl(attention_kernel<FMT, D>, dim3(ctas), dim3(kAttThreads), smem, s, a, partial, pieces,
                   static_cast<int>(whole)) != cudaSuccess)
      return TWELL_ERR_CUDA;
  }
  if (whole || ctas == 1) return TWELL_OK;
  LaunchScope scope(TWELL_KERNEL_KV_JOIN, s);
  return launch_pdl(join_kernel<D>, dim3(ctas - 1), dim3(kAttThreads), 0, s, a, static_cast<const float*>(partial),
                    static_cast<const Piece*>(pieces)) == cudaSuccess
             ? TWELL_OK
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
  return (2 * kMaxCtas * static_cast<size_t>(kAttRows) * (head_dim + 4) * sizeof(float) + kMaxCtas * sizeof(Piece) + 255) /
         256 * 256;
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
    return cache->head_dim == 64 ? launch_attention<TWELL_KV_E4M3, 64>(a, max_kv_len, max_q_len, workspace, s)
                                 : launch_attention<TWELL_KV_E4M3, 128>(a, max_kv_len, max_q_len, workspace, s);
  return cache->head_dim == 64 ? launch_attention<TWELL_KV_INT8, 64>(a, max_kv_len, max_q_len, workspace, s) : launch_attention<TWELL_KV_INT8, 128>(a, max_kv_len, max_q_len, workspace, s);
}
