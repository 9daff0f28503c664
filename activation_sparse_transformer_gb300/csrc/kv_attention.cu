// Attention over the 8-bit paged cache (twell_kv_attention).
//
// For token t of request r and query head h (key / value head h / G):
//   x_j = c q . k_j,  o = sum_j exp(x_j) v_j / sum_j exp(x_j),  j < L
// with k_j = s_k code, v_j = s_v code, one scale per page and head.  The rows
// (token, query head) of one request that share a key / value head form the
// 16 rows of an mma tile, so each cached byte is read once for all of them.
// Per 16 cached tokens a warp computes
//   S = Q K^T                 fp16 x fp16 -> fp32, codes exact in fp16
//   l = S (c log2(e) 2^k s_k) + log2 s_v   (2^k: the row's own factor, see convert_q)
//   w = 2^(l - n)  ->  fp16,  O += w V,  sum += w / s_v
// in one pass.  n is the row's reference: it follows the largest l (kRoom below it), that is,
// the largest weight that a code is multiplied with, so the fp16 weights stay in their
// range whatever the pages' scales are; the sum is fp32 and may differ from O's
// scale by as much as the scales do (pages 2^100 apart are told apart still).
//
// The products are computed transposed, S^T = K Q^T and O^T = V^T P^T, with the
// cached tokens (or the dims) on the 16-wide side of the mma and the rows on the
// 8-wide one: a decode step has 1 to 8 rows for a key head, and half the mma's,
// exponentials and registers of the other orientation.  The reduction index of an
// mma may be permuted as long as both operands agree, and so may the rows of
// its result.  K's lanes therefore take 16 consecutive bytes of one token (two
// loads for D = 128) and Q is gathered to match; V's lanes take the same 16 (D =
// 128) or 8 bytes of four tokens, whose bytes are paired to fp16 registers, and the output's
// dims come out in runs.  No transposition lies between the cache and the mma;
// P's 8 x 8 blocks are turned by movmatrix.
//
// Below, W is a CTA's warps: 4, or 8 where a segment has an SM to itself.
//
// Each cached byte is read once, so HBM bounds long caches: 4 x 65536 to 131072 tokens, 8 key heads of 128, e4m3:
// 133 us, 5.8 TB/s.  Heads with one query row each and 64 dims are bound by the chain of
// dependent instructions of a warp's step (480 for 32 tokens, a third of them conversions; 54 % of the issue slots busy,
// the largest stall their fixed latency): 250 ragged requests, int8, 137 us, 4.2 TB/s.
// Short caches are bound by the latencies in a row (lengths, table, codes, softmax): 16 x 1000 tokens 10.5 us.
#include <algorithm>
#include <cfloat>

#include "kv_attention.h"

namespace twell {
namespace {

constexpr int kAttWarps = 4;
constexpr int kWideWarps = 8;  // of a CTA that has an SM to itself
constexpr int kMaxTiles = 2;    // a row block is 1 or 2 tiles of 8 rows
constexpr int kMaxRows = 8 * kMaxTiles;
constexpr int kAttGroup = 16;   // cached tokens of one mma, all of one page
constexpr int kAttStep = 2 * kAttGroup;  // cached tokens of one warp step
constexpr int kAttMaxRequests = 4096;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A row block: NT = 1 or 2 tiles of 8 rows, or (0) 4 rows in every other column of a tile.
template <int NT>
constexpr int kTiles = NT == 0 ? 1 : NT;
template <int NT>
constexpr int kCols = NT == 0 ? 1 : 2;  // of a tile, in a lane
template <int NT>
constexpr int kRows = NT == 0 ? 4 : 8 * NT;
template <int NT>
__device__ __forceinline__ int row_in(int t, int quad, int c) { return NT == 0 ? quad : 8 * t + 2 * quad + c; }

// One row block's running state in a warp: rows row_in(t, quad, c) of its
// tiles t, whose statistics the 8 lanes of a quad column share.
template <int D, int NT>
struct TileState {
  float acc[kTiles<NT>][D / 16][4];   // i: dims (D / 8) g + 2 i (both rows), then + 1 (both rows)
  float n[kTiles<NT>][2];     // the reference (0 before the first value)
  float pass[kTiles<NT>][2];  // what an exponent must pass to move it
  float sum[kTiles<NT>][2];   // sum of 2^(l - n - kRoom) / s_v
};

template <int D, int NT>
__device__ __forceinline__ void reset(TileState<D, NT>& s) {
#pragma unroll
  for (int t = 0; t < kTiles<NT>; ++t) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s.acc[t][i][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s.n[t][i] = s.sum[t][i] = 0.0f;
      s.pass[t][i] = -INFINITY;
    }
  }
}

// The block's rows as fp16 fragments.  A row enters as q 2^-k with its largest
// magnitude in [1, 2): exact in fp16 for components above 2^-14 and off by at
// most 2^-25 below, which is less than the fp32 sum's own rounding.  factor
// returns c log2(e) 2^k of rows 2 quad and 2 quad + 1.
template <int D, int NT>
struct RawQ {
  uint4 w[kTiles<NT>][D / 32];
};

template <int D, int NT>
__device__ __forceinline__ void load_q(const AttArgs& a, int64_t t0, int n_rows, int row0, int head,
                                       RawQ<D, NT>& raw) {
  const int lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
#pragma unroll
  for (int t = 0; t < kTiles<NT>; ++t) {
    const int row = NT == 0 ? row0 + g / 2 : row0 + 8 * t + g, token = row / a.group;
    const bool on = row < n_rows && (NT > 0 || g % 2 == 0);
    const uint16_t* src = a.q + (t0 + token) * a.ldq + (static_cast<int64_t>(head) * a.group + row % a.group) * D;
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        raw.w[t][2 * i + j] = on ? __ldg(reinterpret_cast<const uint4*>(src + 64 * i + 16 * quad + 8 * j))
                                           : make_uint4(0, 0, 0, 0);
  }
}

template <int D, int NT>
__device__ __forceinline__ void convert_q(const AttArgs& a, const RawQ<D, NT>& raw, uint32_t (&qb)[kTiles<NT>][D / 16][2],
                                          float (&factor)[kTiles<NT>][2]) {
  const int quad = threadIdx.x & 3;
#pragma unroll
  for (int t = 0; t < kTiles<NT>; ++t) {
    const uint32_t* u = &raw.w[t][0].x;
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(u[i])), fabsf(bf16_hi(u[i]))));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int k = min(max((__float_as_int(amax) >> 23) - 127, -126), 126);
    const float inv = __int_as_float((127 - k) << 23);
    const float f = a.scale_log2 * __int_as_float((127 + k) << 23);
    factor[t][0] = __shfl_sync(0xffffffffu, f, 8 * quad);
    if (NT > 0) factor[t][1] = __shfl_sync(0xffffffffu, f, 8 * quad + 4);
    // word j of a lane's code vectors holds dims 4 j .. 4 j + 3 = u[2 j], u[2 j + 1]
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p) qb[t][j][p] = pack_f16(bf16_lo(u[2 * j + p]) * inv, bf16_hi(u[2 * j + p]) * inv);
  }
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// One warp step: the 32 cached tokens [j0, j0 + 32), two groups of 16 that may
// lie in two pages, from a stage of the ring: keys of both groups, then values.
// limit: tokens each row sees; least: the smallest of them; len: the request's tokens.
template <int FMT, int D, int NT>
__device__ __forceinline__ void step32(TileState<D, NT>& s, const uint32_t (&qb)[kTiles<NT>][D / 16][2],
                                       const float (&factor)[kTiles<NT>][2], const uint8_t* stage, const float (&ks)[2],
                                       const float (&lvs)[2], const float (&ivs)[2], int j0,
                                       const int (&limit)[kTiles<NT>][2], int least, int len) {
  const int lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
  float x[2][kTiles<NT>][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t kw[2][D / 16];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        *reinterpret_cast<uint4*>(&kw[r][4 * i]) =
            *reinterpret_cast<const uint4*>(stage + (16 * h + 8 * r + g) * D + 64 * i + 16 * quad);
#pragma unroll
    for (int t = 0; t < kTiles<NT>; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[h][t][i] = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint32_t ka[4];
      codes_to_f16<FMT>(kw[0][j], ka[0], ka[2]);
      codes_to_f16<FMT>(kw[1][j], ka[1], ka[3]);
#pragma unroll
      for (int t = 0; t < kTiles<NT>; ++t) mma_f16(x[h][t], ka, qb[t][j][0], qb[t][j][1]);
    }
  }
  const bool mask = j0 + kAttStep > least;
  bool move = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int t = 0; t < kTiles<NT>; ++t)
#pragma unroll
      for (int c = 0; c < kCols<NT>; ++c) {
        const float f = fmaxf(factor[t][c] * ks[h], FLT_MIN);  // a masked -inf stays so
        if (mask) {
          if (j0 + 16 * h + g >= limit[t][c]) x[h][t][c] = -INFINITY;
          if (j0 + 16 * h + g + 8 >= limit[t][c]) x[h][t][2 + c] = -INFINITY;
        }
        x[h][t][c] = fmaf(x[h][t][c], f, lvs[h]);
        x[h][t][2 + c] = fmaf(x[h][t][2 + c], f, lvs[h]);
        move |= fmaxf(x[h][t][c], x[h][t][2 + c]) > s.pass[t][c];
      }
  }
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int t = 0; t < kTiles<NT>; ++t)
#pragma unroll
      for (int c = 0; c < kCols<NT>; ++c) {
        float n = fmaxf(fmaxf(x[0][t][c], x[0][t][2 + c]), fmaxf(x[1][t][c], x[1][t][2 + c]));
#pragma unroll
        for (int d = 4; d <= 16; d *= 2) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, d));
        if (n == -INFINITY) continue;  // nothing seen here
        // The reference only grows; before the first value it is 0 and nothing has been added.  (Not
        // told by the sum: that is of this lane's tokens, acc of all tokens for this lane's dims.)
        n = fmaxf(n, s.pass[t][c] - kLazy);
        const float f = s.pass[t][c] == -INFINITY ? 0.0f : exp2_fast(s.n[t][c] + kRoom - n);
        s.sum[t][c] *= f;
        s.n[t][c] = n - kRoom;
        s.pass[t][c] = n + kLazy;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          s.acc[t][i][c] *= f;
          s.acc[t][i][2 + c] *= f;
        }
      }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t pb[kTiles<NT>][2];
#pragma unroll
    for (int t = 0; t < kTiles<NT>; ++t) {
      float w[4] = {};
#pragma unroll
      for (int c = 0; c < kCols<NT>; ++c) {
        w[c] = exp2_fast(x[h][t][c] - s.n[t][c]);
        w[2 + c] = exp2_fast(x[h][t][2 + c] - s.n[t][c]);
        const float both = w[c] + w[2 + c];
        if (both != 0.0f) s.sum[t][c] = fmaf(both, ivs[h], s.sum[t][c]);  // a page that is not seen may have any scale
      }
      pb[t][0] = transpose8(pack_f16(w[0], w[1]));
      pb[t][1] = transpose8(pack_f16(w[2], w[3]));
    }
    uint32_t vw[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* src = stage + (kAttStep + 16 * h + (i >> 1) * 8 + 2 * quad + (i & 1)) * D + (D / 8) * g;
      if constexpr (D == 128)
        *reinterpret_cast<uint4*>(vw[i]) = *reinterpret_cast<const uint4*>(src);
      else
        *reinterpret_cast<uint2*>(vw[i]) = *reinterpret_cast<const uint2*>(src);
    }
    if (mask) {
      // Past the request's tokens the page (or the stage) may hold anything, and so may a token
      // that not all rows see, but 0 * NaN is not 0: zeros in their place, and NaN
      // for the rows that do see such a token.
      uint32_t bad = 0;  // tokens of the group with a NaN among their codes
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int token = (i >> 1) * 8 + 2 * quad + (i & 1);
        uint32_t nan = 0;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          if (j0 + 16 * h + token >= len) vw[i][w] = 0;
          if (FMT == TWELL_KV_E4M3) nan |= nan_codes(vw[i][w]);
        }
        if (nan) bad |= 1u << token;
      }
      if (FMT == TWELL_KV_E4M3) bad = __reduce_or_sync(0xffffffffu, bad);
      if (bad) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int w = 0; w < D / 32; ++w)
            if (bad >> ((i >> 1) * 8 + 2 * quad + (i & 1)) & 1) vw[i][w] = 0;
#pragma unroll
        for (int t = 0; t < kTiles<NT>; ++t)
#pragma unroll
          for (int c = 0; c < kCols<NT>; ++c)
            if (limit[t][c] >= j0 + 16 * h + __ffs(bad)) {
#pragma unroll
              for (int i = 0; i < D / 16; ++i) s.acc[t][i][c] = s.acc[t][i][2 + c] = __int_as_float(0x7FC00000);
            }
      }
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      // bytes of two neighbouring tokens side by side, then to fp16 pairs
      uint32_t va[2][4];
      codes_to_f16<FMT>(__byte_perm(vw[0][w], vw[1][w], 0x5140), va[0][0], va[0][1]);
      codes_to_f16<FMT>(__byte_perm(vw[0][w], vw[1][w], 0x7362), va[1][0], va[1][1]);
      codes_to_f16<FMT>(__byte_perm(vw[2][w], vw[3][w], 0x5140), va[0][2], va[0][3]);
      codes_to_f16<FMT>(__byte_perm(vw[2][w], vw[3][w], 0x7362), va[1][2], va[1][3]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < kTiles<NT>; ++t) mma_f16(s.acc[t][2 * w + i], va[i], pb[t][0], pb[t][1]);
    }
  }
}

template <int D>
__device__ __forceinline__ void zero_row(const AttArgs& a, int64_t t, int tid, int n_threads) {
  for (int i = tid; i < a.q_heads * (D / 8); i += n_threads)
    *reinterpret_cast<uint4*>(a.o + t * a.ldo + i * 8) = make_uint4(0, 0, 0, 0);
  if (a.lse)
    for (int i = tid; i < a.q_heads; i += n_threads) a.lse[t * a.q_heads + i] = -INFINITY;
}

// ------------------------------------------------------------ work split
// A segment is one row block of one key head with all its cached tokens, in
// units of a step of each warp (32 W of them).  The segments of all requests, laid end to end, are
// cut into as many equal pieces as CTAs run, so the lengths of the requests do
// not matter for the balance; every CTA sums up the requests itself (a few loads a
// thread) rather than wait for another kernel.  A piece's cut segments leave partial
// results in the workspace (two a CTA: of the segment it starts in the middle of, and of
// the one it ends in the middle of), which join_kernel adds in order.  (Adding them in the CTA
// that finishes last costs more: one CTA's loads have to bring in all parts.)  Short
// segments are not cut, see launch_attention.
constexpr int kUnit = kAttStep * kAttWarps;  // cached tokens of a unit with 4 warps: a step of each
constexpr int kMaxCtas = 608;
constexpr int kMaxSmem = 224 * 1024;  // dynamic, of a CTA
// Segments of up to this many units are never cut: their join would cost more
// than the imbalance of leaving them whole.
constexpr int kWholeUnits = 2;
// Segments of up to this many steps (512 tokens) go to single warps: the groups that
// the 32 lanes of run_stream look after, which it loads once for all of a warp's segments.
constexpr int kWarpSteps = 16;

struct Piece {   // of a segment that goes on in the next CTA, for join_kernel
  int32_t t0, n_rows, row0, head, last_cta, pad[3];
};

template <int D>
constexpr size_t partial_floats() { return static_cast<size_t>(kMaxRows) * (D + 4); }

template <int W>
__device__ __forceinline__ int units_of(const Request& q) { return (q.len + (kAttStep * W) - 1) / (kAttStep * W); }
template <int NT>
__device__ __forceinline__ int row_blocks_of(const Request& q) {
  return (q.n_rows + kRows<NT> - 1) / kRows<NT>;
}

// How the segments are dealt out.
enum Split {
  kCut,    // equal units, segments cut
  kWhole,  // equal units, the cuts moved to segments' starts: no join
  kEach    // every segment to a CTA of its own (there are CTAs enough): no join
};

// What a segment counts for in the split.
template <int W>
__device__ __forceinline__ int span_of(const Request& q, int split) {
  const int units = units_of<W>(q);
  return split == kEach ? min(units, 1) : units;
}

// start[r] = units of the requests before r, start[n_requests] = all; by the whole CTA.
template <int NT, int W>
__device__ __forceinline__ void scan_requests(const AttArgs& a, int64_t* start, int64_t* warp_sum, int split) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_requests + (32 * W) - 1) / (32 * W);
  const int r0 = min(a.n_requests, tid * per), r1 = min(a.n_requests, r0 + per);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) {
    const Request q = request(a, r);
    const int64_t w =
        q.n_rows > a.chunk_rows ? 0 : static_cast<int64_t>(span_of<W>(q, split)) * row_blocks_of<NT>(q) * a.heads;
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
  for (int w = 0; w < W; ++w) {
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
template <int W>
__device__ __forceinline__ int64_t cut_at(const AttArgs& a, const int64_t* start, int64_t b, int64_t n_cuts,
                                          int split) {
  const int64_t all = start[a.n_requests];
  const int64_t u = b * all / n_cuts;
  if (b == 0 || u >= all) return b == 0 ? 0 : all;
  const int r = request_at(start, a.n_requests, u);
  if (split == kEach) return u;
  const int units = units_of<W>(request(a, r));
  return split == kWhole || units <= kWholeUnits ? u - (u - start[r]) % units : u;
}

// A warp's own ring of stages in shared memory: a step's keys, then its values,
// each D bytes a token as in the cache.
template <int D>
struct Ring {
  // with as many CTAs on an SM as its registers allow, and with one
  static constexpr int kLeast = D == 128 ? 2 : 3, kMost = D == 128 ? 6 : 12;
  static constexpr int kGroup = kAttGroup * D, kStage = 4 * kGroup;
  static_assert(kLeast * kStage >= static_cast<int>(partial_floats<D>() * 4), "a warp's results take the ring's place");
  int stages;
  uint8_t* data;
  uint64_t* full;   // [stages] mbarriers, two arrivals each: one a group
  volatile int* abort;
  int slot;         // the stage of the next step
  uint32_t phases;  // bit i: the parity that full[i] completes next
};

// One warp's way through the segments seg, seg + W, ... < seg_end of a request
// (row blocks of a head, then the next head): n_steps steps of 32 cached
// tokens each, j_stride tokens apart from j_first on.
struct Stream {
  const int32_t* table;
  int len, j_first, j_stride, n_steps, seg, seg_end, blocks;
};

// The copies (bulk copies of 16 D bytes, the keys and the values of a group) run
// a ring less one step ahead of the arithmetic, over the ends of segments too.  Lane l
// looks after the groups l, l + 32, ... of a segment: it holds the page's
// place and scales and issues the copies.  Only a stream of one segment may have more than 32 groups
// (kWarpSteps steps): the places of the first 32 are not loaded again for the next segment.
// False when a wait expired: the segment has no result, and no copy is in flight any more.
template <int FMT, int D, int NT, int W, typename Emit>
__device__ __forceinline__ bool run_stream(const AttArgs& a, const Stream& st, const Request& q, Ring<D>& ring,
                                           Emit emit) {
  using R = Ring<D>;
  if (st.seg >= st.seg_end) return true;
  const int lane = threadIdx.x & 31, quad = lane & 3;
  const int page_mask = (1 << a.page_shift) - 1;
  const int64_t head_bytes = static_cast<int64_t>(D) << a.page_shift;
  struct Batch {
    int64_t cell;   // of head 0
    int64_t at;     // its place in head 0, in bytes
    bool on;        // there is such a group
    float ks, lvs, ivs;  // key scale, log2 of the value scale, 2^-kRoom over it
  };
  const auto scales_of = [&](Batch& b, int head) {
    if (b.on) {
      const float vs = __ldg(a.v_scale + b.cell + head);
      b.ks = __ldg(a.k_scale + b.cell + head);
      b.lvs = log2_scale(vs);
      b.ivs = kUnroom / vs;
    }
  };
  const auto batch_from = [&](int step, int head) {
    Batch b = {0, 0, false, 1.0f, 0.0f, 1.0f};
    const int mine = step + lane / 2;
    const int j = st.j_first + mine * st.j_stride + (lane & 1) * kAttGroup;
    if (mine < st.n_steps && j < st.len) {
      int page = st.table[j >> a.page_shift];
      if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.n_pages)) {
        report_error(a.status, TWELL_ERR_BAD_FORMAT);
        page = 0;
      }
      b.cell = static_cast<int64_t>(page) * a.heads;
      b.at = b.cell * head_bytes + (j & page_mask) * D;
      b.on = true;
    }
    scales_of(b, head);
    return b;
  };
  int head = st.seg / st.blocks;
  Batch now = batch_from(0, head), ahead = now;  // of the arithmetic's steps and the next ones
  if (st.n_steps > 16) ahead = batch_from(16, head);
  Batch copies = now;
  int f_seg = st.seg, f_step = 0, f_slot = ring.slot;
  int64_t f_base = head * head_bytes;  // of the head that is being fetched
  const auto fetch = [&]() {
    if (f_seg >= st.seg_end || st.n_steps == 0) return;
    if (f_step > 0 && (f_step & 15) == 0) copies = ahead;
    if (lane / 2 == (f_step & 15)) {
      uint64_t* const bar = ring.full + f_slot;
      if (copies.on) {
        uint8_t* const stage = ring.data + f_slot * R::kStage + (lane & 1) * R::kGroup;
        const int64_t at = copies.at + f_base;
        mbar_arrive_expect_tx(bar, 2 * R::kGroup);
        bulk_load(stage, a.k + at, R::kGroup, bar);
        bulk_load(stage + 2 * R::kGroup, a.v + at, R::kGroup, bar);
      } else {
        mbar_arrive(bar);
      }
    }
    f_slot = f_slot + 1 == ring.stages ? 0 : f_slot + 1;
    if (++f_step == st.n_steps) {
      f_step = 0;
      f_seg += W;
      f_base = f_seg / st.blocks * head_bytes;
    }
  };
#pragma unroll 1
  for (int i = 0; i < ring.stages - 1; ++i) fetch();
  RawQ<D, NT> raw;
  load_q<D, NT>(a, q.t0, q.n_rows, st.seg % st.blocks * kRows<NT>, head, raw);
  int limit[kTiles<NT>][2], least = st.len;
  for (int seg = st.seg; seg < st.seg_end; seg += W) {
    const int row0 = (seg - head * st.blocks) * kRows<NT>;
    const int next_head = (seg + W) / st.blocks;
    // what each row sees; rows past the last see everything and are not stored.
    // The same in every head, so only several row blocks need it again.
    if (seg == st.seg || st.blocks > 1) {
      least = st.len;
#pragma unroll
      for (int t = 0; t < kTiles<NT>; ++t)
#pragma unroll
        for (int c = 0; c < kCols<NT>; ++c) {
          const int row = row0 + row_in<NT>(t, quad, c);
          limit[t][c] = INT32_MAX;
          if (row < q.n_rows) {
            const int p = a.positions[q.t0 + row / a.group];
            limit[t][c] = max(0, min(p < INT32_MAX ? p + 1 : p, q.len));
            least = min(least, limit[t][c]);
          }
        }
      least = min(least, __shfl_xor_sync(0xffffffffu, least, 1));
      least = min(least, __shfl_xor_sync(0xffffffffu, least, 2));
    }
    uint32_t qb[kTiles<NT>][D / 16][2];
    float factor[kTiles<NT>][2];
    convert_q<D, NT>(a, raw, qb, factor);
    if (seg != st.seg) now = ahead;
    if (seg + W < st.seg_end) {
      // the next segment's rows and scales, a segment ahead
      load_q<D, NT>(a, q.t0, q.n_rows, (seg + W - next_head * st.blocks) * kRows<NT>, next_head, raw);
      scales_of(ahead, next_head);
    }
    TileState<D, NT> s;
    reset(s);
    for (int step = 0; step < st.n_steps; ++step) {
      if (step > 0 && (step & 15) == 0) {
        now = ahead;
        if (step + 16 < st.n_steps) ahead = batch_from(step + 16, head);
      }
      __syncwarp();  // all lanes have read the stage that fetch fills again
      fetch();
      if (!__all_sync(0xffffffffu,
                      mbar_wait(ring.full + ring.slot, (ring.phases >> ring.slot) & 1u, a.wait_ns, ring.abort))) {
        if (lane == 0) report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
        // let the copies already in flight land: the stages from this one up to the next to be fetched
        int slot = ring.slot;
        do {
          volatile int never = 0;
          mbar_wait(ring.full + slot, (ring.phases >> slot) & 1u, kDrainNs, &never);
          slot = slot + 1 == ring.stages ? 0 : slot + 1;
        } while (slot != f_slot);
        return false;
      }
      ring.phases ^= 1u << ring.slot;
      const uint8_t* const stage = ring.data + ring.slot * R::kStage;
      ring.slot = ring.slot + 1 == ring.stages ? 0 : ring.slot + 1;
      const int from = 2 * (step & 15);
      const float ks[2] = {__shfl_sync(0xffffffffu, now.ks, from), __shfl_sync(0xffffffffu, now.ks, from + 1)};
      const float lvs[2] = {__shfl_sync(0xffffffffu, now.lvs, from), __shfl_sync(0xffffffffu, now.lvs, from + 1)};
      const float ivs[2] = {__shfl_sync(0xffffffffu, now.ivs, from), __shfl_sync(0xffffffffu, now.ivs, from + 1)};
      step32<FMT, D, NT>(s, qb, factor, stage, ks, lvs, ivs, st.j_first + step * st.j_stride, limit, least, st.len);
    }
    __syncwarp();
#pragma unroll
    for (int t = 0; t < kTiles<NT>; ++t)
#pragma unroll
      for (int c = 0; c < kCols<NT>; ++c) {
#pragma unroll
        for (int d = 4; d <= 16; d *= 2) s.sum[t][c] += __shfl_xor_sync(0xffffffffu, s.sum[t][c], d);
        if (s.sum[t][c] == 0.0f) s.n[t][c] = -INFINITY;  // nothing seen
      }
    emit(s, head, row0);
    head = next_head;
  }
  return true;
}

template <int FMT, int D, int NT, int W>
__global__ void __launch_bounds__(32 * W, W > kAttWarps ? 1 : NT <= 1 ? (D == 64 ? 4 : 3) : D == 64 ? 3 : 2)
    attention_kernel(const AttArgs a, float* partial, Piece* pieces, int given_split, int stages) {
  const int split = W > kAttWarps ? kEach : given_split;
  using R = Ring<D>;
  extern __shared__ __align__(16) uint8_t ring_all[];
  const int ring_bytes = stages * R::kStage;  // of a warp
  int64_t* const start = reinterpret_cast<int64_t*>(ring_all + W * ring_bytes);
  __shared__ int64_t warp_sum[W];
  __shared__ uint64_t full[W][R::kMost];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, quad = lane & 3;
  Ring<D> ring = {stages, ring_all + warp * ring_bytes, full[warp], &abort_flag, 0, 0};
  if (tid == 0) abort_flag = 0;
  if (lane < stages) mbar_init(full[warp] + lane, lane == 0 ? 2 + a.stall : 2);
  mbar_fence_init();
  grid_dependency_wait();
  scan_requests<NT, W>(a, start, warp_sum, split);
  const int64_t all = start[a.n_requests];
  // at least a unit for each CTA that works, so that every CTA between a cut
  // segment's first and last has a part of it
  const int64_t cta = blockIdx.x, n_ctas = min(static_cast<int64_t>(gridDim.x), all);
  const int64_t end = cta < n_ctas ? cut_at<W>(a, start, cta + 1, n_ctas, split) : 0;
  int64_t pos = cta < n_ctas ? cut_at<W>(a, start, cta, n_ctas, split) : 0;
  if (tid == 0) pieces[cta].last_cta = -1;
  // requests without cached tokens, and tokens of no request
  for (int r = blockIdx.x; r < a.n_requests; r += gridDim.x) {
    const Request q = request(a, r);
    if (q.len == 0 && q.n_rows <= a.chunk_rows)
      for (int t = 0; t < q.n_rows / a.group; ++t) zero_row<D>(a, q.t0 + t, tid, (32 * W));
  }
  for (int t = min(max(a.cu_q[a.n_requests], 0), a.n_tokens) + blockIdx.x; t < a.n_tokens; t += gridDim.x)
    zero_row<D>(a, t, tid, (32 * W));

  int turn = 0;  // of the warps at whole segments
  bool ok = true;  // no wait of this warp has expired
  while (pos < end) {
    const int r = request_at(start, a.n_requests, pos);
    const Request q = request(a, r);
    const int units = units_of<W>(q), blocks = row_blocks_of<NT>(q);
    const int span = split == kEach ? 1 : units;
    const int64_t seg0 = (pos - start[r]) / span;
    const int unit0 = static_cast<int>((pos - start[r]) % span);
    Stream st;
    st.table = a.block_table + static_cast<int64_t>(r) * a.max_blocks;
    st.len = q.len;
    const int64_t left = static_cast<int64_t>(blocks) * a.heads - seg0;
    const int count = static_cast<int>(min(left, (end - pos) / span));
    const int steps = (q.len + kAttStep - 1) / kAttStep;
    if (unit0 == 0 && steps <= kWarpSteps && count >= W) {
      // short segments that lie whole in this piece: each warp takes every W-th
      st.j_first = 0;
      st.j_stride = kAttStep;
      st.n_steps = steps;
      st.seg = static_cast<int>(seg0) + ((warp - turn) & (W - 1));
      st.seg_end = static_cast<int>(seg0) + count;
      st.blocks = blocks;
      turn += count;
      pos += static_cast<int64_t>(count) * span;
      ok = ok && run_stream<FMT, D, NT, W>(a, st, q, ring, [&](TileState<D, NT>& s, int head, int row0) {
#pragma unroll
        for (int t = 0; t < kTiles<NT>; ++t)
#pragma unroll
          for (int c = 0; c < kCols<NT>; ++c) {
            const int row = row0 + row_in<NT>(t, quad, c);
            if (row >= q.n_rows) continue;
#pragma unroll
            for (int i0 = 0; i0 < D / 8; i0 += 8) {
              float o[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = s.acc[t][(i0 + i) / 2][2 * (i & 1) + c];
              store_row<D>(a, q.t0, row, head, (D / 8) * g + i0, s.n[t][c], s.sum[t][c], o);
            }
          }
      });
      continue;
    }
    const int n_units =
        split == kEach ? units : static_cast<int>(min(static_cast<int64_t>(units - unit0), end - pos));
    pos += split == kEach ? 1 : n_units;
    st.j_first = unit0 * (kAttStep * W) + warp * kAttStep;
    st.j_stride = (kAttStep * W);
    const int seen = min(n_units * (kAttStep * W), q.len - unit0 * (kAttStep * W)) - warp * kAttStep;
    st.n_steps = seen > 0 ? (seen + (kAttStep * W) - 1) / (kAttStep * W) : 0;
    st.seg = static_cast<int>(seg0);
    st.seg_end = st.seg + 1;
    st.blocks = blocks;
    // the warps' results of the tile, joined in warp order; they take the ring's place
    ok = ok && run_stream<FMT, D, NT, W>(a, st, q, ring, [&](TileState<D, NT>& s, int, int row0) {
      float* const mine = reinterpret_cast<float*>(ring.data);
#pragma unroll
      for (int t = 0; t < kTiles<NT>; ++t)
#pragma unroll
        for (int c = 0; c < kCols<NT>; ++c) {
          const int row = row_in<NT>(t, quad, c);
          if (row0 + row >= q.n_rows) continue;
          float* const at = mine + row * (D + 4);
          if (g == 0) at[D] = s.n[t][c], at[D + 1] = s.sum[t][c];
#pragma unroll
          for (int i = 0; i < D / 8; ++i) at[(D / 8) * g + i] = s.acc[t][i / 2][2 * (i & 1) + c];
        }
    });
    if (__syncthreads_or(!ok)) return;
    const int head = st.seg / blocks, row0 = st.seg % blocks * kRows<NT>;
    constexpr int kLanes = D / 8;
    const bool complete = n_units == units;
    // a cut segment's part: slot 1 where it starts here, slot 0 where it came from the CTA before
    float* const out = partial + (2 * cta + (unit0 == 0 ? 1 : 0)) * partial_floats<D>();
    if (unit0 == 0 && !complete && tid == 0) {
      // cuts inside a segment that may be cut are where the even split puts
      // them, so the CTA of its last unit follows from the split alone
      const int64_t seg_end = pos + (units - n_units);
      pieces[cta] = {q.t0, q.n_rows, row0, head, static_cast<int32_t>((seg_end * n_ctas - 1) / all), {0, 0, 0}};
    }
    for (int row = tid / kLanes; row < min(kRows<NT>, q.n_rows - row0); row += 32 * W / kLanes) {
      const int d0 = (tid % kLanes) * 8;
      float n = -INFINITY, sum = 0.0f, o[8] = {};
#pragma unroll
      for (int w = 0; w < W; ++w)
        n = fmaxf(n, reinterpret_cast<const float*>(ring_all + w * ring_bytes)[row * (D + 4) + D]);
      if (n > -INFINITY) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float* at = reinterpret_cast<const float*>(ring_all + w * ring_bytes) + row * (D + 4);
          const float f = exp2_fast(at[D] - n);
          sum += at[D + 1] * f;
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += at[d0 + i] * f;
        }
      }
      if (complete) {
        store_row<D>(a, q.t0, row0 + row, head, d0, n, sum, o);
      } else {
        float* const to = out + row * (D + 4);
        *reinterpret_cast<float4*>(to + d0) = make_float4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<float4*>(to + d0 + 4) = make_float4(o[4], o[5], o[6], o[7]);
        if (d0 == 0) *reinterpret_cast<float4*>(to + D) = make_float4(n, sum, 0.0f, 0.0f);
      }
    }
    fence_async_shared();  // the results' place is the copies' again
    __syncthreads();
  }
}

// Adds a cut segment's parts: a CTA for each row of a segment that starts in one
// CTA of attention_kernel and goes on in others.  Teams of D / 8 lanes take the
// parts in turn, eight loads of each lane in flight, and are added in order.
constexpr int kTeams = 16;
template <int D, int NT>
__global__ void __launch_bounds__(kTeams * D / 8) join_kernel(const AttArgs a, const float* partial, const Piece* pieces) {
  constexpr int kLanes = D / 8, kMost = 8;
  __shared__ float sh_o[kTeams][D + 4], sh_n[kTeams], sh_sum[kTeams];
  grid_dependency_wait();
  const int cta = blockIdx.x, row = blockIdx.y, tid = threadIdx.x;
  const Piece p = pieces[cta];
  if (p.last_cta <= cta || p.row0 + row >= p.n_rows) return;
  const int team = tid / kLanes, d0 = (tid % kLanes) * 8;
  float n = -INFINITY, sum = 0.0f, o[8] = {};
  for (int c0 = cta + team; c0 <= p.last_cta; c0 += kTeams * kMost) {
    float4 lo[kMost], hi[kMost];
    float2 st[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int c = c0 + i * kTeams;
      st[i] = make_float2(-INFINITY, 0.0f);
      lo[i] = hi[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (c <= p.last_cta) {
        const float* const at =
            partial + (2 * static_cast<int64_t>(c) + (c == cta ? 1 : 0)) * partial_floats<D>() + row * (D + 4);
        st[i] = *reinterpret_cast<const float2*>(at + D);
        lo[i] = *reinterpret_cast<const float4*>(at + d0);
        hi[i] = *reinterpret_cast<const float4*>(at + d0 + 4);
      }
    }
    float m = n;
#pragma unroll
    for (int i = 0; i < kMost; ++i) m = fmaxf(m, st[i].x);
    if (m == -INFINITY) continue;
    const float f0 = exp2_fast(n - m);
    n = m;
    sum *= f0;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= f0;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const float f = exp2_fast(st[i].x - m);
      sum += st[i].y * f;
      o[0] += lo[i].x * f, o[1] += lo[i].y * f, o[2] += lo[i].z * f, o[3] += lo[i].w * f;
      o[4] += hi[i].x * f, o[5] += hi[i].y * f, o[6] += hi[i].z * f, o[7] += hi[i].w * f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sh_o[team][d0 + i] = o[i];
  if (d0 == 0) sh_n[team] = n, sh_sum[team] = sum;
  __syncthreads();
  if (team > 0) return;
  n = -INFINITY;
#pragma unroll
  for (int w = 0; w < kTeams; ++w) n = fmaxf(n, sh_n[w]);
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.0f;
  if (n > -INFINITY) {
#pragma unroll
    for (int w = 0; w < kTeams; ++w) {
      const float f = exp2_fast(sh_n[w] - n);
      sum += sh_sum[w] * f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += sh_o[w][d0 + i] * f;
    }
  }
  store_row<D>(a, p.t0, p.row0 + row, p.head, d0, n, sum, o);
}

template <int FMT, int D, int NT>
int launch_attention(const AttArgs& a, int max_kv_len, int max_q_len, void* workspace, cudaStream_t s) {
  float* const partial = static_cast<float*>(workspace);
  Piece* const pieces = reinterpret_cast<Piece*>(partial + 2 * kMaxCtas * partial_floats<D>());
  const size_t sums = sizeof(int64_t) * (static_cast<size_t>(a.n_requests) + 1);
  // no more CTAs than the units that the caller's bounds allow
  const int64_t blocks = (static_cast<int64_t>(max_q_len) * a.group + kRows<NT> - 1) / kRows<NT>;
  const int64_t units = (static_cast<int64_t>(max_kv_len) + kUnit - 1) / kUnit;
  // Cutting evens out the CTAs' loads and costs the join and the search for the cuts.  A
  // segment with an SM to itself takes 5.7 us and 0.57 more a unit (8 warps share its steps), cut segments
  // 8 to 18 us and, by how many there are, 0.07 to 0.44 a unit: about even at units = segments / 2
  // (heads of 128, blocks of 8 rows, 128 segments of up to 1000 tokens: 10.8 us, cut 20; of 4000 26.1 and 32.2, of 9000
  // 49 and 50; 32 segments of 1500: 12.8 and 13.1, of 4000 24.1 and 18.1; 8 of 4000: 23.8 and 10.6).
  // More segments than SMs: whole ones are better up to 16 units (256 segments of 1500 tokens 26.0, cut 30.1;
  // of 2500 38.3 and 36.7), and up to 32 where there are so many that they even out
  // (8000 of up to 4001, 32 units, 143 and 146: little, and the one size that was measured); beyond, one long segment
  // among short ones would be all a CTA's work.  All but 16 x 1000 and 16 x 4000 measured with blocks of 8 rows.
  const int64_t segments = a.n_requests * a.heads * std::max<int64_t>(1, blocks);
  const int64_t sms = sm_count();
  const int split = segments <= sms ? 2 * units <= std::max<int64_t>(8, segments) ? kEach : kCut
                    : units <= (segments >= 8 * sms ? 32 : 16) ? kWhole : kCut;
  const int warps = split == kEach ? kWideWarps : kAttWarps;
  const auto kernel = split == kEach ? attention_kernel<FMT, D, NT, kWideWarps> : attention_kernel<FMT, D, NT, kAttWarps>;
  const void* fn = reinterpret_cast<const void*>(kernel);
  KV_TRY(set_max_dynamic_smem(fn, kMaxSmem));
  const int stage_bytes = warps * Ring<D>::kStage;
  const int resident = resident_ctas_per_sm(fn, 32 * warps, Ring<D>::kLeast * stage_bytes + sums);
  if (resident < 1) return TWELL_ERR_CUDA;
  const int64_t most = std::max<int64_t>(1, split == kEach ? segments : segments * std::max<int64_t>(1, units));
  const int ctas = static_cast<int>(std::min<int64_t>(most, std::min(kMaxCtas, sm_count() * resident)));
  // where fewer CTAs share an SM each has more of its shared memory: more copies ahead
  const int share = (ctas + sm_count() - 1) / sm_count();
  const int stages = std::min<int>(Ring<D>::kMost, std::max<int>(Ring<D>::kLeast, static_cast<int>(
      (kMaxSmem / share - static_cast<int>(sums) - 2048) / stage_bytes)));
  const size_t smem = static_cast<size_t>(stages) * stage_bytes + sums;
  {
    LaunchScope scope(TWELL_KERNEL_KV_ATTENTION, s);
    if (launch_pdl(kernel, dim3(ctas), dim3(32 * warps), smem, s, a, partial, pieces, split, stages) != cudaSuccess)
      return TWELL_ERR_CUDA;
  }
  if (split != kCut || ctas == 1) return TWELL_OK;
  const int rows = static_cast<int>(std::min<int64_t>(kRows<NT>, static_cast<int64_t>(a.n_tokens) * a.group));
  LaunchScope scope(TWELL_KERNEL_KV_JOIN, s);
  return launch_pdl(join_kernel<D, NT>, dim3(ctas - 1, rows), dim3(kTeams * D / 8), 0, s, a,
                    static_cast<const float*>(partial), static_cast<const Piece*>(pieces)) == cudaSuccess
             ? TWELL_OK
             : TWELL_ERR_CUDA;
}

template <int FMT>
int launch_dim(const AttArgs& a, int dim, int max_kv_len, int max_q_len, void* workspace, cudaStream_t s) {
  // Row blocks of 16 where a request has more than 8 rows: the codes' conversion is then shared by
  // twice the rows.  Blocks of 4 where none has more: a lane's second column stays empty
  // and half the exponentials go (250 ragged requests with a row each 143 -> 136 us, 4 x 131072 tokens with 4 134 -> 130).
  const int64_t rows = static_cast<int64_t>(std::max(max_q_len, 1)) * a.group;
  const auto fn = dim == 64 ? rows <= 4   ? launch_attention<FMT, 64, 0>
                              : rows <= 8 ? launch_attention<FMT, 64, 1>
                                          : launch_attention<FMT, 64, 2>
                  : rows <= 4 ? launch_attention<FMT, 128, 0>
                  : rows <= 8 ? launch_attention<FMT, 128, 1>
                              : launch_attention<FMT, 128, 2>;
  return fn(a, max_kv_len, max_q_len, workspace, s);
}

size_t decode_workspace_bytes(int dim) {
  return (2 * kMaxCtas * static_cast<size_t>(kMaxRows) * (dim + 4) * sizeof(float) + kMaxCtas * sizeof(Piece) + 255) /
         256 * 256;
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
  const int64_t rows = static_cast<int64_t>(n_tokens) * (n_q_heads / n_kv_heads);
  return decode_workspace_bytes(head_dim) + (chunk_workspace_bytes(rows, head_dim) + 255) / 256 * 256;
}

namespace {

int kv_attention(const uint16_t* Q, int64_t ldq, const twell_kv_t* cache, const int32_t* block_table,
                 int32_t max_blocks, const int32_t* cu_q, const int32_t* positions, const int32_t* kv_lens,
                 int32_t n_tokens, int32_t n_requests, int32_t n_q_heads, int32_t max_kv_len, int32_t max_q_len,
                 float softmax_scale, uint16_t* O, int64_t ldo, float* lse, void* workspace, size_t workspace_bytes,
                 twell_stream_t stream, int stall, uint64_t wait_ns) {
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
  a.chunk_rows = INT32_MAX;
  a.stall = stall;
  a.wait_ns = wait_ns;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n_requests > 0 && static_cast<int64_t>(max_q_len) * a.group > kChunkRows) {
    a.chunk_rows = kChunkRows;
    KV_TRY(launch_chunk_attention(a, cache->format, cache->head_dim, max_kv_len,
                                  static_cast<uint8_t*>(workspace) + decode_workspace_bytes(cache->head_dim), s));
  }
  return cache->format == TWELL_KV_E4M3 ? launch_dim<TWELL_KV_E4M3>(a, cache->head_dim, max_kv_len, max_q_len, workspace, s)
                                        : launch_dim<TWELL_KV_INT8>(a, cache->head_dim, max_kv_len, max_q_len, workspace, s);
}

}  // namespace

extern "C" TWELL_API int twell_kv_attention(const uint16_t* Q, int64_t ldq, const twell_kv_t* cache,
                                            const int32_t* block_table, int32_t max_blocks, const int32_t* cu_q,
                                            const int32_t* positions, const int32_t* kv_lens, int32_t n_tokens,
                                            int32_t n_requests, int32_t n_q_heads, int32_t max_kv_len,
                                            int32_t max_q_len, float softmax_scale, uint16_t* O, int64_t ldo,
                                            float* lse, void* workspace, size_t workspace_bytes,
                                            twell_stream_t stream) {
  return kv_attention(Q, ldq, cache, block_table, max_blocks, cu_q, positions, kv_lens, n_tokens, n_requests, n_q_heads,
                      max_kv_len, max_q_len, softmax_scale, O, ldo, lse, workspace, workspace_bytes, stream, 0,
                      kWaitLimitNs);
}

extern "C" TWELL_API int twell_selftest_kv_attention_stall(
    const uint16_t* Q, int64_t ldq, const twell_kv_t* cache, const int32_t* block_table, int32_t max_blocks,
    const int32_t* cu_q, const int32_t* positions, const int32_t* kv_lens, int32_t n_tokens, int32_t n_requests,
    int32_t n_q_heads, int32_t max_kv_len, int32_t max_q_len, float softmax_scale, uint16_t* O, int64_t ldo, float* lse,
    void* workspace, size_t workspace_bytes, uint64_t limit_ns, twell_stream_t stream) {
  if (limit_ns < 100000ull || limit_ns > 1000000000ull) return TWELL_ERR_INVALID_ARG;
  return kv_attention(Q, ldq, cache, block_table, max_blocks, cu_q, positions, kv_lens, n_tokens, n_requests, n_q_heads,
                      max_kv_len, max_q_len, softmax_scale, O, ldo, lse, workspace, workspace_bytes, stream, 1,
                      limit_ns);
}
