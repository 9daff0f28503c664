// Log probabilities of tokens from hidden rows H [N][d] and output weights
// W [V][d] (twell_linear_logprobs) and their gradient (..._bwd): the logits
// x = H W^T / T live in tensor memory only, a tile at a time.
//
// Forward: each 128 x 256 tile of x leaves a row's maximum m, S = sum 2^(y - m)
// and U = sum 2^(y - m) (y - m) over the tile's columns, y = x log2(e); a second
// kernel joins the tiles of a row:
//   lse = ln2 (m + log2 S),  logprob = x_t - lse,  entropy = ln2 (log2 S - U / S).
// Backward, in pieces of the vocabulary: x again, from it
//   G = (g (1[t] - p) - ge p (log p + entropy)) / T,  p = exp(x - lse),
// as bf16 into the workspace (the tensor cores take bf16, and each entry is then
// off by 2^-9 of itself on average, as the bf16 results are), then
// dH += G W_piece and dW_piece = G^T H with fp32 sums.  A launch runs the products
// of one piece together with G of the next one, which needs a buffer of its own.
//
// All products are tiles of one persistent kernel on the 5th-generation tensor cores:
// operands by TMA into 128-byte swizzled stages, accumulators twice in TMEM, one
// warp for the copies, one for the MMAs, eight for the epilogue.  The two gradient products read
// G and H or W along their rows, so those operands go in M- or N-major.
#include <algorithm>

#include "kv_internal.h"

namespace twell {
namespace {

constexpr int kBM = 128, kBN = 256, kBK = 64, kUmmaK = 16;
constexpr int kStages = 4;
constexpr int kThreads = 384, kEpiThreads = 256;
constexpr uint32_t kABytes = kBM * kBK * 2, kBBytes = kBN * kBK * 2;
constexpr uint32_t kPipeBytes = kStages * (kABytes + kBBytes);
constexpr uint32_t kBarBytes = 256;
constexpr uint32_t kEpiBytes = 2 * 128 * 3 * sizeof(float);  // one half's sums, for the other half
constexpr uint32_t kSmemBytes = 1024 + kPipeBytes + kBarBytes + kEpiBytes;
constexpr int kMaxJobs = 3;
constexpr int kPlanSms = 152;            // plans do not depend on the device, workspaces neither
constexpr int64_t kPieceBytes = 1 << 27; // of G: what the L2 cache can hold
constexpr int kMinPiece = 4096;          // columns; dH's sums are read and written once a piece
constexpr int kMaxKSplit = 32;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

enum JobType { kJobSums, kJobGrad, kJobDHidden, kJobDWeight };

// One product C[M][N] = A . B^T in tiles, K cut into ksplit ranges.
struct Job {
  int type;
  int m, n;                 // rows and columns of C
  int num_m, num_n, num_k;  // tiles, steps of K
  int ksplit;
  int col0;                 // first vocabulary column of the piece
  int units;
  int a_mn, b_mn;           // operand stored [K][M] / [K][N]
  int add, round;           // dH: earlier pieces have left sums; these are the last
};

struct Maps {
  CUtensorMap a[kMaxJobs], b[kMaxJobs];
};

struct Args {
  Job job[kMaxJobs];
  int num_jobs;
  int n_rows, d_model, vocab;
  const int32_t* targets;
  float inv_t;
  // forward
  float* part;        // [3][num_n][n_rows]: m, S, U
  float* of_target;   // [n_rows] x of the target
  // backward
  const float *lse, *entropy, *g, *ge;
  uint16_t* grad;     // G of the piece: [n_rows][ld_grad]
  int64_t ld_grad;
  float* dh_sum;      // [ksplit][n_rows][d_model]
  uint16_t* dh;
  uint16_t* dw;
  int64_t lddh, lddw;
  int32_t* status;
  uint64_t wait_limit_ns;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Element i of 32, by a tree of selections (an indexed array would go to local memory).
__device__ __forceinline__ float pick(const uint32_t (&r)[32], int i) {
  uint32_t a[16], b[8], c[4], d[2];
#pragma unroll
  for (int k = 0; k < 16; ++k) a[k] = (i & 16) ? r[k + 16] : r[k];
#pragma unroll
  for (int k = 0; k < 8; ++k) b[k] = (i & 8) ? a[k + 8] : a[k];
#pragma unroll
  for (int k = 0; k < 4; ++k) c[k] = (i & 4) ? b[k + 4] : b[k];
#pragma unroll
  for (int k = 0; k < 2; ++k) d[k] = (i & 2) ? c[k + 2] : c[k];
  return __uint_as_float((i & 1) ? d[1] : d[0]);
}

// A row's running sums in base 2 relative to m (as y = acc c).
struct Sums {
  float m = -INFINITY, s = 0.0f, u = 0.0f;
  // joins sums that are relative to m2
  __device__ __forceinline__ void join(float m2, float s2, float u2) {
    const float top = fmaxf(m, m2);
    if (top == -INFINITY) {  // neither has an entry above -inf: S is 0, or NaN where there was one
      s += s2, u += u2;
      return;
    }
    // a side without entries has S = U = 0 and m = -inf: its factor is 0, and so is its shift times S
    const float d1 = fmaxf(m - top, -1e30f), d2 = fmaxf(m2 - top, -1e30f);
    const float f1 = ex2(d1), f2 = ex2(d2);
    u = f1 * fmaf(d1, s, u) + f2 * fmaf(d2, s2, u2);
    s = f1 * s + f2 * s2;
    m = top;
  }
};

struct Tile {
  int row, col0;     // this thread's row, the tile's first column
  uint32_t taddr;
  int half, lg;      // column half, lane quarter
  bool valid;        // the row exists
};

// Sums of the tile's columns; both halves of a row are joined through shared memory.
__device__ __forceinline__ void epilogue_sums(const Args& a, const Job& j, const Tile& t, int n_blk, float* shared,
                                              int turn) {
  const float c = a.inv_t * kLog2e;
  const int target = t.valid && a.targets ? a.targets[t.row] : -1;
  Sums all;
#pragma unroll 1
  for (int k = t.half * (kBN / 2); k < (t.half + 1) * (kBN / 2); k += 32) {
    uint32_t r[32];
    tmem_ld32(t.taddr + k, r);
    tmem_ld_wait();
    const int col = t.col0 + k, left = j.n - col;
    if (left <= 0) break;  // the same for all threads of the CTA
    if (left < 32) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i >= left) r[i] = 0xFF800000u;
    }
    if (target >= col && target < col + 32) a.of_target[t.row] = pick(r, target - col) * a.inv_t;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = fmaxf(top, __uint_as_float(r[i]));
    const float m = top * c, ref = m == -INFINITY ? 0.0f : m;
    float s = 0.0f, u = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float y = fmaf(__uint_as_float(r[i]), c, -ref), e = ex2(y);
      s += e;
      u = fmaf(e, fmaxf(y, -1e30f), u);  // 0 for an entry of -inf
    }
    all.join(m, s, u);
  }
  float* const at = shared + turn * 128 * 3 + (t.lg * 32 + (threadIdx.x & 31)) * 3;
  if (t.half == 1) at[0] = all.m, at[1] = all.s, at[2] = all.u;
  asm volatile("bar.sync %0, 64;" ::"r"(t.lg + 1) : "memory");
  if (t.half == 1 || !t.valid) return;
  all.join(at[0], at[1], at[2]);
  const int64_t plane = static_cast<int64_t>(j.num_n) * a.n_rows;
  float* const out = a.part + static_cast<int64_t>(n_blk) * a.n_rows + t.row;
  out[0] = all.m, out[plane] = all.s, out[2 * plane] = all.u;
}

// G of the tile as bf16.
__device__ __forceinline__ void epilogue_grad(const Args& a, const Job& j, const Tile& t) {
  float lse = 0.0f, a0 = 0.0f, a1 = 0.0f, g = 0.0f;
  int target = -1;
  if (t.valid) {
    lse = a.lse[t.row];
    if (a.targets) {
      target = a.targets[t.row];
      if (target >= 0 && target < a.vocab) g = a.inv_t * a.g[t.row];
    }
    a0 = -g;
    if (a.ge) {
      a1 = -a.inv_t * a.ge[t.row];
      a0 = fmaf(a1, a.entropy[t.row], a0);
    }
    if (lse == -INFINITY) lse = 0.0f, a0 = 0.0f, a1 = 0.0f, g = 0.0f;  // a row of -inf only: zeros
  }
#pragma unroll 1
  for (int k = t.half * (kBN / 2); k < (t.half + 1) * (kBN / 2); k += 32) {
    uint32_t r[32];
    tmem_ld32(t.taddr + k, r);
    tmem_ld_wait();
    const int col = t.col0 + k;
    if (col >= j.n) break;
    const int own = target - j.col0 - col;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float q[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = fmaf(__uint_as_float(r[i + e]), a.inv_t, -lse);
        q[e] = ex2(x * kLog2e) * fmaf(a1, fmaxf(x, -1e30f), a0) + (own == i + e ? g : 0.0f);
      }
      w[i / 2] = bf16_pair(q[0], q[1]);
    }
    if (!t.valid) continue;
    // rows of G are a multiple of 256 columns apart: what lies past the piece is never read
    uint4* const out = reinterpret_cast<uint4*>(a.grad + t.row * a.ld_grad + col);
#pragma unroll
    for (int q = 0; q < 4; ++q) out[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  }
}

// bf16 rows of a gradient; dH adds what earlier pieces left, and keeps fp32 until the last one.
__device__ __forceinline__ void epilogue_store(const Args& a, const Job& j, const Tile& t, int ks) {
  const bool dh = j.type == kJobDHidden;
  float* const sum =
      dh ? a.dh_sum + (static_cast<int64_t>(ks) * a.n_rows + t.row) * a.d_model + t.col0 : nullptr;
  uint16_t* const out = dh ? a.dh + t.row * a.lddh + t.col0 : a.dw + (t.row + static_cast<int64_t>(j.col0)) * a.lddw + t.col0;
  const bool add = dh && j.add, round = !dh || j.round;
#pragma unroll 1
  for (int k = t.half * (kBN / 2); k < (t.half + 1) * (kBN / 2); k += 32) {
    uint32_t r[32];
    tmem_ld32(t.taddr + k, r);
    tmem_ld_wait();
    if (t.col0 + k >= j.n) break;
    if (!t.valid) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (t.col0 + k + 8 * q >= j.n) break;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(r[8 * q + e]);
      float4* const at = reinterpret_cast<float4*>(sum + k + 8 * q);
      if (add) {
        const float4 x = at[0], y = at[1];
        f[0] += x.x, f[1] += x.y, f[2] += x.z, f[3] += x.w, f[4] += y.x, f[5] += y.y, f[6] += y.z, f[7] += y.w;
      }
      if (round) {
        *reinterpret_cast<uint4*>(out + k + 8 * q) =
            make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
      } else {
        at[0] = make_float4(f[0], f[1], f[2], f[3]);
        at[1] = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
  }
}

struct Unit {
  int job, m_blk, n_blk, ks, kb0, kb1;
};

// The u-th tile of the launch: jobs one after the other, m fastest, so that CTAs working side by
// side share the columns' operand and all rows stay in L2.
__device__ __forceinline__ Unit unit_of(const Args& a, int u) {
  int i = 0;
  while (i + 1 < a.num_jobs && u >= a.job[i].units) u -= a.job[i++].units;
  const Job& j = a.job[i];
  Unit x;
  x.job = i;
  x.m_blk = u % j.num_m;
  u /= j.num_m;
  x.n_blk = u % j.num_n;
  x.ks = u / j.num_n;
  x.kb0 = static_cast<int>(static_cast<int64_t>(x.ks) * j.num_k / j.ksplit);
  x.kb1 = static_cast<int>(static_cast<int64_t>(x.ks + 1) * j.num_k / j.ksplit);
  return x;
}

__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a) {
  constexpr int S = kStages;
  grid_dependency_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const sA = smem;
  uint8_t* const sB = smem + S * kABytes;
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + kPipeBytes);
  uint64_t* const empty = full + S;
  uint64_t* const tfull = empty + S;
  uint64_t* const tempty = tfull + 2;
  uint64_t* const drain = tempty + 2;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* const abort = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* const issued = const_cast<int*>(abort) + 1;  // [S] parity of the last fill of each stage, -1: none
  float* const epi = reinterpret_cast<float*>(smem + kPipeBytes + kBarBytes);
  static_assert((2 * S + 5) * 8 + 8 + S * 4 <= static_cast<int>(kBarBytes), "barrier region");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int units = 0;
  for (int i = 0; i < a.num_jobs; ++i) units += a.job[i].units;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      issued[s] = -1;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kEpiThreads);
    }
    mbar_init(drain, 1);
    *abort = 0;
    mbar_fence_init();
  }
  if (warp == 0 && lane < 2 * a.num_jobs) tma_prefetch_desc(lane & 1 ? &maps.b[lane >> 1] : &maps.a[lane >> 1]);
  if (warp == 2) tmem_alloc(tmem_holder, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const uint64_t limit = a.wait_limit_ns;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- copies
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const Unit x = unit_of(a, u);
        const Job& j = a.job[x.job];
        const CUtensorMap* const ma = &maps.a[x.job];
        const CUtensorMap* const mb = &maps.b[x.job];
        for (int kb = x.kb0; kb < x.kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, limit, abort)) {
            ok = false;
            break;
          }
          uint8_t* const da = sA + stage * kABytes;
          uint8_t* const db = sB + stage * kBBytes;
          mbar_arrive_expect_tx(&full[stage], kABytes + kBBytes);
          if (j.a_mn) {  // [K][M]: boxes of 64 columns by 64 rows of K
#pragma unroll
            for (int q = 0; q < kBM / 64; ++q)
              tma_load_2d(da + q * 8192, ma, &full[stage], x.m_blk * kBM + q * 64, kb * kBK);
          } else {
            tma_load_2d(da, ma, &full[stage], kb * kBK, x.m_blk * kBM);
          }
          if (j.b_mn) {
#pragma unroll
            for (int q = 0; q < kBN / 64; ++q)
              tma_load_2d(db + q * 8192, mb, &full[stage], x.n_blk * kBN + q * 64, kb * kBK);
          } else {
            tma_load_2d(db, mb, &full[stage], kb * kBK, x.n_blk * kBN);
          }
          issued[stage] = static_cast<int>(phase);
          if (++stage == S) stage = 0, phase ^= 1u;
        }
      }
      if (!ok) {
        report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
        for (int s = 0; s < S; ++s)  // the copies in flight land before the CTA leaves
          if (issued[s] >= 0) {
            volatile int never = 0;
            mbar_wait(&full[s], static_cast<uint32_t>(issued[s]), 10000000ull, &never);
          }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- products
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const Unit x = unit_of(a, u);
        const Job& j = a.job[x.job];
        const uint32_t idesc = idesc_bf16_f32(kBM, kBN) | (j.a_mn ? 1u << 15 : 0u) | (j.b_mn ? 1u << 16 : 0u);
        // a step of 16 along K: 32 bytes of a K-major row, 16 rows of 128 bytes of the others
        const uint64_t a_step = j.a_mn ? 128u : 2u, b_step = j.b_mn ? 128u : 2u;
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, limit, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kBN);
        for (int kb = x.kb0; kb < x.kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, limit, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t pa = smem_u32(sA + stage * kABytes), pb = smem_u32(sB + stage * kBBytes);
          const uint64_t ad = j.a_mn ? smem_desc_sw128_nmajor(pa, 8192) : smem_desc_sw128(pa);
          const uint64_t bd = j.b_mn ? smem_desc_sw128_nmajor(pb, 8192) : smem_desc_sw128(pb);
#pragma unroll
          for (int k = 0; k < kBK / kUmmaK; ++k)
            mma_bf16(d, ad + k * a_step, bd + k * b_step, idesc, (kb > x.kb0 || k > 0) ? 1u : 0u);
          mma_commit(&empty[stage]);
          if (++stage == S) stage = 0, phase ^= 1u;
        }
        if (!ok) break;
        mma_commit(&tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) {
        report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
        mma_commit(drain);  // the MMAs already issued end before TMEM is released
        volatile int never = 0;
        mbar_wait(drain, 0, 10000000ull, &never);
      }
    }
  } else if (warp >= 4) {
    // ---------------- epilogue: thread = row of the tile (a TMEM lane), two warps share a row's columns
    Tile t;
    t.lg = warp & 3;
    t.half = (warp - 4) >> 2;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const Unit x = unit_of(a, u);
      const Job& j = a.job[x.job];
      if (!mbar_wait(&tfull[acc], acc_phase, limit, abort)) {
        report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
        break;
      }
      tc_fence_after();
      t.row = x.m_blk * kBM + t.lg * 32 + lane;
      t.col0 = x.n_blk * kBN;
      t.valid = t.row < j.m;
      t.taddr = tmem_base + (static_cast<uint32_t>(t.lg * 32) << 16) + static_cast<uint32_t>(acc * kBN);
      if (j.type == kJobSums)
        epilogue_sums(a, j, t, x.n_blk, epi, acc);
      else if (j.type == kJobGrad)
        epilogue_grad(a, j, t);
      else
        epilogue_store(a, j, t, x.ks);
      tc_fence_before();
      mbar_arrive(&tempty[acc]);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

struct JoinArgs {
  const float *part, *of_target;
  int num_n, n_rows, vocab;
  const int32_t* targets;
  float *logprob, *entropy, *lse;
};

// The tiles' sums of 32 rows: a lane a row, the warps take tiles in turn and are joined in order.
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(kJoinWarps * 32) linear_join_kernel(const JoinArgs a) {
  __shared__ float sh[kJoinWarps][3][32];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x * 32 + lane;
  Sums all;
  if (row < a.n_rows) {
    const int64_t plane = static_cast<int64_t>(a.num_n) * a.n_rows;
#pragma unroll 4
    for (int k = warp; k < a.num_n; k += kJoinWarps) {
      const float* const at = a.part + static_cast<int64_t>(k) * a.n_rows + row;
      all.join(at[0], at[plane], at[2 * plane]);
    }
  }
  sh[warp][0][lane] = all.m, sh[warp][1][lane] = all.s, sh[warp][2][lane] = all.u;
  __syncthreads();
  if (warp > 0 || row >= a.n_rows) return;
  for (int w = 1; w < kJoinWarps; ++w) all.join(sh[w][0][lane], sh[w][1][lane], sh[w][2][lane]);
  const float log_s = log2f(all.s), lse = kLn2 * (all.m + log_s);
  if (a.lse) a.lse[row] = lse;
  if (a.entropy) a.entropy[row] = all.s == 0.0f ? 0.0f : kLn2 * (log_s - all.u / all.s);
  if (a.logprob) {
    const int t = a.targets[row];
    // a row of -inf only: -inf, as all its log probabilities
    a.logprob[row] = t < 0 || t >= a.vocab ? 0.0f : all.s == 0.0f ? -INFINITY : a.of_target[row] - lse;
  }
}

struct ReduceArgs {
  const float* sum;
  int ksplit, n_rows, dim;
  uint16_t* out;
  int64_t ld;
};

// dH from the sums of K's ranges, added in order; 8 elements a thread.
__global__ void __launch_bounds__(256) linear_reduce_kernel(const ReduceArgs a) {
  grid_dependency_wait();
  const int64_t vecs = a.dim / 8, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= vecs * a.n_rows) return;
  const int64_t row = i / vecs, c = i % vecs * 8, plane = static_cast<int64_t>(a.n_rows) * a.dim;
  const float* const at = a.sum + row * a.dim + c;
  float f[8] = {};
  for (int k = 0; k < a.ksplit; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(at + k * plane), y = *reinterpret_cast<const float4*>(at + k * plane + 4);
    f[0] += x.x, f[1] += x.y, f[2] += x.z, f[3] += x.w, f[4] += y.x, f[5] += y.y, f[6] += y.z, f[7] += y.w;
  }
  *reinterpret_cast<uint4*>(a.out + row * a.ld + c) =
      make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }
size_t round_up(size_t x, size_t to) { return (x + to - 1) / to * to; }

// How a backward call is cut.
struct Plan {
  int pieces, piece;  // columns of a piece, a multiple of 256
  int ksplit;         // ranges of the vocabulary in dH's product of a piece
  size_t grad_bytes, sum_bytes, bytes;
};

Plan plan_bwd(int64_t n_rows, int64_t d, int64_t vocab) {
  Plan p;
  const int64_t most = std::max<int64_t>(kMinPiece, kPieceBytes / (2 * std::max<int64_t>(n_rows, 1)));
  p.pieces = ceil_div(vocab, most);
  p.piece = ceil_div(ceil_div(vocab, p.pieces), 256) * 256;
  p.pieces = ceil_div(vocab, p.piece);
  // dH's tiles have long sums: where they are few, K is cut so that none takes longer than a
  // CTA's share of the two products
  const int64_t num_k = ceil_div(std::min<int64_t>(p.piece, vocab), kBK);
  const int64_t dh = ceil_div(n_rows, kBM) * static_cast<int64_t>(ceil_div(d, kBN)) * num_k;
  const int64_t dw = ceil_div(std::min<int64_t>(p.piece, vocab), kBM) * static_cast<int64_t>(ceil_div(d, kBN)) *
                     ceil_div(n_rows, kBK);
  const int64_t share = std::max<int64_t>(8, (dh + dw) / kPlanSms);
  p.ksplit = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({num_k, kMaxKSplit, ceil_div(num_k, share)})));
  p.grad_bytes = round_up(static_cast<size_t>(n_rows) * p.piece * 2, 256);
  p.sum_bytes = p.pieces > 1 || p.ksplit > 1 ? round_up(static_cast<size_t>(p.ksplit) * n_rows * d * 4, 256) : 0;
  p.bytes = p.grad_bytes * (p.pieces > 1 ? 2 : 1) + p.sum_bytes + 256;
  return p;
}

size_t fwd_bytes(int64_t n_rows, int64_t vocab) {
  return round_up(static_cast<size_t>(n_rows) * 4 * (3 * ceil_div(vocab, kBN) + 1), 256) + 256;
}

// A: [m][k], or [k][m] with mn; likewise B.  rows of either lie ld elements apart.
int set_job(Maps* maps, Args* args, Job j, const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb, int k) {
  const int i = args->num_jobs++;
  j.num_m = ceil_div(j.m, kBM), j.num_n = ceil_div(j.n, kBN), j.num_k = ceil_div(k, kBK);
  j.ksplit = std::min(j.ksplit, j.num_k);
  const int64_t units = static_cast<int64_t>(j.num_m) * j.num_n * j.ksplit;
  if (units > (1 << 29)) return TWELL_ERR_UNSUPPORTED;
  j.units = static_cast<int>(units);
  args->job[i] = j;
  if (j.a_mn)
    KV_TRY(encode_tmap_2d(&maps->a[i], A, j.m, k, lda * 2, 64, kBK));
  else
    KV_TRY(encode_tmap_2d(&maps->a[i], A, k, j.m, lda * 2, kBK, kBM));
  if (j.b_mn) return encode_tmap_2d(&maps->b[i], B, j.n, k, ldb * 2, 64, kBK);
  return encode_tmap_2d(&maps->b[i], B, k, j.n, ldb * 2, kBK, kBN);
}

int launch_jobs(const Maps& maps, const Args& args, int kernel_id, cudaStream_t s) {
  KV_TRY(set_max_dynamic_smem(reinterpret_cast<const void*>(linear_kernel), static_cast<int>(kSmemBytes)));
  int64_t units = 0;
  for (int i = 0; i < args.num_jobs; ++i) units += args.job[i].units;
  const int grid = static_cast<int>(std::min<int64_t>(units, sm_count()));
  LaunchScope scope(kernel_id, s);
  return launch_pdl(linear_kernel, dim3(grid), dim3(kThreads), kSmemBytes, s, maps, args) == cudaSuccess
             ? TWELL_OK
             : TWELL_ERR_CUDA;
}

int check_linear(const uint16_t* H, int64_t ldh, const uint16_t* W, int64_t ldw, int n_rows, int d, int vocab,
                 float inv_t) {
  if (n_rows < 0 || d < 1 || vocab < 1) return TWELL_ERR_INVALID_ARG;
  if (!(inv_t > 0.0f) || inv_t > 3.0e38f) return TWELL_ERR_INVALID_ARG;
  if (d % 8 != 0) return TWELL_ERR_UNSUPPORTED;
  if (ldw < d || ldw % 8 != 0) return TWELL_ERR_INVALID_ARG;
  KV_TRY(check_array(W, 16));
  if (n_rows == 0) return TWELL_OK;
  if (ldh < d || ldh % 8 != 0) return TWELL_ERR_INVALID_ARG;
  return check_array(H, 16);
}

int check_vectors(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned_to(p, 4)) return TWELL_ERR_MISALIGNED;
  return TWELL_OK;
}

}  // namespace
}  // namespace twell

using namespace twell;

extern "C" TWELL_API size_t twell_linear_logprobs_workspace_bytes(int32_t n_rows, int32_t d_model, int32_t vocab) {
  if (n_rows < 0 || d_model < 8 || d_model % 8 != 0 || vocab < 1) return 0;
  return fwd_bytes(n_rows, vocab);
}

extern "C" TWELL_API int twell_linear_logprobs(const uint16_t* H, int64_t ldh, const uint16_t* W, int64_t ldw,
                                               int32_t n_rows, int32_t d_model, int32_t vocab, const int32_t* targets,
                                               float inv_temperature, float* logprob, float* entropy, float* lse,
                                               void* workspace, size_t workspace_bytes, int32_t* status,
                                               twell_stream_t stream) {
  KV_TRY(check_linear(H, ldh, W, ldw, n_rows, d_model, vocab, inv_temperature));
  KV_TRY(check_array(status, 4));
  if (n_rows > 0) {
    if (!targets != !logprob) return TWELL_ERR_INVALID_ARG;
    KV_TRY(check_vectors({targets, logprob, entropy, lse}));
    if (!workspace || workspace_bytes < fwd_bytes(n_rows, vocab)) return TWELL_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return TWELL_ERR_MISALIGNED;
  }
  if (!device_is_sm103()) return TWELL_ERR_NO_DEVICE;
  if (n_rows == 0) return TWELL_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Maps maps;
  Args a = {};
  a.n_rows = n_rows, a.d_model = d_model, a.vocab = vocab, a.targets = targets, a.inv_t = inv_temperature;
  a.status = status, a.wait_limit_ns = kWaitLimitNs;
  a.of_target = static_cast<float*>(workspace);
  a.part = a.of_target + n_rows;
  Job j = {};
  j.type = kJobSums, j.m = n_rows, j.n = vocab, j.ksplit = 1;
  KV_TRY(set_job(&maps, &a, j, H, ldh, W, ldw, d_model));
  KV_TRY(launch_jobs(maps, a, TWELL_KERNEL_LINEAR_LOGPROBS, s));
  const JoinArgs join{a.part, a.of_target, a.job[0].num_n, n_rows, vocab, targets, logprob, entropy, lse};
  LaunchScope scope(TWELL_KERNEL_LINEAR_LOGPROBS, s);
  return launch_pdl(linear_join_kernel, dim3(ceil_div(n_rows, 32)), dim3(kJoinWarps * 32), 0, s, join) == cudaSuccess
             ? TWELL_OK
             : TWELL_ERR_CUDA;
}

extern "C" TWELL_API size_t twell_linear_logprobs_bwd_workspace_bytes(int32_t n_rows, int32_t d_model,
                                                                      int32_t vocab) {
  if (n_rows < 0 || d_model < 8 || d_model % 8 != 0 || vocab < 1) return 0;
  return plan_bwd(n_rows, d_model, vocab).bytes;
}

extern "C" TWELL_API int twell_linear_logprobs_bwd(const uint16_t* H, int64_t ldh, const uint16_t* W, int64_t ldw,
                                                   int32_t n_rows, int32_t d_model, int32_t vocab,
                                                   const int32_t* targets, float inv_temperature, const float* lse,
                                                   const float* entropy, const float* d_logprob,
                                                   const float* d_entropy, uint16_t* dH, int64_t lddh, uint16_t* dW,
                                                   int64_t lddw, void* workspace, size_t workspace_bytes,
                                                   int32_t* status, twell_stream_t stream) {
  KV_TRY(check_linear(H, ldh, W, ldw, n_rows, d_model, vocab, inv_temperature));
  KV_TRY(check_array(status, 4));
  if (dW && (lddw < d_model || lddw % 8 != 0)) return TWELL_ERR_INVALID_ARG;
  if (!aligned_to(dW, 16)) return TWELL_ERR_MISALIGNED;
  const Plan plan = plan_bwd(n_rows, d_model, vocab);
  if (n_rows > 0) {
    KV_TRY(check_array(lse, 4));
    if (!targets != !d_logprob || !entropy != !d_entropy) return TWELL_ERR_INVALID_ARG;
    if (!dH && !dW) return TWELL_ERR_INVALID_ARG;
    if (dH && (lddh < d_model || lddh % 8 != 0)) return TWELL_ERR_INVALID_ARG;
    if (!aligned_to(dH, 16)) return TWELL_ERR_MISALIGNED;
    KV_TRY(check_vectors({targets, entropy, d_logprob, d_entropy}));
    if (!workspace || workspace_bytes < plan.bytes) return TWELL_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return TWELL_ERR_MISALIGNED;
  }
  if (!device_is_sm103()) return TWELL_ERR_NO_DEVICE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n_rows == 0) {  // no row: dW is zero
    if (dW && cudaMemset2DAsync(dW, lddw * 2, 0, d_model * 2, vocab, s) != cudaSuccess) return TWELL_ERR_CUDA;
    return TWELL_OK;
  }
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  uint16_t* const buffer[2] = {reinterpret_cast<uint16_t*>(ws),
                               reinterpret_cast<uint16_t*>(ws + (plan.pieces > 1 ? plan.grad_bytes : 0))};
  Args base = {};
  base.n_rows = n_rows, base.d_model = d_model, base.vocab = vocab, base.targets = targets;
  base.inv_t = inv_temperature, base.lse = lse, base.entropy = entropy, base.g = d_logprob, base.ge = d_entropy;
  base.ld_grad = plan.piece;
  base.dh_sum = reinterpret_cast<float*>(ws + plan.grad_bytes * (plan.pieces > 1 ? 2 : 1));
  base.dh = dH, base.lddh = lddh, base.dw = dW, base.lddw = lddw;
  base.status = status, base.wait_limit_ns = kWaitLimitNs;
  for (int p = 0; p <= plan.pieces; ++p) {
    Maps maps;
    Args a = base;
    if (p > 0) {  // the products of piece p - 1
      const int col0 = (p - 1) * plan.piece, width = std::min(plan.piece, vocab - col0);
      const uint16_t* const G = buffer[(p - 1) & 1];
      const uint16_t* const Wp = W + static_cast<int64_t>(col0) * ldw;
      Job j = {};
      j.col0 = col0, j.add = p > 1, j.round = p == plan.pieces && plan.ksplit == 1;
      if (dH) {
        j.type = kJobDHidden, j.m = n_rows, j.n = d_model, j.b_mn = 1;
        // the first piece fills all ranges' sums; a narrower last one adds to no more than it has steps
        j.ksplit = plan.ksplit;
        KV_TRY(set_job(&maps, &a, j, G, plan.piece, Wp, ldw, width));
      }
      if (dW) {
        j.type = kJobDWeight, j.m = width, j.n = d_model, j.a_mn = j.b_mn = 1, j.ksplit = 1;
        KV_TRY(set_job(&maps, &a, j, G, plan.piece, H, ldh, n_rows));
      }
    }
    if (p < plan.pieces) {  // G of piece p
      const int col0 = p * plan.piece;
      Job j = {};
      j.type = kJobGrad, j.m = n_rows, j.n = std::min(plan.piece, vocab - col0), j.ksplit = 1, j.col0 = col0;
      a.grad = buffer[p & 1];
      KV_TRY(set_job(&maps, &a, j, H, ldh, W + static_cast<int64_t>(col0) * ldw, ldw, d_model));
    }
    KV_TRY(launch_jobs(maps, a, TWELL_KERNEL_LINEAR_LOGPROBS_BWD, s));
  }
  if (!dH || plan.ksplit == 1) return TWELL_OK;
  const ReduceArgs r{base.dh_sum, plan.ksplit, n_rows, d_model, dH, lddh};
  LaunchScope scope(TWELL_KERNEL_LINEAR_LOGPROBS_BWD, s);
  return launch_pdl(linear_reduce_kernel, dim3(ceil_div(static_cast<int64_t>(n_rows) * (d_model / 8), 256)), dim3(256),
                    0, s, r) == cudaSuccess
             ? TWELL_OK
             : TWELL_ERR_CUDA;
}
