// Log probabilities of tokens from hidden rows H [N][d] and output weights
// W [V][d] (twell_linear_logprobs) and their gradient (..._bwd): the logits
// x = H W^T / T live in tensor memory only, a tile at a time.
//
// Forward: with l = H W^T and d = (l - m) log2(e) / T, each 128 x 256 tile leaves a row's maximum m of l,
// S = sum 2^d and U = sum 2^d d over the tile's columns; a second kernel joins the tiles of a row:
//   lse = m / T + ln2 log2 S,  logprob = (l_t - m) / T - ln2 log2 S,  entropy = ln2 (log2 S - U / S).
// m and l_t are kept as they were multiplied, and what is scaled is their distance: so neither the size of the
// logits nor the ends of fp32 count, and as S >= 1 no log probability comes out above 0 (with x_t - lse
// a token of all but 1e-9 of the mass came out off by 9e-7 at logits of 20 and 1e-5 at 400, a tenth of them above 0).
// Backward, in pieces of the vocabulary: x again, from it
//   G = (g (1[t] - p) - ge p (log p + entropy)) / T,  p = exp(x - lse),
// as bf16 into the workspace (the tensor cores take bf16, and each entry is then
// off by up to 2^-8 of itself, as the bf16 results are), then
// dH += G W_piece and dW_piece = G^T H with fp32 sums.  A launch runs the products
// of one piece together with G of the next one, which needs a buffer of its own.
//
// All products are tiles of one persistent kernel on the 5th-generation tensor cores:
// operands by TMA into 128-byte swizzled stages, accumulators twice in TMEM, a
// warp for each operand's copies, one for the MMAs, eight for the epilogue.  The two gradient products read
// G and H or W along their rows, so those operands go in M- or N-major.
// A pair of CTAs shares a tile of 256 x 256 (each keeps half of either operand and half of the
// rows' sums), which halves what shared memory feeds to the tensor cores; up to 128 rows there is
// nothing for a second CTA, and a CTA takes 128 x 256 alone.
//
// Few tiles are cut along K, so that all CTAs have work: dH's and dW's with fp32 sums that linear_reduce_kernel adds, the
// logits' with linear_ranges_kernel.
//
// The tensor cores cut off what does not fit when they add, one step in 16 products, so a
// logit of d = 4096 would come out 4e-6 too near to zero.  Logits are therefore added up in registers in runs of
// 512 products, rounding to nearest, while the next run is multiplied (forward 2 % slower than all at once, gradient 1 %,
// with d = 128 3 %): by the forward pass, with or without ranges of K, and for G alike, so that p = exp(x - lse) is made
// of the logits that lse was made of, bit for bit.  (With all of K at once p was too small by |x| 4e-6, which is all of
// the 1 - p of a token at x = 20 that has all but 1e-4 of the mass.)
#include <algorithm>

#include "kv_internal.h"

namespace twell {
namespace {

// A tile: kBM rows a CTA, kBN columns.  Narrower tiles do not pay even where they leave fewer CTAs idle in the last round:
// 413 x 1032 x 50001 takes 257 ns and 0.59 a column for a step of K (192 columns 54 us, 128 73, 256 52).
constexpr int kBM = 128, kBN = 256, kBK = 64, kUmmaK = 16;
constexpr int kThreads = 384, kEpiWarps = 8;
constexpr int kRun = 8;  // steps of K that logits are added up over in tensor memory
constexpr uint32_t kABytes = kBM * kBK * 2;
constexpr uint32_t kBarBytes = 256;
constexpr int kSlots = 4;                                    // forward: one half's sums, for the other half
constexpr uint32_t kSumBytes = kSlots * 128 * sizeof(float4);
constexpr uint32_t kBoxBytes = 32 * 128;                     // backward: a box of 32 rows on its way out,
constexpr uint32_t kOutBytes = kEpiWarps * 2 * kBoxBytes;    // two a warp
constexpr uint32_t kMaxShared = 232448;
// What a launch does: the forward pass's tiles, logits of ranges of K (see linear_ranges_kernel), the backward pass's jobs.
enum Mode { kSums, kRanges, kJobs };
// R CTAs to a tile; SUMS: the forward pass.  As many stages as there is room for.
template <int R, bool SUMS>
struct Cfg {
  static constexpr uint32_t kBBytes = kBN / R * kBK * 2;  // of a CTA
  static constexpr uint32_t kRest = 1024 + kBarBytes + (SUMS ? kSumBytes : kOutBytes);
  static constexpr int kStages = static_cast<int>((kMaxShared - kRest) / (kABytes + kBBytes));
  static constexpr uint32_t kShared = kRest + kStages * (kABytes + kBBytes);
};
constexpr int kBandWide = 64, kBandGradients = 8;
constexpr int kMaxJobs = 3;
constexpr int kMaxSize = 1 << 30;        // rows, columns: indexes of whole tiles fit in 32 bits
constexpr int kPlanSms = 152;            // plans do not depend on the device, workspaces neither
// Of G.  It comes back from memory, not from L2, but smaller pieces leave the last rounds of their launches emptier (single
// calls of 8192 x 2048 x 32768: 32 MB 2165 us, 64 MB 1850, 128 MB 1772, 256 MB 1756 for twice the workspace).
constexpr int64_t kPieceBytes = 1 << 27;
constexpr int kMinPiece = 4096;          // columns; dH's sums are read and written once a piece
constexpr int kMaxKSplit = 32;
constexpr int kRangeSteps = kRun, kRangesSave = 12;  // of K: see logit_ranges
constexpr int kJoinCols = 64;                // of ranges that are added by a CTA
constexpr int kTileSteps = 5;            // of K, that a tile takes at least: until its results have left
constexpr float kFarthest = 16777216.0f;  // of |lse|: a step of fp32 is 2 from there on
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

enum JobType { kJobSums, kJobGrad, kJobDHidden, kJobDWeight };

// One product C[M][N] = A . B^T in tiles, K cut into ksplit ranges.
struct Job {
  int type;
  int m, n;                 // rows and columns of C
  int num_m, num_n, num_k;  // tiles, steps of K
  int ksplit;
  int col0;                 // first vocabulary column of the piece
  int units, band;          // tiles, rows of tiles that are taken together
  int start, light0, light, extra;  // how the tiles are dealt, see Walk
  int a_mn, b_mn;           // operand stored [K][M] / [K][N]
  int add, round;           // earlier pieces have left dH's sums; these are the last
  int sum_rows;             // of one range's sums
};

struct Maps {
  CUtensorMap a[kMaxJobs], b[kMaxJobs], out[kMaxJobs];
};

struct Args {
  Job job[kMaxJobs];
  int num_jobs;
  int n_rows, d_model, vocab;
  const int32_t* targets;
  float inv_t;
  // forward
  float4* part;       // [n_rows][parts of the columns]: m, S, U
  float* of_target;   // [n_rows] the target's logit, unscaled
  float* ranges;      // [ksplit][num_m][num_n][kBN][rows of a tile]: logits of ranges of K, unscaled
  // backward
  const float *lse, *entropy, *g, *ge;
  const float* dh_sum;  // [ksplit][rows, up to whole tiles][d_model]
  int32_t* status;
  uint64_t wait_limit_ns;
  int stall;  // arrivals that every stage waits for in vain (the self-test)
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The shared memory of another CTA of the cluster.
__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A pair's hand-over: the second CTA's copies to the first one's MMAs, and accumulators back.  Arrivals, and the waits for
// them, have the cluster's scope (without one they have a CTA's, which promises nothing to the other) and order
// shared memory by fences for it alone.  With arrive.release.cluster, which orders global memory too,
// 8192 x 2048 x 32768 takes 1403 us, not 577 to 600, and its gradient 5496.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
      : "memory");
}
template <int R>
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile int* abort) {
  const bool ok = mbar_wait<R == 2>(bar, parity, limit_ns, abort);
  if (R == 2) asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
  return ok;
}

// The gradient's epilogue holds a row's logits while it makes G of them: its warps take registers that the issuing ones have
// no use for (without, they spill: gradient of 8192 x 1024 x 32768 1000 us, so 955; 8192 x 640 x 32768 842 and 738).
constexpr int kRegsIssue = 88, kRegsEpilogue = 208;
static_assert(4 * kRegsIssue + kEpiWarps * kRegsEpilogue == kThreads / 32 * 168, "the launch's registers");
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The issuing warps stay converged and one elected lane issues: the operands then sit in uniform registers,
// without a move for each of them (issued from a lane's own branch, four MMAs and their commit took
// 640 cycles of the 512 that they run: 8192 x 2048 x 32768 in 642 us without any copies).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ void expect_bytes(uint32_t leader, uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void load_box(uint32_t leader, void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(leader)
      : "memory");
}

// The tensor-core operations of a CTA alone and of a pair, whose first CTA issues for both.
template <int R>
struct Tc;
template <>
struct Tc<1> {
  static __device__ __forceinline__ void alloc(uint32_t* holder) { tmem_alloc(holder, 512); }
  static __device__ __forceinline__ void dealloc(uint32_t base) { tmem_dealloc(base, 512); }
  static __device__ __forceinline__ void mma(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(leader)
        : "memory");
  }
  static __device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(leader)
        : "memory");
  }
  static __device__ __forceinline__ void sync() { __syncthreads(); }
};
template <>
struct Tc<2> {
  static __device__ __forceinline__ void alloc(uint32_t* holder) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(holder)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  static __device__ __forceinline__ void dealloc(uint32_t base) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(512) : "memory");
  }
  static __device__ __forceinline__ void mma(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(leader)
        : "memory");
  }
  // arrives at the same barrier of both CTAs
  static __device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3)), "r"(leader)
        : "memory");
  }
  static __device__ __forceinline__ void sync() { cluster_sync(); }
};

// Two fp32 lanes of one instruction.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 lanes(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A row's running sums in base 2 relative to the unscaled logit m.
struct Sums {
  float m = -INFINITY, s = 0.0f, u = 0.0f;
  // joins sums that are relative to m2; c scales logits to base 2
  __device__ __forceinline__ void join(float m2, float s2, float u2, float c) {
    const float top = fmaxf(m, m2);
    if (top == -INFINITY) {  // neither has an entry above -inf: S is 0, or NaN where there was one
      s += s2, u += u2;
      return;
    }
    // a side without entries has S = U = 0 and m = -inf: its factor is 0, and so is its shift times S
    const float d1 = fmaxf((m - top) * c, -1e30f), d2 = fmaxf((m2 - top) * c, -1e30f);
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

// A thread's share of a tile: its row's logits (unscaled) of half of the columns, two a word.
struct Half {
  F2 v[kBN / 4];
};

// Adds a run's sums to those of the runs before, or (FIRST) takes them.
template <bool FIRST = false>
__device__ __forceinline__ void add_run(Half& x, uint32_t taddr) {
#pragma unroll
  for (int k = 0; k < kBN / 2; k += 32) {
    uint32_t r[32];
    tmem_ld32(taddr + k, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const F2 v = pair(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
      x.v[k / 2 + i] = FIRST ? v : add2(x.v[k / 2 + i], v);
    }
  }
}

// Sums of the tile's columns.  A row's right half hands its sums to the left one through shared memory, with the
// number of the tile (turn, from 1 on) as word that they are there: a wait that can expire, as a barrier of both
// could not.  The right half is at most two tiles ahead (it cannot get an accumulator that the left one has not read), so
// four places in turn are enough.
__device__ __forceinline__ bool epilogue_sums(const Args& a, const Job& j, const Tile& t, int n_blk, Half& x,
                                              float4* shared, int turn, volatile int* abort) {
  const float c = a.inv_t * kLog2e;
  const int target = t.valid && a.targets ? a.targets[t.row] : -1;
  const int col = t.col0 + t.half * (kBN / 2), left = min(j.n - col, kBN / 2);
  if (left < kBN / 2) {  // columns past the vocabulary
#pragma unroll
    for (int i = 0; i < kBN / 4; ++i) {
      const float2 f = lanes(x.v[i]);
      x.v[i] = pair(2 * i < left ? f.x : -INFINITY, 2 * i + 1 < left ? f.y : -INFINITY);
    }
  }
  if (target >= col && target < col + left) {
    F2 own = 0;
#pragma unroll
    for (int i = 0; i < kBN / 4; ++i)  // in asm: as C++ it becomes an indexed read, and x goes to local memory
      asm("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %2, %3;\n\t@p mov.b64 %0, %1;\n\t}"
          : "+l"(own)
          : "l"(x.v[i]), "r"((target - col) / 2), "r"(i));
    a.of_target[t.row] = (target - col) & 1 ? lanes(own).y : lanes(own).x;
  }
  Sums all;
#pragma unroll
  for (int i = 0; i < kBN / 4; ++i) all.m = fmaxf(all.m, fmaxf(lanes(x.v[i]).x, lanes(x.v[i]).y));
  const float ref = all.m == -INFINITY ? 0.0f : all.m;
  const F2 c2 = pair(c, c), minus = pair(-ref, -ref);
  F2 s[2] = {0, 0}, u[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kBN / 4; ++i) {
    const float2 y = lanes(mul2(add2(x.v[i], minus), c2));
    const F2 e = pair(ex2(y.x), ex2(y.y));
    s[i & 1] = add2(s[i & 1], e);
    u[i & 1] = fma2(e, pair(fmaxf(y.x, -1e30f), fmaxf(y.y, -1e30f)), u[i & 1]);  // 0 for an entry of -inf
  }
  const float2 sums = lanes(add2(s[0], s[1])), shifted = lanes(add2(u[0], u[1]));
  all.s = sums.x + sums.y, all.u = shifted.x + shifted.y;
  volatile float* const at =
      reinterpret_cast<volatile float*>(shared + (turn % kSlots) * 128 + t.lg * 32 + (threadIdx.x & 31));
  if (t.half == 1) {
    at[0] = all.m, at[1] = all.s, at[2] = all.u;
    __threadfence_block();
    at[3] = __int_as_float(turn);
    return true;
  }
  const uint64_t t0 = global_timer_ns();
  while (__float_as_int(at[3]) != turn) {
    if (*abort) return false;
    if (global_timer_ns() - t0 > a.wait_limit_ns) {
      *abort = 1;
      return false;
    }
  }
  __threadfence_block();
  if (!t.valid) return true;
  all.join(at[0], at[1], at[2], c);
  a.part[static_cast<int64_t>(t.row) * j.num_n + n_blk] = make_float4(all.m, all.s, all.u, 0.0f);
  return true;
}

// A range's logits, columns by rows: a warp's stores are whole lines.  at: of this thread's row and its first column.
__device__ __forceinline__ void store_range(float* at, int pitch, int left, const Half& x) {
#pragma unroll
  for (int i = 0; i < kBN / 4; ++i) {
    const float2 f = lanes(x.v[i]);
    if (2 * i < left) at[2 * i * pitch] = f.x;
    if (2 * i + 1 < left) at[(2 * i + 1) * pitch] = f.y;
  }
}

// Results leave through shared memory by TMA, a box of 32 rows of 128 bytes a time, so that memory gets whole
// lines and edges are cut by the copy (a row's 64 bytes from each thread are half sectors, 16 bytes at
// a time).  Two boxes a warp: one is filled while the other is read.
struct Box {
  uint8_t* base;  // this warp's two
  int turn;
  // the box to fill: its last copy has been read
  __device__ __forceinline__ uint8_t* open() {
    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
    return base + (turn ^= 1) * kBoxBytes;
  }
  // 16-byte piece c of this thread's row, swizzled as the copy reads it
  static __device__ __forceinline__ void put(uint8_t* box, int lane, int c, const uint4& w) {
    *reinterpret_cast<uint4*>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) = w;
  }
  template <bool ADD>
  static __device__ __forceinline__ void send(const uint8_t* box, const CUtensorMap* map, int x, int y) {
    fence_async_shared();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      if (ADD)
        asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                     "r"(smem_u32(box)), "r"(x), "r"(y)
                     : "memory");
      else
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                     "r"(smem_u32(box)), "r"(x), "r"(y)
                     : "memory");
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
};

// What G needs of a row.
struct GradRow {
  F2 inv_t, minus_lse, a0, a1;
  float g;
  int target;
  __device__ __forceinline__ GradRow(const Args& a, int row, bool valid) {
    float lse = 0.0f, f0 = 0.0f, f1 = 0.0f;
    g = 0.0f, target = -1;
    if (valid) {
      lse = a.lse[row];
      if (a.targets) {
        target = a.targets[row];
        if (target >= 0 && target < a.vocab) g = a.inv_t * a.g[row];
      }
      f0 = -g;
      if (a.ge) {
        f1 = -a.inv_t * a.ge[row];
        f0 = fmaf(f1, a.entropy[row], f0);
      }
      // a row of -inf only, or one so far from zero that fp32 tells lse to no better than 1, and so p to no
      // better than a factor e (all tokens at -3e38: p = 1 for each): zeros
      if (fabsf(lse) >= kFarthest) lse = INFINITY, f0 = 0.0f, f1 = 0.0f, g = 0.0f;
    }
    inv_t = pair(a.inv_t, a.inv_t), minus_lse = pair(-lse, -lse), a0 = pair(f0, f0), a1 = pair(f1, f1);
  }
  // G of two logits, without the target's part
  __device__ __forceinline__ float2 of(F2 logits) const {
    const F2 x = fma2(logits, inv_t, minus_lse);
    const float2 y = lanes(mul2(x, pair(kLog2e, kLog2e))), xs = lanes(x);
    return lanes(mul2(pair(ex2(y.x), ex2(y.y)), fma2(a1, pair(fmaxf(xs.x, -1e30f), fmaxf(xs.y, -1e30f)), a0)));
  }
};

// G of the tile as bf16: 32 columns for a box that takes 64, from the logits v(0 .. 15), two a word.
template <typename F>
__device__ __forceinline__ void put_grad(const GradRow& row, int target, uint8_t* box, int h, F v) {
  const int lane = threadIdx.x & 31;
  const bool here = __any_sync(0xffffffffu, target >= 0 && target < 32);
#pragma unroll
  for (int q = 0; q < 32; q += 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = q; i < q + 8; i += 2) {
      float2 f = row.of(v(i / 2));
      if (here) f.x += target == i ? row.g : 0.0f, f.y += target == i + 1 ? row.g : 0.0f;
      w[(i - q) / 2] = bf16_pair(f.x, f.y);
    }
    Box::put(box, lane, 4 * h + q / 8, make_uint4(w[0], w[1], w[2], w[3]));
  }
}
// from the sums of several runs
__device__ __forceinline__ void epilogue_grad(const Args& a, const Job& j, const Tile& t, const Half& x,
                                              const CUtensorMap* map, Box& out) {
  const GradRow row(a, t.row, t.valid);
#pragma unroll
  for (int k = 0; k < kBN / 2; k += 64) {
    const int col = t.col0 + t.half * (kBN / 2) + k;
    if (col >= j.n) return;
    uint8_t* const box = out.open();
#pragma unroll
    for (int h = 0; h < 2; ++h)
      put_grad(row, row.target - j.col0 - col - 32 * h, box, h, [&](int i) { return x.v[(k + 32 * h) / 2 + i]; });
    Box::send<false>(box, map, col, t.row - (threadIdx.x & 31));
  }
}
// from tensor memory, where one run is all
__device__ __forceinline__ void epilogue_grad(const Args& a, const Job& j, const Tile& t, const CUtensorMap* map,
                                              Box& out) {
  const GradRow row(a, t.row, t.valid);
  const int from = t.half * (kBN / 2);
#pragma unroll 1
  for (int k = from; k < from + kBN / 2; k += 64) {
    const int col = t.col0 + k;
    if (col >= j.n) break;
    uint8_t* const box = out.open();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t r[32];
      tmem_ld32(t.taddr + k + 32 * h, r);
      tmem_ld_wait();
      put_grad(row, row.target - j.col0 - col - 32 * h, box, h,
               [&](int i) { return pair(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])); });
    }
    Box::send<false>(box, map, col, t.row - (threadIdx.x & 31));
  }
}

// A gradient's tile: bf16, or sums in fp32 while pieces (dH) or ranges are still to be added.
__device__ __forceinline__ void epilogue_store(const Args& a, const Job& j, const Tile& t, int ks,
                                               const CUtensorMap* map, Box& out) {
  const int lane = threadIdx.x & 31, from = t.half * (kBN / 2);
  if (!j.round) {
    const int y = ks * j.sum_rows + t.row - lane;
#pragma unroll 1
    for (int k = from; k < from + kBN / 2; k += 32) {
      if (t.col0 + k >= j.n) break;
      uint32_t r[32];
      tmem_ld32(t.taddr + k, r);
      tmem_ld_wait();
      uint8_t* const box = out.open();
#pragma unroll
      for (int q = 0; q < 8; ++q)
        Box::put(box, lane, q, make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]));
      if (j.add)
        Box::send<true>(box, map, t.col0 + k, y);
      else
        Box::send<false>(box, map, t.col0 + k, y);
    }
    return;
  }
#pragma unroll 1
  for (int k = from; k < from + kBN / 2; k += 64) {
    if (t.col0 + k >= j.n) break;
    uint8_t* const box = out.open();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t r[32];
      tmem_ld32(t.taddr + k + 32 * h, r);
      tmem_ld_wait();
      if (j.add && t.valid) {  // what the earlier pieces left
        const float* const sum = a.dh_sum + static_cast<int64_t>(t.row) * a.d_model + t.col0 + k + 32 * h;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (t.col0 + k + 32 * h + 4 * q >= j.n) break;
          const float4 s = *reinterpret_cast<const float4*>(sum + 4 * q);
          r[4 * q] = __float_as_uint(__uint_as_float(r[4 * q]) + s.x);
          r[4 * q + 1] = __float_as_uint(__uint_as_float(r[4 * q + 1]) + s.y);
          r[4 * q + 2] = __float_as_uint(__uint_as_float(r[4 * q + 2]) + s.z);
          r[4 * q + 3] = __float_as_uint(__uint_as_float(r[4 * q + 3]) + s.w);
        }
      }
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = bf16_pair(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
#pragma unroll
      for (int q = 0; q < 4; ++q)
        Box::put(box, lane, 4 * h + q, make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]));
    }
    Box::send<false>(box, map, t.col0 + k, t.row - lane);
  }
}

struct Unit {
  int job, m_blk, n_blk, ks, kb0, kb1;
};

// The tiles of one CTA (or pair): jobs one after the other, in a job K's ranges, then bands of rows of tiles, in a
// band the rows fastest.  Tiles are dealt in turn, beginning where the job before has ended; before
// that a job of short tiles behind one of long ones gives `extra` rounds to those that had one long tile less
// (`light` of them from light0 on).
struct Walk {
  int who, all;  // this CTA (or pair) of how many
  int job = 0, k = 0;
  __device__ __forceinline__ bool next(const Args& a, Unit& x) {
    for (; job < a.num_jobs; ++job, k = 0) {
      const Job& j = a.job[job];
      const int q = who - j.light0;
      if (k < j.extra && (q < 0 || q >= j.light)) k = j.extra;
      int u;
      if (k < j.extra) {
        u = k * j.light + q;
      } else {
        int turn = who - j.start;
        turn += turn < 0 ? all : 0;
        u = j.extra * j.light + turn + (k - j.extra) * all;
        if (u >= j.units) continue;
      }
      ++k;
      x.job = job;
      x.ks = u / (j.num_m * j.num_n);
      u -= x.ks * j.num_m * j.num_n;
      const int band = u / (j.band * j.num_n), rows = min(j.band, j.num_m - band * j.band);
      u -= band * j.band * j.num_n;
      x.n_blk = u / rows;
      x.m_blk = band * j.band + u - x.n_blk * rows;
      x.kb0 = static_cast<int>(static_cast<int64_t>(x.ks) * j.num_k / j.ksplit);
      x.kb1 = static_cast<int>(static_cast<int64_t>(x.ks + 1) * j.num_k / j.ksplit);
      return true;
    }
    return false;
  }
};

// R CTAs a tile; kSums, kRanges: one job.
template <int R, Mode MODE>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a) {
  grid_dependency_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr bool SUMS = MODE != kJobs;
  using C = Cfg<R, SUMS>;
  constexpr int S = C::kStages;
  uint8_t* const sA = smem;
  uint8_t* const sB = smem + S * kABytes;
  uint8_t* const extra = sB + S * C::kBBytes;  // forward: sums, backward: boxes
  // of the first CTA: full, tempty (and its own of the others); of both: empty, tfull
  uint64_t* const full = reinterpret_cast<uint64_t*>(extra + (SUMS ? kSumBytes : kOutBytes));
  uint64_t* const empty = full + S;
  uint64_t* const tfull = empty + S;
  uint64_t* const tempty = tfull + 2;
  uint64_t* const drain = tempty + 2;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* const abort = reinterpret_cast<volatile int*>(tmem_holder + 1);
  static_assert((2 * S + 5) * 8 + 8 <= static_cast<int>(kBarBytes), "barrier region");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = R == 1 ? 0 : static_cast<int>(cluster_rank());
  Walk walk{static_cast<int>(blockIdx.x) / R, static_cast<int>(gridDim.x) / R};
  Unit x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      // A, B; of the first CTA also word of the second one's
      mbar_init(&full[s], (rank == 0 ? R + 1 : 2) + a.stall);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], R * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort = 0;
    mbar_fence_init();
  }
  if (MODE == kSums)  // no tile has been there yet
    for (int i = threadIdx.x; i < kSlots * 128; i += kThreads) reinterpret_cast<float4*>(extra)[i].w = __int_as_float(0);
  if (warp == 0 && lane < 2 * a.num_jobs) tma_prefetch_desc(lane & 1 ? &maps.b[lane >> 1] : &maps.a[lane >> 1]);
  __syncwarp();
  if (warp == 2) Tc<R>::alloc(tmem_holder);
  tc_fence_before();
  Tc<R>::sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const uint64_t limit = a.wait_limit_ns;

  if (warp < 4) {
    if (MODE == kJobs) fewer_registers<kRegsIssue>();
    if (warp == 0 || warp == 2) {
      // ---------------- copies: one warp brings A, the other B (one for both takes longer to issue them than they
      // are multiplied)
      const uint32_t leader = elect_one();
      const bool is_b = warp == 2;
      uint8_t* const base = is_b ? sB : sA;
      const uint32_t pitch = is_b ? C::kBBytes : kABytes;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && walk.next(a, x)) {
        const Job& j = a.job[x.job];
        const CUtensorMap* const map = is_b ? &maps.b[x.job] : &maps.a[x.job];
        const int at = is_b ? x.n_blk * kBN + rank * (kBN / R) : (x.m_blk * R + rank) * kBM;
        const bool mn = is_b ? j.b_mn : j.a_mn;  // [K][at]: boxes of 64 columns by 64 rows of K; else one of 64 columns of K
        const int rows = is_b ? kBN / R : kBM, boxes = mn ? rows / 64 : 1;
        const uint32_t bytes = rows * kBK * 2;
        const int dx = mn ? 0 : kBK, dy = mn ? kBK : 0;
        int cx = mn ? at : x.kb0 * kBK, cy = mn ? x.kb0 * kBK : at;
        for (int n = x.kb1 - x.kb0; n > 0; --n, cx += dx, cy += dy) {
          if (!wait_pair<R>(&empty[stage], phase ^ 1u, limit, abort)) {
            ok = false;
            break;
          }
          uint8_t* const dst = base + stage * pitch;
          expect_bytes(leader, &full[stage], bytes);
          load_box(leader, dst, map, &full[stage], cx, cy);
          for (int q = 1; q < boxes; ++q) load_box(leader, dst + q * 8192, map, &full[stage], cx + q * 64, cy);
          if (++stage == S) stage = 0, phase ^= 1u;
        }
      }
      if (!ok) {
        report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
        // the copies in flight land before the CTA leaves
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 10000000ull) __nanosleep(1000);
      }
    } else if (warp == 1 && rank == 0) {
      // ---------------- products
      const uint32_t leader = elect_one();
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      const uint32_t a_stage = kABytes >> 4, b_stage = C::kBBytes >> 4;
      while (ok && walk.next(a, x)) {
        const Job& j = a.job[x.job];
        const uint32_t idesc = idesc_bf16_f32(kBM * R, kBN) | (j.a_mn ? 1u << 15 : 0u) | (j.b_mn ? 1u << 16 : 0u);
        // a step of 16 along K: 32 bytes of a K-major row, 16 rows of 128 bytes of the others
        const uint64_t a_step = j.a_mn ? 128u : 2u, b_step = j.b_mn ? 128u : 2u;
        const uint64_t ad0 = j.a_mn ? smem_desc_sw128_nmajor(smem_u32(sA), 8192) : smem_desc_sw128(smem_u32(sA));
        const uint64_t bd0 = j.b_mn ? smem_desc_sw128_nmajor(smem_u32(sB), 8192) : smem_desc_sw128(smem_u32(sB));
        for (int k0 = x.kb0; ok && k0 < x.kb1;) {
          const int k1 = SUMS || j.type == kJobGrad ? min(k0 + kRun, x.kb1) : x.kb1;
          if (!wait_pair<R>(&tempty[acc], acc_phase ^ 1u, limit, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kBN);
          uint32_t add = 0;
          for (int n = k1 - k0; n > 0; --n) {
            if (!wait_pair<R>(&full[stage], phase, limit, abort)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t ad = ad0 + stage * a_stage, bd = bd0 + stage * b_stage;
#pragma unroll
            for (int k = 0; k < kBK / kUmmaK; ++k) {
              Tc<R>::mma(leader, d, ad + k * a_step, bd + k * b_step, idesc, add);
              add = 1;
            }
            Tc<R>::commit(leader, &empty[stage]);
            if (++stage == S) stage = 0, phase ^= 1u;
          }
          if (!ok) break;
          Tc<R>::commit(leader, &tfull[acc]);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
          k0 = k1;
        }
      }
      if (!ok) {
        report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
        Tc<R>::commit(leader, drain);  // the MMAs already issued end before TMEM is released
        volatile int never = 0;
        mbar_wait(drain, 0, 10000000ull, &never);
      }
    }
    if (R == 2 && warp == 3 && lane == 0 && rank == 1) {
      // ---------------- word to the first CTA that the second one's copies have landed (counted there by the
      // copies themselves, their many completions cross over one by one: 8192 x 2048 x 32768 in 712 us, not 630)
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && walk.next(a, x)) {
        for (int kb = x.kb0; kb < x.kb1; ++kb) {
          ok = mbar_wait(&full[stage], phase, limit, abort);
          if (!ok) break;
          arrive_at(map_rank(&full[stage], 0));
          if (++stage == S) stage = 0, phase ^= 1u;
        }
      }
      if (!ok) report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
    }
    __syncwarp();
  } else {
    // ---------------- epilogue: thread = row of the tile (a TMEM lane), two warps share a row's columns
    if (MODE == kJobs) more_registers<kRegsEpilogue>();
    Tile t;
    t.lg = warp & 3;
    t.half = (warp - 4) >> 2;
    int acc = 0, turn = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(t.lg * 32) << 16);
    Box out{extra + (warp - 4) * 2 * kBoxBytes, 0};
    while (ok && walk.next(a, x)) {
      const Job& j = a.job[x.job];
      t.row = (x.m_blk * R + rank) * kBM + t.lg * 32 + lane;
      t.col0 = x.n_blk * kBN;
      t.valid = t.row < j.m;
      auto wait_full = [&]() {
        ok = wait_pair<R>(&tfull[acc], acc_phase, limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
        tc_fence_after();
        t.taddr = lane_base + static_cast<uint32_t>(acc * kBN);
        return ok;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (R == 1)
            mbar_arrive(&tempty[acc]);
          else
            arrive_at(map_rank(&tempty[acc], 0));
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      };
      const bool here = t.row - lane < j.m;  // else the warp's rows are all past the end
      if constexpr (SUMS) {
        Half sums = {};
#pragma unroll 1
        for (int k = MODE == kSums ? 0 : x.kb0; k < (MODE == kSums ? j.num_k : x.kb1); k += kRun) {
          if (!wait_full()) break;
          add_run(sums, t.taddr + t.half * (kBN / 2));
          release();
        }
        if (!ok) break;
        if constexpr (MODE == kRanges) {
          constexpr int kRows = kBM * R;
          const int64_t tile = (static_cast<int64_t>(x.ks) * j.num_m + x.m_blk) * j.num_n + x.n_blk;
          const int col = t.half * (kBN / 2);
          if (here)
            store_range(a.ranges + (tile * kBN + col) * kRows + t.row - x.m_blk * kRows, kRows, j.n - t.col0 - col, sums);
          continue;
        }
        ok = __all_sync(0xffffffffu, epilogue_sums(a, j, t, x.n_blk, sums, reinterpret_cast<float4*>(extra), ++turn, abort));
        if (!ok) report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
      } else if (j.type == kJobGrad && j.num_k > kRun) {
        Half sums;
        if (!wait_full()) break;
        add_run<true>(sums, t.taddr + t.half * (kBN / 2));
        release();
#pragma unroll 1
        for (int k = kRun; k < j.num_k; k += kRun) {
          if (!wait_full()) break;
          add_run(sums, t.taddr + t.half * (kBN / 2));
          release();
        }
        if (!ok) break;
        if (here) epilogue_grad(a, j, t, sums, &maps.out[x.job], out);
      } else {
        if (!wait_full()) break;
        if (here) {
          if (j.type == kJobGrad)
            epilogue_grad(a, j, t, &maps.out[x.job], out);
          else
            epilogue_store(a, j, t, x.ks, &maps.out[x.job], out);
        }
        release();
      }
    }
    if (!SUMS) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // what leaves this CTA has left
  }
  tc_fence_before();
  Tc<R>::sync();
  if (warp == 2) {
    tc_fence_after();
    Tc<R>::dealloc(tmem_base);
  }
}

// Where the tiles are few, each is multiplied in ranges of K by several CTAs, and this adds a tile's ranges in order, four on
// the way at a time (one after the other with 32 columns a thread: 10 x 3640 x 500 in 17 us, not 13), 32 rows (a lane
// each) and kJoinCols columns a CTA: their sums for the join as the forward epilogue leaves a tile's, or (GRAD) G.
template <bool GRAD>
__global__ void __launch_bounds__(256) linear_ranges_kernel(const __grid_constant__ Args a, uint16_t* G, int64_t ldg) {
  grid_dependency_wait();
  constexpr int C = kJoinCols / 8;  // columns a thread
  __shared__ float s[3][8][32];
  const Job& j = a.job[0];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int parts = (j.n + kJoinCols - 1) / kJoinCols;
  const int block = blockIdx.x % parts, row0 = blockIdx.x / parts * 32, row = row0 + lane;
  const int tile_rows = j.sum_rows, m_blk = row0 / tile_rows;
  const int col = block * kJoinCols + warp * C, left = min(j.n - col, C);
  const float* const at = a.ranges + (static_cast<int64_t>(m_blk) * j.num_n * kBN + col) * tile_rows + row - m_blk * tile_rows;
  const int64_t plane = static_cast<int64_t>(j.num_m) * j.num_n * kBN * tile_rows;
  float x[C] = {};
#pragma unroll 1
  for (int k = 0; k < j.ksplit; k += 4) {
    float r[4][C];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < C; ++i) r[e][i] = k + e < j.ksplit && i < left ? at[(k + e) * plane + i * tile_rows] : 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < C; ++i) x[i] += r[e][i];
  }
  const bool valid = row < j.m;
  if constexpr (GRAD) {
    if (!valid || left <= 0) return;
    const GradRow of(a, row, valid);
    const int own = of.target - col;
    uint32_t w[C / 2];
#pragma unroll
    for (int i = 0; i < C; i += 2) {
      float2 f = of.of(pair(x[i], x[i + 1]));
      f.x += own == i ? of.g : 0.0f, f.y += own == i + 1 ? of.g : 0.0f;
      w[i / 2] = bf16_pair(f.x, f.y);
    }
    static_assert(C == 8, "16 bytes");
    *reinterpret_cast<uint4*>(G + row * ldg + col) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    const int target = valid && a.targets ? a.targets[row] - col : -1;
    if (target >= 0 && target < left) {
      float own = 0.0f;
      for (int k = 0; k < j.ksplit; ++k) own += at[k * plane + target * tile_rows];
      a.of_target[row] = own;
    }
    const float c = a.inv_t * kLog2e;
    Sums all;
#pragma unroll
    for (int i = 0; i < C; ++i) all.m = i < left ? fmaxf(all.m, x[i]) : all.m;
    const float ref = all.m == -INFINITY ? 0.0f : all.m;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const float y = i < left ? (x[i] - ref) * c : -INFINITY, e = ex2(y);
      all.s += e, all.u = fmaf(e, fmaxf(y, -1e30f), all.u);
    }
    s[0][warp][lane] = all.m, s[1][warp][lane] = all.s, s[2][warp][lane] = all.u;
    __syncthreads();
    if (warp > 0 || !valid) return;
    for (int k = 1; k < 8; ++k) all.join(s[0][k][lane], s[1][k][lane], s[2][k][lane], c);
    a.part[static_cast<int64_t>(row) * parts + block] = make_float4(all.m, all.s, all.u, 0.0f);
  }
}

struct JoinArgs {
  const float4* part;
  const float* of_target;
  int num_n, n_rows, vocab;
  const int32_t* targets;
  float inv_t;
  float *logprob, *entropy, *lse;
};

// The tiles' sums of a row: a warp a row, each lane tiles in turn, then lanes by halves.
__global__ void __launch_bounds__(32) linear_join_kernel(const JoinArgs a) {
  grid_dependency_wait();
  const int lane = threadIdx.x;
  const float c = a.inv_t * kLog2e;
  for (int row = blockIdx.x; row < a.n_rows; row += gridDim.x) {
    const float4* const at = a.part + static_cast<int64_t>(row) * a.num_n;
    Sums all;
#pragma unroll 4
    for (int k = lane; k < a.num_n; k += 32) {
      const float4 p = at[k];
      all.join(p.x, p.y, p.z, c);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      // both lanes of a pair join the lower one's sums first, so that all come to the same bits
      const float m = __shfl_xor_sync(0xffffffffu, all.m, o), s = __shfl_xor_sync(0xffffffffu, all.s, o),
                  u = __shfl_xor_sync(0xffffffffu, all.u, o);
      Sums low = all, high;
      high.m = m, high.s = s, high.u = u;
      if (lane & o) low = high, high = all;
      low.join(high.m, high.s, high.u, c);
      all = low;
    }
    if (lane > 0) continue;
    // where the largest logit is finite and its scaled value is not, the row is as one of that value
    const float top = a.inv_t * all.m;
    if (top == INFINITY) all.s = __int_as_float(0x7FC00000);
    if (top == -INFINITY && all.s >= 1.0f) all.s = 0.0f;
    const float log_s = log2f(all.s);
    if (a.lse) a.lse[row] = fmaf(a.inv_t, all.m, kLn2 * log_s);
    if (a.entropy) a.entropy[row] = all.s == 0.0f ? 0.0f : kLn2 * (log_s - all.u / all.s);
    if (a.logprob) {
      const int t = a.targets[row];
      // a row of -inf only: -inf, as all its log probabilities
      a.logprob[row] = t < 0 || t >= a.vocab ? 0.0f
                       : all.s == 0.0f       ? -INFINITY
                                             : fmaf(a.inv_t, a.of_target[row] - all.m, -kLn2 * log_s);
    }
  }
}

// A gradient whose K was cut.
struct Ranges {
  const float* sum;
  int ksplit, rows, sum_rows;
  uint16_t* out;
  int64_t ld;
  int blocks;
};
struct ReduceArgs {
  Ranges of[2];  // dH, dW; no blocks: nothing to do
  int dim;
};

// dH and dW from the sums of K's ranges, added in order, 8 of them on the way at a time; 4 elements a thread.
__global__ void __launch_bounds__(256) linear_reduce_kernel(const __grid_constant__ ReduceArgs a) {
  grid_dependency_wait();
  int block = blockIdx.x;
  const Ranges& r = a.of[block < a.of[0].blocks ? 0 : 1];
  if (block >= a.of[0].blocks) block -= a.of[0].blocks;
  const int64_t vecs = a.dim / 4, i = static_cast<int64_t>(block) * 256 + threadIdx.x;
  if (i >= vecs * r.rows) return;
  const int64_t row = i / vecs, c = i % vecs * 4, plane = static_cast<int64_t>(r.sum_rows) * a.dim;
  const float* const at = r.sum + row * a.dim + c;
  float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int k = 0; k < r.ksplit; k += 8) {
    float4 x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = k + e < r.ksplit ? *reinterpret_cast<const float4*>(at + (k + e) * plane) : make_float4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) f.x += x[e].x, f.y += x[e].y, f.z += x[e].z, f.w += x[e].w;
  }
  *reinterpret_cast<uint2*>(r.out + row * r.ld + c) = make_uint2(bf16_pair(f.x, f.y), bf16_pair(f.z, f.w));
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }
size_t round_up(size_t x, size_t to) { return (x + to - 1) / to * to; }

// CTAs to a tile: a pair from 129 rows on.
int ctas_of(int64_t n_rows) { return n_rows > kBM ? 2 : 1; }

// Rows of fp32 sums: whole tiles, as a tile leaves whole.
int64_t sum_rows(int64_t rows, int ctas) { return (rows + kBM * ctas - 1) / (kBM * ctas) * (kBM * ctas); }

// What ranges of a product's K may take at most, whatever rows there are up to these: there are never more tiles than CTAs.
size_t split_bytes(int64_t ranges, int64_t rows, int64_t cols) {
  constexpr int64_t kMost = static_cast<int64_t>(kPlanSms) * kBM * kBN;
  const int64_t area = (rows + 255) / 256 * 256 * cols;
  return ranges < 2 ? 0 : round_up(static_cast<size_t>(area > kMost / ranges ? kMost : ranges * area) * 4, 256);
}

// Ranges of K that logits are multiplied in, where the tiles leave CTAs (or pairs) without one: a CTA's copies bound a step
// (0.4 us), whatever the others do.  Adding the ranges costs a launch and their way through memory, about what 12 steps and
// one for each MB take.  10 x 3640 x 500 in 31 us alone, 13 in ranges; 16 x 4096 x 8192 30 and 22, 4096 x 8192 x 256 46 and 32;
// below the limit 1000 x 1024 x 1000 13 and 17, 2000 x 4096 x 1000 (at it) 28 and 29.
int logit_ranges(int64_t n_rows, int64_t d, int64_t vocab) {
  const int ctas = ctas_of(n_rows);
  const int64_t tiles = ceil_div(n_rows, kBM * ctas) * static_cast<int64_t>(ceil_div(vocab, kBN)), num_k = ceil_div(d, kBK);
  const int64_t n = std::min<int64_t>(kPlanSms / ctas / std::max<int64_t>(tiles, 1), num_k / kRangeSteps);
  const int64_t written = n * ((n_rows + 31) / 32 * 32) * vocab * 4;
  return n >= 2 && num_k - ceil_div(num_k, n) >= kRangesSave + (written >> 20) ? static_cast<int>(n) : 1;
}
size_t ranges_bytes(int64_t n_rows, int64_t d, int64_t vocab) {
  const int n = logit_ranges(n_rows, d, vocab);
  return n == 1 ? 0 : static_cast<size_t>(n) * sum_rows(n_rows, ctas_of(n_rows)) * ceil_div(vocab, kBN) * kBN * 4;
}

// How a backward call is cut.
struct Plan {
  int pieces, piece;  // columns of a piece, a multiple of 256
  int ksplit;         // ranges of the vocabulary in dH's product of a piece
  int wsplit;         // ranges of the rows in dW's product
  int ranges;         // of K in G's
  size_t grad_bytes, sum_bytes, wsum_bytes, bytes;
};

Plan plan_bwd(int64_t n_rows, int64_t d, int64_t vocab) {
  Plan p;
  const int64_t most = std::max<int64_t>(kMinPiece, kPieceBytes / (2 * std::max<int64_t>(n_rows, 1)));
  p.pieces = ceil_div(vocab, most);
  p.piece = ceil_div(ceil_div(vocab, p.pieces), 256) * 256;
  p.pieces = ceil_div(vocab, p.piece);
  // dH's tiles have long sums: where there are fewer than CTAs (or pairs), K is cut so that all have one.
  // A CTA asks for 57 to 83 GB/s alone, so all of them are needed even where the other product could fill
  // them (16 x 4096 x 131072: 612 us with three ranges, dH's 48 CTAs the last to end).
  const int ctas = ctas_of(n_rows);
  const int64_t tiles = ceil_div(n_rows, kBM * ctas) * static_cast<int64_t>(ceil_div(d, kBN));
  const int64_t num_k = ceil_div(std::min<int64_t>(p.piece, vocab), kBK);
  p.ksplit = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>({kMaxKSplit, num_k / 8, kPlanSms / ctas / std::max<int64_t>(1, tiles)})));
  p.grad_bytes = round_up(static_cast<size_t>(n_rows) * p.piece * 2, 256);
  p.sum_bytes = p.pieces > 1 || p.ksplit > 1 ? round_up(static_cast<size_t>(p.ksplit) * sum_rows(n_rows, ctas) * d * 4, 256) : 0;
  // So is dW's, over many rows (9080 x 376 x 232: 63 -> 27 us, 11351 x 520 x 1245 90 -> 60); with several pieces it
  // has tiles enough.
  const int64_t wtiles = ceil_div(vocab, kBM * ctas) * static_cast<int64_t>(ceil_div(d, kBN));
  p.wsplit = p.pieces > 1 ? 1
                          : static_cast<int>(std::max<int64_t>(
                                1, std::min<int64_t>({kMaxKSplit, ceil_div(n_rows, kBK) / 8, kPlanSms / ctas / wtiles})));
  p.wsum_bytes = p.wsplit > 1 ? round_up(static_cast<size_t>(p.wsplit) * sum_rows(vocab, ctas) * d * 4, 256) : 0;
  // G's logits in ranges, as the forward pass has them (which cuts no more tiles than a piece has), lie where the products'
  // sums come afterwards
  p.ranges = p.pieces > 1 ? 1 : logit_ranges(n_rows, d, vocab);
  const size_t ranged = p.ranges > 1 ? ranges_bytes(n_rows, d, vocab) : 0;
  p.bytes = p.grad_bytes * (p.pieces > 1 ? 2 : 1) + std::max(p.sum_bytes + p.wsum_bytes, ranged) + 256;
  return p;
}

// Workspaces that are asked for hold what any fewer rows take, too: fewer rows have fewer tiles, which are cut into more ranges.
size_t most_ranges_bytes(int64_t n_rows, int64_t d, int64_t vocab) {
  return 2 * ceil_div(vocab, kBN) > kPlanSms
             ? 0
             : split_bytes(ceil_div(d, kBK) / kRangeSteps, n_rows, static_cast<int64_t>(ceil_div(vocab, kBN)) * kBN);
}
size_t most_bwd_bytes(int64_t n_rows, int64_t d, int64_t vocab) {
  const Plan p = plan_bwd(n_rows, d, vocab);
  // G: a piece is at most 255 columns wider than its limit
  const size_t n = n_rows, rounded = 256 * n * 2;
  const size_t grad = p.pieces == 1 ? p.grad_bytes
                                    : 2 * round_up(std::max<size_t>(kPieceBytes, n * kMinPiece * 2) + rounded, 256);
  const int64_t wtiles = ceil_div(vocab, 2 * kBM) * static_cast<int64_t>(ceil_div(d, kBN));
  const size_t sum = std::max(p.pieces == 1 ? 0 : round_up(static_cast<size_t>(sum_rows(n_rows, 2)) * d * 4, 256),
                              split_bytes(std::min(kMaxKSplit, ceil_div(vocab, kBK) / 8), n_rows, d));
  const size_t wsum = 4 * wtiles > kPlanSms ? 0 : split_bytes(std::min(kMaxKSplit, ceil_div(n_rows, kBK) / 8), vocab, d);
  return grad + std::max(sum + wsum, most_ranges_bytes(n_rows, d, vocab)) + 256;
}

// Parts of the columns that the forward pass leaves sums of.
int parts_of(int64_t n_rows, int64_t d, int64_t vocab) {
  return ceil_div(vocab, logit_ranges(n_rows, d, vocab) > 1 ? kJoinCols : kBN);
}
size_t part_bytes(int64_t n_rows, int parts) {
  return round_up(static_cast<size_t>(n_rows) * 4 * (4 * static_cast<size_t>(parts) + 1), 256) + 512;
}
size_t fwd_bytes(int64_t n_rows, int64_t d, int64_t vocab) {
  return part_bytes(n_rows, parts_of(n_rows, d, vocab)) + ranges_bytes(n_rows, d, vocab);
}
size_t most_fwd_bytes(int64_t n_rows, int64_t d, int64_t vocab) {
  const size_t ranged = most_ranges_bytes(n_rows, d, vocab);
  return part_bytes(n_rows, ceil_div(vocab, ranged > 0 ? kJoinCols : kBN)) + ranged;
}

// CTAs (or pairs) that work at a time.
int slots_of(int ctas) { return std::max(1, sm_count() / ctas); }

// Adds a job.  A: [m][k], or [k][m] with a_mn; likewise B; their rows lie lda, ldb elements apart.
int set_job(Maps* maps, Args* args, int ctas, Job j, const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb,
            int k) {
  const int i = args->num_jobs++;
  j.num_m = ceil_div(j.m, kBM * ctas), j.num_n = ceil_div(j.n, kBN), j.num_k = ceil_div(k, kBK);
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
  return encode_tmap_2d(&maps->b[i], B, k, j.n, ldb * 2, kBK, kBN / ctas);
}

// Deals the jobs' tiles to the CTAs or pairs (see Walk); returns how many of those there are.
int deal(Args* args, int slots) {
  int64_t units = 0;
  for (int i = 0; i < args->num_jobs; ++i) units += args->job[i].units;
  const int all = static_cast<int>(std::min<int64_t>(units, slots));
  int start = 0;
  int64_t cost_before = 0;
  for (int i = 0; i < args->num_jobs; ++i) {
    Job& j = args->job[i];
    const int64_t cost = std::max(kTileSteps, j.num_k / j.ksplit);
    j.start = start, j.light0 = start, j.light = all - start;
    j.extra = start > 0 ? static_cast<int>(std::min<int64_t>(cost_before / cost, j.units / j.light)) : 0;
    if (j.extra < 2) j.extra = 0;  // a round more for some is what beginning there gives, too
    start = static_cast<int>((start + j.units - static_cast<int64_t>(j.extra) * j.light) % all);
    cost_before = cost;
  }
  return all;
}

template <int R, Mode MODE>
int launch_jobs(const Maps& maps, Args args, int id, cudaStream_t s) {
  constexpr bool SUMS = MODE != kJobs;
  const auto kernel = linear_kernel<R, MODE>;
  KV_TRY(set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(Cfg<R, SUMS>::kShared)));
  const int all = deal(&args, slots_of(R));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(all) * R);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<R, SUMS>::kShared;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = R;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  LaunchScope scope(id, s);
  return cudaLaunchKernelEx(&cfg, kernel, maps, args) == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

template <Mode MODE>
int launch_jobs(int ctas, const Maps& maps, const Args& args, int id, cudaStream_t s) {
  return ctas == 2 ? launch_jobs<2, MODE>(maps, args, id, s) : launch_jobs<1, MODE>(maps, args, id, s);
}

// Logits in ranges of K, and from them the tiles' sums or G.
template <bool GRAD>
int launch_ranges(int ctas, const Maps& maps, const Args& args, uint16_t* G, int64_t ldg, int id, cudaStream_t s) {
  KV_TRY(launch_jobs<kRanges>(ctas, maps, args, id, s));
  LaunchScope scope(id, s);
  return launch_pdl(linear_ranges_kernel<GRAD>, dim3(ceil_div(args.job[0].n, kJoinCols) * ceil_div(args.n_rows, 32)), dim3(256), 0, s, args,
                    G, ldg) == cudaSuccess
             ? TWELL_OK
             : TWELL_ERR_CUDA;
}

int check_linear(const uint16_t* H, int64_t ldh, const uint16_t* W, int64_t ldw, int n_rows, int d, int vocab,
                 float inv_t) {
  if (n_rows < 0 || d < 1 || vocab < 1) return TWELL_ERR_INVALID_ARG;
  if (!(inv_t > 0.0f) || inv_t > 2.0e38f) return TWELL_ERR_INVALID_ARG;  // times log2(e) it is finite
  if (d % 8 != 0 || std::max({n_rows, d, vocab}) > kMaxSize) return TWELL_ERR_UNSUPPORTED;
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
  if (n_rows < 0 || d_model < 8 || d_model % 8 != 0 || vocab < 1 || std::max({n_rows, d_model, vocab}) > kMaxSize) return 0;
  return most_fwd_bytes(n_rows, d_model, vocab);
}

namespace {

int linear_logprobs(const uint16_t* H, int64_t ldh, const uint16_t* W, int64_t ldw, int n_rows, int d_model, int vocab,
                    const int32_t* targets, float inv_temperature, float* logprob, float* entropy, float* lse,
                    void* workspace, size_t workspace_bytes, int32_t* status, uint64_t limit_ns, int stall,
                    cudaStream_t s) {
  KV_TRY(check_linear(H, ldh, W, ldw, n_rows, d_model, vocab, inv_temperature));
  KV_TRY(check_array(status, 4));
  if (n_rows > 0) {
    if (!targets != !logprob) return TWELL_ERR_INVALID_ARG;
    KV_TRY(check_vectors({targets, logprob, entropy, lse}));
    if (!workspace || workspace_bytes < fwd_bytes(n_rows, d_model, vocab)) return TWELL_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return TWELL_ERR_MISALIGNED;
  }
  if (!device_is_sm103()) return TWELL_ERR_NO_DEVICE;
  if (n_rows == 0) return TWELL_OK;
  Maps maps;
  Args a = {};
  a.n_rows = n_rows, a.d_model = d_model, a.vocab = vocab, a.targets = targets, a.inv_t = inv_temperature;
  a.status = status, a.wait_limit_ns = limit_ns, a.stall = stall;
  a.of_target = static_cast<float*>(workspace);
  a.part = reinterpret_cast<float4*>(static_cast<uint8_t*>(workspace) + round_up(static_cast<size_t>(n_rows) * 4, 256));
  Job j = {};
  j.type = kJobSums, j.band = kBandWide, j.m = n_rows, j.n = vocab;
  const int ctas = ctas_of(n_rows), parts = parts_of(n_rows, d_model, vocab);
  j.ksplit = logit_ranges(n_rows, d_model, vocab), j.sum_rows = kBM * ctas;
  a.ranges = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + part_bytes(n_rows, parts));
  KV_TRY(set_job(&maps, &a, ctas, j, H, ldh, W, ldw, d_model));
  if (j.ksplit > 1)
    KV_TRY(launch_ranges<false>(ctas, maps, a, nullptr, 0, TWELL_KERNEL_LINEAR_LOGPROBS, s));
  else
    KV_TRY(launch_jobs<kSums>(ctas, maps, a, TWELL_KERNEL_LINEAR_LOGPROBS, s));
  const JoinArgs join{a.part, a.of_target, parts, n_rows, vocab, targets, inv_temperature, logprob, entropy, lse};
  LaunchScope scope(TWELL_KERNEL_LINEAR_LOGPROBS, s);
  return launch_pdl(linear_join_kernel, dim3(std::min(n_rows, 24 * sm_count())), dim3(32), 0, s, join) == cudaSuccess
             ? TWELL_OK
             : TWELL_ERR_CUDA;
}

}  // namespace

extern "C" TWELL_API int twell_linear_logprobs(const uint16_t* H, int64_t ldh, const uint16_t* W, int64_t ldw,
                                               int32_t n_rows, int32_t d_model, int32_t vocab, const int32_t* targets,
                                               float inv_temperature, float* logprob, float* entropy, float* lse,
                                               void* workspace, size_t workspace_bytes, int32_t* status,
                                               twell_stream_t stream) {
  return linear_logprobs(H, ldh, W, ldw, n_rows, d_model, vocab, targets, inv_temperature, logprob, entropy, lse,
                         workspace, workspace_bytes, status, kWaitLimitNs, 0, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" TWELL_API int twell_selftest_linear_stall(const uint16_t* H, int64_t ldh, const uint16_t* W, int64_t ldw,
                                                     int32_t n_rows, int32_t d_model, int32_t vocab, void* workspace,
                                                     size_t workspace_bytes, int32_t* status, uint64_t limit_ns,
                                                     twell_stream_t stream) {
  if (limit_ns < 100000ull || limit_ns > 1000000000ull) return TWELL_ERR_INVALID_ARG;
  return linear_logprobs(H, ldh, W, ldw, n_rows, d_model, vocab, nullptr, 1.0f, nullptr, nullptr, nullptr, workspace,
                         workspace_bytes, status, limit_ns, 1, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" TWELL_API size_t twell_linear_logprobs_bwd_workspace_bytes(int32_t n_rows, int32_t d_model,
                                                                      int32_t vocab) {
  if (n_rows < 0 || d_model < 8 || d_model % 8 != 0 || vocab < 1 || std::max({n_rows, d_model, vocab}) > kMaxSize) return 0;
  return most_bwd_bytes(n_rows, d_model, vocab);
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
    if ((dH && dH == H) || (dW && dW == W) || (dH && (dH == W || dH == dW)) || (dW && dW == H)) return TWELL_ERR_INVALID_ARG;
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
  float* const dh_sum = reinterpret_cast<float*>(ws + plan.grad_bytes * (plan.pieces > 1 ? 2 : 1));
  float* const dw_sum = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(dh_sum) + plan.sum_bytes);
  base.dh_sum = dh_sum;
  base.status = status, base.wait_limit_ns = kWaitLimitNs;
  const int ctas = ctas_of(n_rows);
  for (int p = 0; p <= plan.pieces; ++p) {
    Maps maps;
    Args a = base;
    if (p > 0) {  // the products of piece p - 1
      const int col0 = (p - 1) * plan.piece, width = std::min(plan.piece, vocab - col0);
      const uint16_t* const G = buffer[(p - 1) & 1];
      const uint16_t* const Wp = W + static_cast<int64_t>(col0) * ldw;
      Job j = {};
      j.col0 = col0, j.band = kBandGradients, j.b_mn = 1;
      if (dH) {
        j.type = kJobDHidden, j.m = n_rows, j.n = d_model, j.add = p > 1;
        j.round = p == plan.pieces && plan.ksplit == 1;
        // the first piece fills all ranges' sums; a narrower last one adds to no more than it has steps
        j.ksplit = plan.ksplit, j.sum_rows = static_cast<int>(sum_rows(n_rows, ctas));
        if (j.round)
          KV_TRY(encode_tmap_2d(&maps.out[a.num_jobs], dH, d_model, n_rows, lddh * 2, 64, 32));
        else
          KV_TRY(encode_tmap_2d_f32(&maps.out[a.num_jobs], dh_sum, d_model,
                                    static_cast<uint64_t>(plan.ksplit) * j.sum_rows,
                                    static_cast<uint64_t>(d_model) * 4, 32, 32));
        KV_TRY(set_job(&maps, &a, ctas, j, G, plan.piece, Wp, ldw, width));
      }
      if (dW) {
        j.type = kJobDWeight, j.m = width, j.n = d_model, j.a_mn = 1, j.add = 0;
        j.round = plan.wsplit == 1, j.ksplit = plan.wsplit, j.sum_rows = static_cast<int>(sum_rows(vocab, ctas));
        if (j.round)
          KV_TRY(encode_tmap_2d(&maps.out[a.num_jobs], dW + static_cast<int64_t>(col0) * lddw, d_model, width, lddw * 2,
                                64, 32));
        else
          KV_TRY(encode_tmap_2d_f32(&maps.out[a.num_jobs], dw_sum, d_model,
                                    static_cast<uint64_t>(plan.wsplit) * j.sum_rows,
                                    static_cast<uint64_t>(d_model) * 4, 32, 32));
        KV_TRY(set_job(&maps, &a, ctas, j, G, plan.piece, H, ldh, n_rows));
      }
    }
    if (p < plan.pieces) {  // G of piece p
      const int col0 = p * plan.piece;
      Job j = {};
      j.type = kJobGrad, j.band = kBandWide, j.m = n_rows, j.n = std::min(plan.piece, vocab - col0);
      j.col0 = col0, j.ksplit = plan.ranges, j.sum_rows = kBM * ctas;
      a.ranges = dh_sum;
      KV_TRY(encode_tmap_2d(&maps.out[a.num_jobs], buffer[p & 1], plan.piece, n_rows,
                            static_cast<uint64_t>(plan.piece) * 2, 64, 32));
      KV_TRY(set_job(&maps, &a, ctas, j, H, ldh, W + static_cast<int64_t>(col0) * ldw, ldw, d_model));
    }
    if (p == 0 && plan.ranges > 1)
      KV_TRY(launch_ranges<true>(ctas, maps, a, buffer[0], plan.piece, TWELL_KERNEL_LINEAR_LOGPROBS_BWD, s));
    else
      KV_TRY(launch_jobs<kJobs>(ctas, maps, a, TWELL_KERNEL_LINEAR_LOGPROBS_BWD, s));
  }
  auto blocks = [&](int rows) { return ceil_div(static_cast<int64_t>(rows) * (d_model / 4), 256); };
  ReduceArgs r = {};
  r.dim = d_model;
  if (dH && plan.ksplit > 1)
    r.of[0] = {dh_sum, plan.ksplit, n_rows, static_cast<int>(sum_rows(n_rows, ctas)), dH, lddh, blocks(n_rows)};
  if (dW && plan.wsplit > 1)
    r.of[1] = {dw_sum, plan.wsplit, vocab, static_cast<int>(sum_rows(vocab, ctas)), dW, lddw, blocks(vocab)};
  const int all = r.of[0].blocks + r.of[1].blocks;
  if (all == 0) return TWELL_OK;
  LaunchScope scope(TWELL_KERNEL_LINEAR_LOGPROBS_BWD, s);
  return launch_pdl(linear_reduce_kernel, dim3(all), dim3(256), 0, s, r) == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}
