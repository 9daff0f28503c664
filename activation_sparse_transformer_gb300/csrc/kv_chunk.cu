// Attention over the 8-bit cache for requests with many rows (prompt chunks) on
// the 5th-generation tensor cores.
//
// One CTA takes 256 rows (token, query head) of one request and key head, as
// two tiles of 128 rows, and walks over the cached tokens 128 at a time.
// Four warpgroups work on it:
//   warps 0-3, 4-7  softmax of tile 0 and 1, one thread a row
//   warps 8-11      codes -> fp16 operands in shared memory, shared by both tiles
//   warp 12         issues the mma's
//   warp 13         copies the codes to shared memory a step ahead
// For tile X and step t:  S_X = Q_X K_t^T (tcgen05, fp32 in TMEM);  w = 2^(S f_j +
// log2 s_v - n) -> fp16 in TMEM over S;  O_X += w V_t (A from TMEM).  f_j is
// the row's factor times the key scale and s_v the value scale of the token's
// page; n follows the row's largest exponent lazily (kRoom below it; when it is passed by 8, O
// is rescaled).  The softmax's own sum needs w / s_v: it is taken per 16
// tokens, which share a page.  While one tile is in its softmax the tensor cores work on
// the other.
//
// 4 D flops for each (row, token): tensor cores bound it, then the exponentials
// and the shared memory that feeds both operands of S.
//
// 4 chunks of 556 to 966 tokens at the end of 5668 to 8192, 32 / 8 heads of 128, e4m3: 355 us,
// 930 TFLOP/s (a step 2.4 us, its mma's alone 1.1).  Taking the blocks as they come,
// uncut, 380; longest first, uncut, 381 (376 blocks are 2.5 waves); longest first with the last wave
// cut 355.  One chunk of 541 tokens at the end of 32768: 534 -> 462 us with up to 4 waves of parts.
#include <algorithm>
#include <cfloat>

#include "kv_attention.h"

namespace twell {
namespace {

constexpr int kTileRows = 128;
constexpr int kBlockRows = 2 * kTileRows;
constexpr int kTokens = 128;   // cached tokens of a step
// A step's weights are handed over in so many runs (heads of 64: 277 us; in one 285, in four 292).
constexpr int kRuns = 2;
constexpr int kGroups = kTokens / 16;
constexpr int kThreads = 16 * 32;
// Registers a thread of each warpgroup (softmax 0, softmax 1, operands, mma's):
// together the 4 x 128 that the launch gives.
constexpr int kRegsSoftmax = 184, kRegsOperands = 88, kRegsMma = 56;
static_assert(2 * kRegsSoftmax + kRegsOperands + kRegsMma == 4 * 128, "register split");
constexpr int kMaxWaves = 4, kMaxParts = kMaxWaves * 152;  // CTAs that leave parts of rows
constexpr int kJoinSteps = 8;
template <int D>
constexpr int kPartFloats = D + 4;  // of a row: the sums over the values, the reference, the sum

template <int D>
struct ChunkSmem {
  static constexpr uint32_t kBlk = kTileRows * 128;        // 128 rows of 64 fp16, 128-byte swizzled
  static constexpr uint32_t kQ = (D / 64) * kBlk;          // one tile
  static constexpr uint32_t kK = (D / 64) * kBlk, kV = kK;
  static constexpr uint32_t kKAt = 2 * kQ, kVAt = kKAt + 2 * kK;
  static constexpr uint32_t kRawAt = kVAt + 2 * kV, kRaw = kTokens * D;  // codes of a step's keys, of its values
  static constexpr uint32_t kScaleAt = kRawAt + 2 * kRaw;
  static constexpr uint32_t kBarAt = kScaleAt + 4 * 3 * kGroups * 4;
  static constexpr uint32_t kBytes = kBarAt + 512;
};

// The issuing warp stays converged and one elected lane issues: the operands
// then sit in uniform registers, without a move for each of them (an issue
// from a lane's own branch took as long as the mma itself).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
// D[tmem] (+)= A * B^T, fp16 inputs, fp32 accumulation: A from shared memory ...
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// ... or from TMEM (two fp16 a column, row = lane).
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Two fp32 lanes of one instruction.
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float f, float c) {
  asm("{\n\t.reg .b64 v, m, k;\n\tmov.b64 v, {%2, %3};\n\tmov.b64 m, {%4, %4};\n\tmov.b64 k, {%5, %5};\n\t"
      "fma.rn.f32x2 v, v, m, k;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(f), "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 v, w;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\t"
      "add.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

// ------------------------------------------------------------ order of the blocks
// The row blocks of all requests with many rows, by the cached tokens that their last
// row sees (128 a step, as positions at the cache's end give it), the longest first and
// then in request order: CTAs start in this order, so the short blocks fill up what the
// long ones leave.
// Each CTA looks up the block of its rank by bisection over the number of steps; counts have a closed form in a request.
// What is left for chunk_join_kernel: the place of a block's rows.
struct Item {
  int32_t t0, n_rows, row0, head, n_parts;
};

struct Order {
  int sums[2][16];
  int request, block;
};

__device__ __forceinline__ int blocks_of(const AttArgs& a, const Request& q) {
  return q.n_rows > a.chunk_rows ? (q.n_rows + kBlockRows - 1) / kBlockRows : 0;
}
// Blocks of q whose last row sees at least min_tokens: all but the first ones.
__device__ __forceinline__ int blocks_from(const AttArgs& a, const Request& q, int64_t min_tokens) {
  const int blocks = blocks_of(a, q);
  if (min_tokens <= 0) return blocks;
  if (q.len < min_tokens) return 0;
  const int64_t before = q.n_rows - (q.len - min_tokens + 1) * a.group;
  return before <= 0 ? blocks : blocks - static_cast<int>(min(static_cast<int64_t>(blocks), before / kBlockRows));
}
// The sum of v over the CTA, in every thread; turn alternates between calls.
__device__ __forceinline__ int cta_sum(Order& o, int turn, int v) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) o.sums[turn & 1][threadIdx.x >> 5] = v;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; w += 4) {
    const int4 x = *reinterpret_cast<const int4*>(&o.sums[turn & 1][w]);
    all += x.x + x.y + x.z + x.w;
  }
  return all;
}
// Waves of parts: each takes a CTA's start, which is little beside 32 steps.
__host__ __device__ inline int max_waves(int max_steps) {
  return max_steps < 64 ? 1 : max_steps < 32 * kMaxWaves ? max_steps / 32 : kMaxWaves;
}
// What CTA x of chunk_kernel does.
struct Work {
  int request, row0, head, part, n_parts, slot;  // slot: among the blocks that are cut
};
// By the whole CTA: false when there is nothing left for it.
__device__ __forceinline__ bool work_at(const AttArgs& a, int n_sms, int max_steps, Order& o, Item* items, Work& w) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_requests + kThreads - 1) / kThreads;
  const int r0 = min(a.n_requests, tid * per), r1 = min(a.n_requests, r0 + per);
  const Request first = r0 < r1 ? request(a, r0) : Request{0, 0, 0};
  const auto count = [&](int steps) {
    const int64_t least = static_cast<int64_t>(steps - 1) * kTokens + 1;  // tokens of that many steps
    int c = r0 < r1 ? blocks_from(a, first, least) : 0;
    for (int r = r0 + 1; r < r1; ++r) c += blocks_from(a, request(a, r), least);
    return c;
  };
  int turn = 0;
  const int items_in_all = cta_sum(o, turn++, count(0)) * a.heads;
  // One item (block, head) for each SM in turn, whole; the rest, fewer than there are SMs, are cut into as
  // many parts as fill the SMs once (or a few times, which pays for long caches), if
  // that gains more than the join takes: about 8 steps, as 3 are what a CTA takes beside its steps.
  const int whole = items_in_all / n_sms * n_sms, rest = items_in_all - whole;
  int n_parts = 1, cost = max_steps + 3 - kJoinSteps;
  for (int waves = 1; rest > 0 && waves <= max_waves(max_steps); ++waves) {
    const int p = waves * n_sms / rest;
    const int c = waves * ((max_steps + p - 1) / p + 3);
    if (p > 1 && c < cost) n_parts = p, cost = c;
  }
  if (blockIdx.x == 0)  // what is not cut is not joined
    for (int i = tid + (n_parts > 1 ? rest : 0); i < n_sms; i += kThreads) items[i] = {0, 0, 0, 0, 0};
  const int x = blockIdx.x, y = x - whole;
  if (y >= rest * n_parts) return false;
  w.slot = y >= 0 ? y / n_parts : 0;
  w.part = y >= 0 ? y % n_parts : 0;
  w.n_parts = y >= 0 ? n_parts : 1;
  const int item = y >= 0 ? whole + w.slot : x;
  const int rank = item / a.heads;
  w.head = item % a.heads;
  // the most steps that more than rank blocks take: those with max_steps or more count as one
  int lo = 0, hi = max_steps;
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (cta_sum(o, turn++, count(mid)) > rank) lo = mid;
    else hi = mid - 1;
  }
  const bool open = lo == max_steps;  // no block is ranked by more steps
  const int above = open ? 0 : count(lo + 1), mine = count(lo) - above;
  int left = rank - cta_sum(o, turn++, above);  // among the blocks of lo steps
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += x;
  }
  if (lane == 31) o.sums[turn & 1][warp] = inc;
  __syncthreads();
  for (int w = 0; w < warp; ++w) left -= o.sums[turn & 1][w];
  left -= inc - mine;
  if (left >= 0 && left < mine) {
    for (int r = r0; r < r1; ++r) {
      const Request q = request(a, r);
      const int out = open ? 0 : blocks_from(a, q, static_cast<int64_t>(lo) * kTokens + 1);
      const int in = blocks_from(a, q, static_cast<int64_t>(lo - 1) * kTokens + 1) - out;
      if (left < in) {
        o.request = r;
        o.block = blocks_of(a, q) - out - in + left;
        break;
      }
      left -= in;
    }
  }
  __syncthreads();
  w.request = __shfl_sync(0xffffffffu, o.request, 0);
  w.row0 = __shfl_sync(0xffffffffu, o.block, 0) * kBlockRows;
  return true;
}

struct Barriers {
  uint64_t raw_full[2], raw_empty[2];  // keys' codes, values' codes
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], scale_full[4], s_full[2], p_full[2][kRuns], o_done[2], drain;
  uint32_t tmem;
  int abort;
  int most, least;  // tokens that the rows of the block see
  int nan_at;       // the first token with NaN among its value's codes that not all rows see
  alignas(16) Order order;
};
static_assert(sizeof(Barriers) <= 512, "barrier region");

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const AttArgs a, int n_sms, int max_steps, float* partial, Item* items) {
  using L = ChunkSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in all lanes, for the compiler too
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* const scales = reinterpret_cast<float*>(smem + L::kScaleAt);  // [4][key, log2 value, 2^-kRoom / value][8]
  Barriers& bar = *reinterpret_cast<Barriers*>(smem + L::kBarAt);
  volatile int* const abort = &bar.abort;
  Work work;
  if (!work_at(a, n_sms, max_steps, bar.order, items, work)) return;
  const int r = work.request, row0 = work.row0, head = work.head;
  const Request q = request(a, r);
  if (work.n_parts > 1 && work.part == 0 && tid == 0)
    items[work.slot] = {q.t0, q.n_rows, row0, head, work.n_parts};
  const int n_tiles = q.n_rows - row0 > kTileRows ? 2 : 1;

  if (tid == 0) {
    mbar_init(&bar.q_full, kTileRows * n_tiles);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.raw_full[i], i == 0 ? kGroups + a.stall : kGroups);
      mbar_init(&bar.raw_empty[i], 128);
      mbar_init(&bar.k_full[i], 128);
      mbar_init(&bar.v_full[i], 128);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_empty[i], 1);
      mbar_init(&bar.s_full[i], 1);
      for (int j = 0; j < kRuns; ++j) mbar_init(&bar.p_full[i][j], kTileRows);
      mbar_init(&bar.o_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&bar.scale_full[i], kGroups);
    mbar_init(&bar.drain, 1);
    bar.abort = 0;
    bar.most = 0;
    bar.least = bar.nan_at = INT32_MAX;
    mbar_fence_init();
  }
  if (warp == 12) tmem_alloc(&bar.tmem, 512);
  __syncthreads();
  // what each row sees, and the most and the least that a row of the block does
  int limit = 0;
  const int row = row0 + tid;
  if (tid < kBlockRows) {
    if (row < q.n_rows) {
      const int p = a.positions[q.t0 + row / a.group];
      limit = max(0, min(p < INT32_MAX ? p + 1 : p, q.len));
    }
    const int most = __reduce_max_sync(0xffffffffu, limit);
    const int least = __reduce_min_sync(0xffffffffu, row < q.n_rows ? limit : INT32_MAX);
    if (lane == 0) atomicMax(&bar.most, most), atomicMin(&bar.least, least);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int all_steps = (bar.most + kTokens - 1) / kTokens;
  const int first = static_cast<int>(static_cast<int64_t>(all_steps) * work.part / work.n_parts);
  const int n_steps = static_cast<int>(static_cast<int64_t>(all_steps) * (work.part + 1) / work.n_parts) - first;
  const int j0 = first * kTokens;  // the part's first token
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem, 0);
  const uint64_t limit_ns = a.wait_ns;
  bool ok = true;

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    more_registers<kRegsSoftmax>();
    const int t_id = warp >> 2, r_in = tid & 127;
    if (t_id < n_tiles) {
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t s_tm = tmem + lanes + t_id * 128, o_tm = tmem + lanes + 256 + t_id * D;
      const int token = row / a.group, h = head * a.group + row % a.group;
      float factor;
      {
        // the row as fp16, 2^-k q with its largest magnitude in [1, 2), in the
        // swizzled layout of a K-major operand
        uint4 w[D / 8];
        const uint16_t* src = a.q + static_cast<int64_t>(q.t0 + token) * a.ldq + static_cast<int64_t>(h) * D;
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          w[i] = row < q.n_rows ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
          const uint32_t* u = &w[i].x;
#pragma unroll
          for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(u[j])), fabsf(bf16_hi(u[j]))));
        }
        const int k = min(max((__float_as_int(amax) >> 23) - 127, -126), 126);
        const float inv = __int_as_float((127 - k) << 23);
        factor = a.scale_log2 * __int_as_float((127 + k) << 23);
        uint8_t* const dst = smem + t_id * L::kQ + r_in * 128;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t* u = &w[i].x;
          uint32_t f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = pack_f16(bf16_lo(u[j]) * inv, bf16_hi(u[j]) * inv);
          *reinterpret_cast<uint4*>(dst + (i >> 3) * L::kBlk + (((i & 7) ^ (r_in & 7)) << 4)) =
              make_uint4(f[0], f[1], f[2], f[3]);
        }
        fence_async_shared();
        mbar_arrive(&bar.q_full);
      }
      float n = 0.0f, pass = -INFINITY, sum = 0.0f;  // the reference, what must be passed to move it, the sum
      for (int t = 0; t < n_steps; ++t) {
        ok = mbar_wait(&bar.s_full[t_id], t & 1, limit_ns, abort) &&
             mbar_wait(&bar.scale_full[t & 3], (t >> 2) & 1, limit_ns, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const float* const sc = scales + (t & 3) * 3 * kGroups;
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_tm + 32 * c, v[c]);
        float ks[kGroups], lvs[kGroups], ivs[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; i += 4) {
          *reinterpret_cast<float4*>(ks + i) = *reinterpret_cast<const float4*>(sc + i);
          *reinterpret_cast<float4*>(lvs + i) = *reinterpret_cast<const float4*>(sc + kGroups + i);
          *reinterpret_cast<float4*>(ivs + i) = *reinterpret_cast<const float4*>(sc + 2 * kGroups + i);
        }
        tmem_ld_wait();
        const int left = limit - j0 - t * kTokens;  // tokens of the step that the row sees
        if (left < kTokens) {  // may be negative
#pragma unroll
          for (int i = 0; i < kTokens; ++i)
            if (i >= left) v[i / 32][i % 32] = 0xFF800000u;
        }
        float top = -INFINITY;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const uint32_t* const u = &v[g / 2][16 * (g % 2)];
          float m = __uint_as_float(u[0]);
#pragma unroll
          for (int i = 1; i < 16; ++i) m = fmaxf(m, __uint_as_float(u[i]));
          ks[g] = fmaxf(ks[g] * factor, FLT_MIN);  // a masked -inf stays so
          top = fmaxf(top, fmaf(m, ks[g], lvs[g]));
        }
        const bool move = top > pass;
        if (__any_sync(0xffffffffu, move)) {
          // O holds the steps before this one: their mma's were waited for before this S was issued
          float f = 1.0f;
          if (move) {
            f = sum == 0.0f ? 0.0f : exp2_fast(n + kRoom - top);
            sum *= f;
            n = top - kRoom;
            pass = top + kLazy;
          }
          if (t > 0) {
#pragma unroll 1
            for (int c = 0; c < D / 8; ++c) {
              uint32_t o[8];
              tmem_ld8(o_tm + 8 * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st8(o_tm + 8 * c, o);
            }
          }
        }
        // w = 2^(S f + log2 s_v - n): fp16 over the columns of S
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int g = 2 * c; g < 2 * c + 2; ++g) {
            const uint32_t* const u = &v[c][16 * (g % 2)];
            const float off = lvs[g] - n;
            float part[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float e0, e1;
              fma2(e0, e1, __uint_as_float(u[i]), __uint_as_float(u[i + 1]), ks[g], off);
              e0 = exp2_fast(e0);
              e1 = exp2_fast(e1);
              add2(part[0], part[1], e0, e1);
              p[8 * (g % 2) + i / 2] = pack_f16(e0, e1);
            }
            const float both = part[0] + part[1];
            if (both != 0.0f) sum = fmaf(both, ivs[g], sum);  // a page that is not seen may have any scale
          }
          tmem_st16(s_tm + 16 * c, p);
          if ((c + 1) % (4 / kRuns) == 0) {
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bar.p_full[t_id][c / (4 / kRuns)]);
          }
        }
      }
      // the finished row
      if (ok && n_steps > 0) ok = mbar_wait(&bar.o_done[t_id], (n_steps - 1) & 1, limit_ns, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
      } else {
        tc_fence_after();
        const bool whole = work.n_parts == 1;
        // a row that sees nothing divides by no sum: zeros
        const float inv = limit > bar.nan_at ? __int_as_float(0x7FC00000) : sum == 0.0f ? 0.0f : whole ? kUnroom / sum : 1.0f;
        uint16_t* const dst = a.o + static_cast<int64_t>(q.t0 + token) * a.ldo + static_cast<int64_t>(h) * D;
        float* const to =
            partial + (static_cast<int64_t>(work.slot * work.n_parts + work.part) * kBlockRows + tid) * kPartFloats<D>;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32] = {};
          if (n_steps > 0) {
            tmem_ld32(o_tm + 32 * c, v);
            tmem_ld_wait();
          }
          if (row >= q.n_rows) continue;
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = sum != 0.0f ? __float_as_uint(__uint_as_float(v[i]) * inv) : 0u;
          if (whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = static_cast<uint32_t>(float_to_bf16_bits(__uint_as_float(v[8 * i + 2 * j]))) |
                       (static_cast<uint32_t>(float_to_bf16_bits(__uint_as_float(v[8 * i + 2 * j + 1]))) << 16);
              reinterpret_cast<uint4*>(dst + 32 * c)[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<uint4*>(to + 32 * c)[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
        if (!whole && row < q.n_rows)
          *reinterpret_cast<float4*>(to + D) = make_float4(sum != 0.0f ? n : -INFINITY, sum, 0.0f, 0.0f);
        if (whole && a.lse && row < q.n_rows)
          a.lse[static_cast<int64_t>(q.t0 + token) * a.q_heads + h] =
              sum != 0.0f ? (n + kRoom + log2f(sum)) * 0.69314718055994531f : -INFINITY;
      }
    }
  } else if (warp < 12) {
    // ---------------------------------------------------------------- codes to operands
    fewer_registers<kRegsOperands>();
    constexpr int kLanes = D / 16;                 // lanes of a token, 16 codes each
    constexpr int kPass = 128 / kLanes;            // tokens of a pass of the four warps
    constexpr int kPasses = kTokens / kPass;
    // The 8 lanes that access shared memory together hold 64 dims each of two
    // neighbouring tokens, the first 64 of one and the last 64 of the other: neither
    // the codes (128 bytes a token) nor the swizzled fp16 pieces share a bank.
    const int dw = warp - 8, half = (lane >> 2) & 1, oct = lane >> 3;
    const int blk = D == 128 ? half ^ (oct & 1) : 0, even = 2 * (lane & 3);
    const int tok = dw * (32 / kLanes) + (D == 128 ? (oct >> 1) * 2 + half : lane >> 2);
    const int least = bar.least;
    const auto load = [&](int v, int t, uint4 (&w)[kPasses]) {
      const uint8_t* const raw = smem + L::kRawAt + v * L::kRaw + blk * 64 + (lane & 3) * 16;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) w[i] = *reinterpret_cast<const uint4*>(raw + (i * kPass + tok) * D);
      if (j0 + (t + 1) * kTokens > least) {
        // Past the request's tokens a page may hold anything, and so may the value of a token that
        // not all rows see, but 0 * NaN is not 0: zeros, and NaN at the end for the rows that see such a token.
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int j = j0 + t * kTokens + i * kPass + tok;
          if (j >= q.len) w[i] = make_uint4(0, 0, 0, 0);
          if (FMT == TWELL_KV_E4M3 && v == 1 &&
              (nan_codes(w[i].x) | nan_codes(w[i].y) | nan_codes(w[i].z) | nan_codes(w[i].w))) {
            atomicMin(&bar.nan_at, j);
            w[i] = make_uint4(0, 0, 0, 0);
          }
        }
      }
    };
    const auto store = [&](uint8_t* dst, uint32_t halves, const uint4 (&w)[kPasses]) {
      // halves: bytes between the two 64-token halves of a value tile (a key tile has its tokens in one run)
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int tk = i * kPass + tok;
        uint32_t f[8];
        codes_to_f16<FMT>(w[i].x, f[0], f[1]);
        codes_to_f16<FMT>(w[i].y, f[2], f[3]);
        codes_to_f16<FMT>(w[i].z, f[4], f[5]);
        codes_to_f16<FMT>(w[i].w, f[6], f[7]);
        uint8_t* const at = halves ? dst + (tk >> 6) * halves + blk * 8192 + (tk & 63) * 128
                                   : dst + blk * L::kBlk + tk * 128;
        *reinterpret_cast<uint4*>(at + ((even ^ (tk & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<uint4*>(at + (((even + 1) ^ (tk & 7)) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
      }
      fence_async_shared();
    };
    for (int t = 0; t < n_steps; ++t) {
      const int st = t & 1;
      uint4 w[kPasses];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bar.raw_full[v], t & 1, limit_ns, abort));
        if (!ok) break;
        load(v, t, w);
        mbar_arrive(&bar.raw_empty[v]);
        ok = __all_sync(0xffffffffu, mbar_wait(v ? &bar.v_empty[st] : &bar.k_empty[st], ((t >> 1) & 1) ^ 1, limit_ns,
                                               abort));
        if (!ok) break;
        if (v == 0) {
          store(smem + L::kKAt + st * L::kK, 0, w);
          mbar_arrive(&bar.k_full[st]);
        } else {
          store(smem + L::kVAt + st * L::kV, (D / 64) * 8192, w);
          mbar_arrive(&bar.v_full[st]);
        }
      }
      if (!ok) break;
    }
    if (!ok) report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
  } else {
    // ---------------------------------------------------------------- mma's
    fewer_registers<kRegsMma>();
    if (warp == 12 && n_steps > 0) {
      const uint32_t leader = elect_one();
      constexpr uint32_t kShape = (1u << 4) | (8u << 24);  // fp32 result, fp16 operands, 128 rows
      constexpr uint32_t kIdescS = kShape | ((kTokens >> 3) << 17);
      constexpr uint32_t kIdescO = kShape | (static_cast<uint32_t>(D >> 3) << 17) | (1u << 16);  // V: dims run fastest
      bool issued = false;
      const auto scores = [&](int t, int x_id) {
        const uint64_t qd = smem_desc_sw128(smem_u32(smem + x_id * L::kQ));
        const uint64_t kd = smem_desc_sw128(smem_u32(smem + L::kKAt + (t & 1) * L::kK));
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t step = (k >> 2) * (L::kBlk >> 4) + 2 * (k & 3);
          mma_ss(leader, tmem + x_id * 128, qd + step, kd + step, kIdescS, k > 0);
        }
        commit(leader, &bar.s_full[x_id]);
      };
      const auto values = [&](int t, int x_id, int run) {
        const uint64_t vd = smem_desc_sw128_nmajor(smem_u32(smem + L::kVAt + (t & 1) * L::kV), 8192);
#pragma unroll
        for (int i = 0; i < kTokens / 16 / kRuns; ++i) {
          const int k = run * (kTokens / 16 / kRuns) + i;
          mma_ts(leader, tmem + 256 + x_id * D, tmem + x_id * 128 + 8 * k,
                 vd + (k >> 2) * ((D / 64) * 8192 >> 4) + 128 * (k & 3), kIdescO, t > 0 || k > 0);
        }
        if (run == kRuns - 1) commit(leader, &bar.o_done[x_id]);
      };
      ok = mbar_wait(&bar.q_full, 0, limit_ns, abort);
      for (int t = 0; ok && t <= n_steps; ++t) {
        if (t < n_steps) ok = mbar_wait(&bar.k_full[t & 1], (t >> 1) & 1, limit_ns, abort);
        for (int x_id = 0; ok && x_id < n_tiles; ++x_id) {
          if (t > 0) {
            // O of the step before; its weights lie over S, so the next S waits for it
            ok = x_id > 0 || mbar_wait(&bar.v_full[(t - 1) & 1], ((t - 1) >> 1) & 1, limit_ns, abort);
#pragma unroll
            for (int run = 0; run < kRuns; ++run) {
              ok = ok && mbar_wait(&bar.p_full[x_id][run], (t - 1) & 1, limit_ns, abort);
              if (!ok) break;
              tc_fence_after();
              values(t - 1, x_id, run);
              issued = true;
            }
            if (!ok) break;
            if (x_id == n_tiles - 1) commit(leader, &bar.v_empty[(t - 1) & 1]);
            if (t < n_steps) ok = mbar_wait(&bar.o_done[x_id], (t - 1) & 1, limit_ns, abort);
            if (!ok) break;
          }
          if (t < n_steps) {
            tc_fence_after();
            scores(t, x_id);
            issued = true;
            if (x_id == n_tiles - 1) commit(leader, &bar.k_empty[t & 1]);
          }
        }
      }
      if (!ok) {
        report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
        if (issued) {
          // wait for the mma's already issued before TMEM is released
          commit(leader, &bar.drain);
          volatile int never = 0;
          mbar_wait(&bar.drain, 0, kDrainNs, &never);
        }
      }
    } else if (warp == 13 && lane < kGroups) {
      // lane l: the l-th group of 16 tokens of every step, which lies in one page
      constexpr uint32_t kGroupBytes = 16 * D;
      const int page_mask = (1 << a.page_shift) - 1;
      const int32_t* const table = a.block_table + static_cast<int64_t>(r) * a.max_blocks;
      const auto page_at = [&](int t) {
        const int64_t j = static_cast<int64_t>(first + t) * kTokens + lane * 16;
        int page = -1;
        if (j < q.len) {
          page = table[j >> a.page_shift];
          if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.n_pages)) {
            report_error(a.status, TWELL_ERR_BAD_FORMAT);
            page = 0;
          }
        }
        return page;
      };
      constexpr uint32_t kMine = (1u << kGroups) - 1;
      int page = page_at(0), next = n_steps > 1 ? page_at(1) : -1, issued = 0;
      for (int t = 0; t < n_steps; ++t) {
        const int after = t + 2 < n_steps ? page_at(t + 2) : -1;
        const int64_t cell = static_cast<int64_t>(max(page, 0)) * a.heads + head;
        const int64_t at = ((cell << a.page_shift) + ((t * kTokens + lane * 16) & page_mask)) * D;
        const float ks = page >= 0 ? a.k_scale[cell] : 1.0f, vs = page >= 0 ? a.v_scale[cell] : 1.0f;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          ok = __all_sync(kMine, mbar_wait(&bar.raw_empty[v], (t & 1) ^ 1, limit_ns, abort));
          if (!ok) break;
          if (page >= 0) {
            mbar_arrive_expect_tx(&bar.raw_full[v], kGroupBytes);
            bulk_load(smem + L::kRawAt + v * L::kRaw + lane * kGroupBytes, (v ? a.v : a.k) + at, kGroupBytes,
                      &bar.raw_full[v]);
          } else {
            mbar_arrive(&bar.raw_full[v]);
          }
          issued = t + 1;
        }
        if (!ok) break;
        // The step's scales, in a slot of four: the keys' codes of step t - 1 have been
        // taken up, after the values of t - 2 were put in place, which waited for the
        // mma's of t - 4: both softmaxes are through with that step's scales.
        float* const sc = scales + (t & 3) * 3 * kGroups + lane;
        sc[0] = ks;
        sc[kGroups] = log2_scale(vs);
        sc[2 * kGroups] = kUnroom / vs;
        mbar_arrive(&bar.scale_full[t & 3]);
        page = next;
        next = after;
      }
      if (!ok) {
        report_error(a.status, TWELL_ERR_WAIT_TIMEOUT);
        // let the copies already in flight land before the CTA leaves
        for (int v = 0; v < 2 && issued > 0; ++v) {
          volatile int never = 0;
          mbar_wait(&bar.raw_full[v], (issued - 1) & 1, kDrainNs, &never);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds the parts of a block's rows, in order: D / 8 lanes a row.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const AttArgs a, const float* partial,
                                                                  const Item* items) {
  constexpr int kLanes = D / 8, kMost = 4;
  grid_dependency_wait();
  const Item p = items[blockIdx.x];
  const int n_parts = p.n_parts;
  const int in = blockIdx.y * (kJoinThreads / kLanes) + threadIdx.x / kLanes, d0 = threadIdx.x % kLanes * 8;
  if (p.row0 + in >= p.n_rows) return;
  const int64_t stride = static_cast<int64_t>(kBlockRows) * kPartFloats<D>;
  const float* const from = partial + blockIdx.x * n_parts * stride + in * kPartFloats<D>;
  float n = -INFINITY, sum = 0.0f, o[8] = {};
  for (int c0 = 0; c0 < n_parts; c0 += kMost) {
    float4 lo[kMost], hi[kMost];
    float2 st[kMost];
    float m = n;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      st[i] = make_float2(-INFINITY, 0.0f);
      lo[i] = hi[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (c0 + i < n_parts) {
        const float* const at = from + (c0 + i) * stride;
        st[i] = *reinterpret_cast<const float2*>(at + D);
        lo[i] = *reinterpret_cast<const float4*>(at + d0);
        hi[i] = *reinterpret_cast<const float4*>(at + d0 + 4);
      }
    }
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
  store_row<D>(a, p.t0, p.row0 + in, p.head, d0, n, sum, o);
}

// Row blocks that n_tokens tokens can come to.
int64_t most_blocks(const AttArgs& a) {
  const int64_t rows = static_cast<int64_t>(a.n_tokens) * a.group;
  return rows / kBlockRows + std::min<int64_t>(a.n_requests, rows / (kChunkRows + 1));
}

template <int FMT, int D>
int launch(const AttArgs& a, int max_kv_len, void* workspace, cudaStream_t s) {
  constexpr size_t smem = ChunkSmem<D>::kBytes + 1024;
  KV_TRY(set_max_dynamic_smem(reinterpret_cast<const void*>(chunk_kernel<FMT, D>), static_cast<int>(smem)));
  float* const partial = static_cast<float*>(workspace);
  Item* const items = reinterpret_cast<Item*>(partial + static_cast<size_t>(kMaxParts) * kBlockRows * kPartFloats<D>);
  const int64_t most = most_blocks(a) * a.heads, sms = std::min(sm_count(), kMaxParts / kMaxWaves);
  if (most == 0) return TWELL_OK;  // no request can have that many rows
  const int max_steps = static_cast<int>((static_cast<int64_t>(max_kv_len) + kTokens - 1) / kTokens);
  // whole items and the parts of the rest, see work_at
  const int64_t ctas = (most / sms + max_waves(max_steps)) * sms;
  {
    LaunchScope scope(TWELL_KERNEL_KV_ATTENTION, s);
    if (launch_pdl(chunk_kernel<FMT, D>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), smem, s, a,
                   static_cast<int>(sms), max_steps, partial, items) != cudaSuccess)
      return TWELL_ERR_CUDA;
  }
  if (max_steps <= kJoinSteps + 1) return TWELL_OK;  // too short for any to be cut: a part's step and 3 are no gain
  LaunchScope scope(TWELL_KERNEL_KV_JOIN, s);
  return launch_pdl(chunk_join_kernel<D>, dim3(static_cast<unsigned>(sms), kBlockRows / (kJoinThreads / (D / 8))),
                    dim3(kJoinThreads), 0, s, a, static_cast<const float*>(partial),
                    static_cast<const Item*>(items)) == cudaSuccess
             ? TWELL_OK
             : TWELL_ERR_CUDA;
}

}  // namespace

size_t chunk_workspace_bytes(int64_t rows, int dim) {
  if (rows <= kChunkRows) return 0;
  return static_cast<size_t>(kMaxParts) * (static_cast<size_t>(kBlockRows) * (dim + 4) * sizeof(float) + sizeof(Item));
}

int launch_chunk_attention(const AttArgs& a, int format, int dim, int max_kv_len, void* workspace, cudaStream_t s) {
  const auto fn = format == TWELL_KV_E4M3 ? dim == 64 ? launch<TWELL_KV_E4M3, 64> : launch<TWELL_KV_E4M3, 128>
                  : dim == 64             ? launch<TWELL_KV_INT8, 64>
                                          : launch<TWELL_KV_INT8, 128>;
  return fn(a, max_kv_len, workspace, s);
}

}  // namespace twell
