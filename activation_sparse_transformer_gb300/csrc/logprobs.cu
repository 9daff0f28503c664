// Log probabilities of given tokens with entropy and best alternatives
// (twell_logprobs) and their gradient (twell_logprobs_bwd).
//
// In base 2, with y = logits log2(e) / T, m = max y, S = sum 2^(y - m),
// U = sum 2^(y - m) (y - m):
//   lse = ln2 (m + log2 S),  logprob = ln2 ((y_t - m) - log2 S),
//   entropy = ln2 (log2 S - U / S).
// A row is read from memory once.  Many rows without alternatives are summed as they are read
// (logprobs_rows_kernel).  Else a CTA (or a cluster of 2 to 8 for long rows
// and few of them) copies its slice to shared memory with asynchronous 16-byte
// copies, finds the maximum there and then sums with it, so no running maximum has
// to be corrected; slices are joined through distributed shared memory.  HBM
// bounds many rows, with the instructions of an element next (5 of them, two
// elements an instruction where there is one); few rows are bound by the latency of one slice.
// 8192 x 32768 bf16: 83 us, its gradient 164 (6.5 TB/s both); with 5 alternatives 154; 16 x 131072 fp32 with 20: 9.2 us.
//
// The k largest: the k-th largest of 64 groups' own maxima is a lower bound of
// the k-th largest value, and hardly more than k values reach it.  Those are
// collected and ranked by counting.  Keys are (value, index) pairs in one
// 64-bit word, so equal values go by index and no two keys are equal.
#include <cooperative_groups.h>

#include <cfloat>
#include <climits>
#include <type_traits>
#include <utility>

#include "kv_internal.h"

namespace cg = cooperative_groups;

namespace twell {
namespace {

constexpr int kBwdThreads = 256;
constexpr int kGroups = 64;    // of the k largest's bound: with k = 20 about 24 values reach it
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr int kCandidates = 1024;
constexpr int kRankLanes = 8;  // threads that rank a key together
constexpr int kMaxVocab = 400000;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float store(float x) { return x; }
  struct Range {
    float hi = -INFINITY, lo = INFINITY;
    __device__ __forceinline__ void add(const uint4& w) {
      float f[4];
      unpack(w, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) hi = fmaxf(hi, f[i]), lo = fminf(lo, f[i]);
    }
    __device__ __forceinline__ float high() const { return hi; }
    __device__ __forceinline__ float low() const { return lo; }
  };
};
template <>
struct Elem<uint16_t> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float load(const uint16_t* p) { return bf16_bits_to_float(*p); }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[8]) {
    f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
    f[4] = bf16_lo(w.z), f[5] = bf16_hi(w.z), f[6] = bf16_lo(w.w), f[7] = bf16_hi(w.w);
  }
  static __device__ __forceinline__ uint32_t pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
  }
  static __device__ __forceinline__ uint16_t store(float x) { return float_to_bf16_bits(x); }
  struct Range {  // of the two elements of a word at once
    uint32_t hi = 0xFF80FF80u, lo = 0x7F807F80u;
    __device__ __forceinline__ void add(const uint4& w) {
      const uint32_t* u = &w.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        asm("max.bf16x2 %0, %0, %1;" : "+r"(hi) : "r"(u[i]));
        asm("min.bf16x2 %0, %0, %1;" : "+r"(lo) : "r"(u[i]));
      }
    }
    __device__ __forceinline__ float high() const { return fmaxf(bf16_lo(hi), bf16_hi(hi)); }
    __device__ __forceinline__ float low() const { return fminf(bf16_lo(lo), bf16_hi(lo)); }
  };
};

struct LogprobsArgs {
  const void* logits;
  int64_t ld;
  int vocab, slice;  // slice: elements a CTA of the cluster takes
  const int32_t* targets;
  float inv_temperature;
  float *logprob, *entropy, *lse;
  int top_k;
  float* top_logprob;
  int32_t* top_index;
};

struct Stat {
  float m, s, u;
};

// A row whose scaled maximum is so far from zero that y's rounding counts, or that y is no number
// where x = logits / T is one (a row masked by its type's lowest value): summed again, from
// memory, by the definition's own x (far_stat), and answered in natural units.
constexpr float kFar = 1.0e6f;
__device__ __forceinline__ bool is_far(float m) { return !(fabsf(m) < kFar); }

// Stats relative to a common maximum; an empty part has s = u = 0.
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b) {
  const float m = fmaxf(a.m, b.m);
  const float da = fmaxf(a.m - m, -2000.0f), db = fmaxf(b.m - m, -2000.0f);  // finite: 0 * da is 0
  const float ea = ex2(da), eb = ex2(db);
  return {m, a.s * ea + b.s * eb, ea * (a.u + a.s * da) + eb * (b.u + b.s * db)};
}

// (value, index) as one word, larger = better: higher value, then lower index.
__device__ __forceinline__ uint64_t key_of(float x, int index) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 equals +0
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (static_cast<uint64_t>(o) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(index));
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int key_index(uint64_t k) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k));
}

template <int NT>
struct LpShared {
  uint64_t key[kMaxCluster * kMaxTop];  // the groups' maxima, then the cluster's lists
  uint64_t candidates[kCandidates];
  uint64_t best[kMaxTop];
  uint64_t bound;
  Stat stat, whole;  // of the slice, of the row
  float warp_hi[NT / 32], warp_lo[NT / 32];
  float2 warp_sum[NT / 32];
  uint64_t warp_key[NT / 32];
  int count;
};

// The part of a row that a CTA holds: whole 16-byte chunks [c0, c1) of
// `chunks`, and the elements before and behind them.
template <typename T>
struct Slice {
  const uint4* chunks;
  int lead, n, c0, c1;  // element i of the slice is element lead + i of the chunks
  __device__ __forceinline__ const T* elems() const { return reinterpret_cast<const T*>(chunks); }
  // position of the e-th element outside the whole chunks; there are edges() < 2 * kVec of them
  __device__ __forceinline__ int head() const { return c1 > c0 ? c0 * Elem<T>::kVec - lead : n; }
  __device__ __forceinline__ int edges() const { return c1 > c0 ? head() + (lead + n - c1 * Elem<T>::kVec) : n; }
  __device__ __forceinline__ int edge(int e) const { return e < head() ? e : c1 * Elem<T>::kVec - lead + (e - head()); }
};

// Number of keys in list[0, n) above `mine`, counted by kShare neighbouring
// threads together (kShare <= 32); all of them get it.
template <int kShare>
__device__ __forceinline__ int rank_in(const uint64_t* list, int n, uint64_t mine) {
  int better = 0;
#pragma unroll 4
  for (int i = threadIdx.x % kShare; i < n; i += kShare) better += list[i] > mine;
#pragma unroll
  for (int d = 1; d < kShare; d *= 2) better += __shfl_xor_sync(0xffffffffu, better, d);
  return better;
}

// The top_k best keys of the slice to sh.best, in order, 0 behind the last.
// best, at: this thread's largest logit and its place (-1: it has none).
template <typename T, int NT>
__device__ void slice_top(LpShared<NT>& sh, const Slice<T>& sl, float inv_t, int k, float best, int at) {
  using E = Elem<T>;
  constexpr int kShare = NT / kGroups;
  const int tid = threadIdx.x;
  uint64_t mine = at >= 0 ? key_of(best * inv_t, at) : 0;
#pragma unroll
  for (int d = 1; d < kShare; d *= 2) {
    const uint64_t o = __shfl_xor_sync(0xffffffffu, mine, d);
    mine = o > mine ? o : mine;
  }
  if (tid % kShare == 0) sh.key[tid / kShare] = mine;
  if (tid < kMaxTop) sh.best[tid] = 0;
  if (tid == 0) {
    sh.count = 0;
    sh.bound = 1;  // every key is larger: fewer than k groups have one
  }
  __syncthreads();
  const int better = rank_in<kShare>(sh.key, kGroups, mine);
  if (better == k - 1 && mine) sh.bound = mine;
  __syncthreads();
  const uint64_t bound = sh.bound;
  // f for every element of a chunk whose largest one is at least `from`
  const auto each = [&](float from, auto&& f) {
    for (int j = sl.c0 + tid; j < sl.c1; j += NT) {
      typename E::Range r;
      r.add(sl.chunks[j]);
      if (r.high() * inv_t < from) continue;
      float x[E::kVec];
      E::unpack(sl.chunks[j], x);
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) f(x[i] * inv_t, j * E::kVec + i - sl.lead);
    }
    if (tid < sl.edges()) {
      const int i = sl.edge(tid);
      f(E::load(sl.elems() + sl.lead + i) * inv_t, i);
    }
  };
  const float least = bound > 1 ? key_value(bound) : -INFINITY;
  each(least, [&](float v, int i) {
    if (v >= least) {
      const uint64_t key = key_of(v, i);
      if (key >= bound) {
        const int c = atomicAdd(&sh.count, 1);
        if (c < kCandidates) sh.candidates[c] = key;
      }
    }
  });
  __syncthreads();
  if (sh.count <= kCandidates) {
    const int n = sh.count;
    for (int c0 = 0; c0 < n; c0 += NT / kRankLanes) {
      const int c = c0 + tid / kRankLanes;
      const uint64_t key = c < n ? sh.candidates[c] : 0;
      const int rank = rank_in<kRankLanes>(sh.candidates, n, key);
      if (c < n && rank < k) sh.best[rank] = key;
    }
  } else {
    // rare: a few groups own most of the largest values; take them one by one
    uint64_t last = ~0ull;
    for (int i = 0; i < k; ++i) {
      uint64_t top = 0;
      each(-INFINITY, [&](float v, int index) {
        const uint64_t key = key_of(v, index);
        if (key < last && key > top) top = key;
      });
#pragma unroll
      for (int d = 16; d > 0; d /= 2) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, top, d);
        top = o > top ? o : top;
      }
      if ((tid & 31) == 0) sh.warp_key[tid / 32] = top;
      __syncthreads();
      for (int w = 0; w < NT / 32; ++w) top = sh.warp_key[w] > top ? sh.warp_key[w] : top;
      if (tid == 0) sh.best[i] = top;
      last = top;
      __syncthreads();
    }
  }
  __syncthreads();
}

// f over the elements of a row by NT threads, t the thread's number among them.
template <typename T, int NT, typename F>
__device__ __forceinline__ void each_of_row(const T* src, int vocab, int t, F f) {
  for (int i = t; i < vocab; i += NT) f(Elem<T>::load(src + i), i);
}
// v of all NT threads (a warp, or a CTA with a place for each of its warps), joined by f.
template <int NT, typename V, typename F>
__device__ __forceinline__ V team_join(V v, V* place, F f) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v = f(v, __shfl_xor_sync(0xffffffffu, v, d));
  if (NT == 32) return v;
  __syncthreads();
  if (threadIdx.x % 32 == 0) place[threadIdx.x / 32] = v;
  __syncthreads();
  v = place[0];
  for (int w = 1; w < NT / 32; ++w) v = f(v, place[w]);
  return v;
}
// The statistics of a far row in all its threads: m the largest x (not times log2 e), s and u as
// always, sums of 2^d and 2^d d with d = (x - m) log2 e.  Two more reads of the row: rare.
template <typename T, int NT>
__device__ __forceinline__ Stat far_stat(const T* src, int vocab, float inv_t, int t, float* place) {
  const auto sum = [](float a, float b) { return a + b; };
  float m = -INFINITY, s = 0.0f, u = 0.0f;
  each_of_row<T, NT>(src, vocab, t, [&](float x, int) { m = fmaxf(m, __fmul_rn(x, inv_t)); });
  m = fmaxf(team_join<NT>(m, place, [](float a, float b) { return fmaxf(a, b); }), -FLT_MAX);
  each_of_row<T, NT>(src, vocab, t, [&](float x, int) {
    const float d = (__fmul_rn(x, inv_t) - m) * kLog2e, e = ex2(d);
    s += e;
    u = fmaf(e, fmaxf(d, -2000.0f), u);
  });
  s = team_join<NT>(s, place, sum);
  return {m, s, team_join<NT>(u, place, sum)};
}

// May a row whose smallest logit is lo and whose maximum is m be summed two elements at a
// time?  Masked tokens (2^-inf * -inf is no number, be they -inf or so low that the product is) and logits
// so large that the rounding of m counts are summed one by one, with products rounded as m's was.
__device__ __forceinline__ bool short_sums(float lo, float m, float c) {
  return __fmul_rn(lo, c) > -FLT_MAX && !is_far(m) && c < 1.0e6f;
}

// (a, b) += ... of two elements in one instruction each.
__device__ __forceinline__ void sum2(float2& s, float2& u, float x0, float x1, float c, float m, float& e0, float& e1) {
  float d0, d1;
  asm("{\n\t.reg .b64 x, c, m;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 c, {%4, %4};\n\tmov.b64 m, {%5, %5};\n\t"
      "fma.rn.f32x2 x, x, c, m;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(x0), "f"(x1), "f"(c), "f"(-m));
  e0 = ex2(d0);
  e1 = ex2(d1);
  asm("{\n\t.reg .b64 s, u, e, d;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 u, {%2, %3};\n\tmov.b64 e, {%4, %5};\n\t"
      "mov.b64 d, {%6, %7};\n\tadd.rn.f32x2 s, s, e;\n\tfma.rn.f32x2 u, e, d, u;\n\t"
      "mov.b64 {%0, %1}, s;\n\tmov.b64 {%2, %3}, u;\n\t}"
      : "+f"(s.x), "+f"(s.y), "+f"(u.x), "+f"(u.y)
      : "f"(e0), "f"(e1), "f"(d0), "f"(d1));
}

// A row's results from its statistics (FAR: those of far_stat); a NaN or +inf among the
// scaled logits makes all of them NaN.
template <bool FAR>
__device__ __forceinline__ float lse_of(const Stat& st, float log_s) {
  return isnan(st.s) ? __int_as_float(0x7FC00000) : st.s == 0.0f ? -INFINITY
         : FAR       ? fmaf(log_s, kLn2, st.m) : (st.m + log_s) * kLn2;
}
template <bool FAR>
__device__ __forceinline__ float logprob_of(const LogprobsArgs& a, const Stat& st, float logit) {
  const float log_s = log2f(st.s);
  float y;
  if (FAR) {
    y = __fmul_rn(logit, a.inv_temperature) - st.m - log_s * kLn2;
  } else {
    const float d = fmaf(logit, a.inv_temperature * kLog2e, -st.m);
    y = (d - log_s) * kLn2;
    // a masked token's d may be no number's
    if (d < -kFar) y = __fmul_rn(logit, a.inv_temperature) - lse_of<FAR>(st, log_s);
  }
  return isnan(st.s) ? __int_as_float(0x7FC00000) : st.s == 0.0f ? -INFINITY : y;
}
template <bool FAR>
__device__ __forceinline__ void store_row(const LogprobsArgs& a, int64_t row, const Stat& st, int target, float logit) {
  const float log_s = log2f(st.s);
  if (a.lse) a.lse[row] = lse_of<FAR>(st, log_s);
  if (a.entropy)
    a.entropy[row] = isnan(st.s) ? __int_as_float(0x7FC00000) : st.s == 0.0f ? 0.0f : (log_s - st.u / st.s) * kLn2;
  if (a.targets) a.logprob[row] = target >= 0 && target < a.vocab ? logprob_of<FAR>(a, st, logit) : 0.0f;
}

template <bool FAR, typename T>
__device__ __forceinline__ void store_target(const LogprobsArgs& a, int64_t row, const Stat& st, const T* src) {
  const int t = a.targets ? a.targets[row] : -1;
  store_row<FAR>(a, row, st, t, t >= 0 && t < a.vocab ? Elem<T>::load(src + t) : 0.0f);
}
// The i-th best of a row.
template <bool FAR, typename T>
__device__ __forceinline__ void store_top(const LogprobsArgs& a, int64_t row, int i, const Stat& st, uint64_t key,
                                          const T* src) {
  const bool broken = isnan(st.s);
  a.top_logprob[row * a.top_k + i] = logprob_of<FAR>(a, st, Elem<T>::load(src + (broken ? 0 : key_index(key))));
  a.top_index[row * a.top_k + i] = broken ? -1 : key_index(key);
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT) logprobs_kernel(const LogprobsArgs a) {
  using E = Elem<T>;
  // copies to another place within 128 bytes cost up to a sixth (8192 x 32768 with 5 alternatives 172 us, so 153)
  extern __shared__ __align__(128) uint4 chunks[];
  __shared__ LpShared<NT> sh;
  grid_dependency_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int64_t row = blockIdx.x / ranks;
  const T* const src = static_cast<const T*>(a.logits) + row * a.ld;
  const int beg = min(rank * a.slice, a.vocab), n = min(a.slice, a.vocab - beg);
  // the slice with the 16-byte pieces it touches; the last, cut piece comes in by elements
  const T* const from = src + beg;
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(from) & 15) / sizeof(T));
  const int whole = n > 0 ? (lead + n) / E::kVec : 0;
  const uint4* const g = reinterpret_cast<const uint4*>(from - lead);
  for (int j = tid; j < whole; j += NT)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(chunks + j)), "l"(g + j) : "memory");
  for (int i = max(whole * E::kVec, lead) + tid; i < lead + n; i += NT) reinterpret_cast<T*>(chunks)[i] = from[i - lead];
  const Slice<T> sl = {chunks, lead, n, lead > 0 ? 1 : 0, whole};
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  // the largest logit (with its place, for the alternatives) and the smallest
  float hi = -INFINITY, lo = INFINITY;
  int at = -1;
  if (a.top_k > 0) {
    for (int j = sl.c0 + tid; j < sl.c1; j += NT) {
      typename E::Range r;
      r.add(chunks[j]);
      lo = fminf(lo, r.low());
      if (r.high() > hi || at < 0) hi = r.high(), at = j;
    }
    if (at >= 0) {
      // the first element of that chunk that is its largest (none where all are NaN)
      float x[E::kVec];
      E::unpack(chunks[at], x);
      int i = 0;
#pragma unroll
      for (int k = E::kVec - 1; k >= 0; --k)
        if (x[k] == hi) i = k;
      at = at * E::kVec + i - lead;
    }
  } else {
    typename E::Range r;
    for (int j = sl.c0 + tid; j < sl.c1; j += NT) r.add(chunks[j]);
    hi = r.high();
    lo = r.low();
  }
  if (tid < sl.edges()) {
    const int i = sl.edge(tid);
    const float x = E::load(sl.elems() + lead + i);
    if (x > hi || at < 0) at = i;
    hi = fmaxf(hi, x);
    lo = fminf(lo, x);
  }
  float m = hi;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
  }
  if ((tid & 31) == 0) sh.warp_hi[tid / 32] = m, sh.warp_lo[tid / 32] = lo;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) m = fmaxf(m, sh.warp_hi[w]), lo = fminf(lo, sh.warp_lo[w]);
  const float c = a.inv_temperature * kLog2e;
  m = fmaxf(__fmul_rn(m, c), -FLT_MAX);

  float2 s = {0.0f, 0.0f}, u = {0.0f, 0.0f};
  const bool plain = short_sums(lo, m, c);
  const auto add = [&](float x) {
    const float d = plain ? fmaf(x, c, -m) : __fmul_rn(x, c) - m, e = ex2(d);
    s.x += e;
    u.x = fmaf(e, fmaxf(d, -2000.0f), u.x);
  };
  if (plain) {
    for (int j = sl.c0 + tid; j < sl.c1; j += NT) {
      float x[E::kVec], e0, e1;
      E::unpack(chunks[j], x);
#pragma unroll
      for (int i = 0; i < E::kVec; i += 2) sum2(s, u, x[i], x[i + 1], c, m, e0, e1);
    }
  } else {
    for (int j = sl.c0 + tid; j < sl.c1; j += NT) {
      float x[E::kVec];
      E::unpack(chunks[j], x);
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) add(x[i]);
    }
  }
  if (tid < sl.edges()) add(E::load(sl.elems() + lead + sl.edge(tid)));
  s.x += s.y;
  u.x += u.y;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    s.x += __shfl_xor_sync(0xffffffffu, s.x, d);
    u.x += __shfl_xor_sync(0xffffffffu, u.x, d);
  }
  if ((tid & 31) == 0) sh.warp_sum[tid / 32] = make_float2(s.x, u.x);
  __syncthreads();
  if (tid == 0) {
    Stat all = {m, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) all.s += sh.warp_sum[w].x, all.u += sh.warp_sum[w].y;
    sh.stat = all;
  }
  if (a.top_k > 0) slice_top<T, NT>(sh, sl, a.inv_temperature, a.top_k, hi, at);
  if (ranks == 1) {
    __syncthreads();
    const Stat st = sh.stat;
    const auto store = [&](const Stat& st, auto far) {
      if (tid == 0) store_target<far.value>(a, row, st, src);
      if (tid < a.top_k) store_top<far.value>(a, row, tid, st, sh.best[tid], src);
    };
    if (is_far(st.m)) store(far_stat<T, NT>(src, a.vocab, a.inv_temperature, tid, sh.warp_hi), std::true_type{});
    else store(st, std::false_type{});
    return;
  }
  cluster.sync();
  // every rank takes all statistics and lists, and places the keys of its own list
  const int n_keys = ranks * a.top_k;
  if (tid < 32 && (rank == 0 || n_keys > 0)) {
    Stat st = {-FLT_MAX, 0.0f, 0.0f};
    if (tid < ranks) st = *cluster.map_shared_rank(&sh.stat, tid);
#pragma unroll
    for (int d = 1; d < kMaxCluster; d *= 2)
      st = join(st, {__shfl_xor_sync(0xffffffffu, st.m, d), __shfl_xor_sync(0xffffffffu, st.s, d),
                     __shfl_xor_sync(0xffffffffu, st.u, d)});
    if (tid == 0) sh.whole = st;
  }
  for (int e = tid - 32; e < n_keys; e += NT - 32) {
    if (e < 0) break;  // the first warp is at the statistics
    const int of = e / a.top_k;
    const uint64_t key = cluster.map_shared_rank(&sh, of)->best[e % a.top_k];
    sh.key[e] = key ? key - static_cast<uint64_t>(of) * a.slice : 0;  // indexes of the row
  }
  auto last = cluster.barrier_arrive();  // no rank leaves before the others have read its shared memory
  __syncthreads();
  if (rank > 0 && n_keys == 0) {  // has placed what it has, without the row's statistics
    cluster.barrier_wait(std::move(last));
    return;
  }
  const auto store = [&](const Stat& st, auto far) {
    if (rank == 0 && tid == 0) store_target<far.value>(a, row, st, src);
    for (int i0 = 0; i0 < a.top_k; i0 += NT / kRankLanes) {
      const int i = i0 + tid / kRankLanes;
      const uint64_t key = i < a.top_k ? sh.key[rank * a.top_k + i] : 0;
      const int better = rank_in<kRankLanes>(sh.key, n_keys, key);
      if (tid % kRankLanes != 0 || i >= a.top_k) continue;
      if (isnan(st.s) ? rank == 0 : key && better < a.top_k)
        store_top<far.value>(a, row, isnan(st.s) ? i : better, st, key, src);
    }
  };
  if (is_far(sh.whole.m)) store(far_stat<T, NT>(src, a.vocab, a.inv_temperature, tid, sh.warp_hi), std::true_type{});
  else store(sh.whole, std::false_type{});
  cluster.barrier_wait(std::move(last));
}

// The same without alternatives, for many rows: nothing is read twice, so nothing needs
// to be kept.  NT threads take a row, each with a maximum of its own that follows what it
// reads, kBatch 16-byte loads at a time; their sums are brought to the row's maximum at the end.
// The next rows' loads run under a row's sums, where a staged row's CTA waits for all of its
// copies first: 8192 x 32768 bf16 83.0 us (6.5 TB/s), staged 101; fp32 149 (7.2 TB/s), staged 212.
constexpr int kRowsThreads = 256, kBatch = 4;
// From 2 rows an SM on (320 x 131072 fp32: 33 us, staged in clusters 40).
constexpr int kManyRows = 2;
// (Six CTAs an SM where one takes a row: far_stat's registers alone would leave five, 85.9 us.)
template <typename T, int NT>
__global__ void __launch_bounds__(kRowsThreads, NT == 32 ? 5 : 6) logprobs_rows_kernel(const LogprobsArgs a, int n_rows) {
  using E = Elem<T>;
  __shared__ Stat sh[kRowsThreads / 32];
  grid_dependency_wait();
  const int t = threadIdx.x % NT;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kRowsThreads / NT) + threadIdx.x / NT;
  if (row >= n_rows) return;  // whole warps, and whole CTAs where a row has several
  const T* const src = static_cast<const T*>(a.logits) + row * a.ld;
  int target = -1;
  float x_target = 0.0f;
  if (t == 0 && a.targets) {
    target = a.targets[row];
    if (target >= 0 && target < a.vocab) x_target = E::load(src + target);
  }
  const float c = a.inv_temperature * kLog2e;
  float m = -FLT_MAX;
  float2 s = {0.0f, 0.0f}, u = {0.0f, 0.0f};
  // moves the reference up to y, and tells if what goes with it may be summed the short way
  const auto meet = [&](float hi, float lo) {
    const float y = __fmul_rn(hi, c);
    if (y > m) {
      const float d = fmaxf(m - y, -2000.0f), f = ex2(d);
      u.x = f * fmaf(s.x, d, u.x), u.y = f * fmaf(s.y, d, u.y);
      s.x *= f, s.y *= f;
      m = y;
    }
    return short_sums(lo, m, c);
  };
  const auto add = [&](float x) {  // with the product rounded as m's was, and for masked tokens
    const float d = __fmul_rn(x, c) - m, e = ex2(d);
    s.x += e;
    u.x = fmaf(e, fmaxf(d, -2000.0f), u.x);
  };
  const auto batch = [&](const uint4* w, auto n) {
    typename E::Range r;
#pragma unroll
    for (int i = 0; i < n.value; ++i) r.add(w[i]);
    const bool plain = meet(r.high(), r.low());
#pragma unroll
    for (int i = 0; i < n.value; ++i) {
      float x[E::kVec], e0, e1;
      E::unpack(w[i], x);
      if (plain) {
#pragma unroll
        for (int k = 0; k < E::kVec; k += 2) sum2(s, u, x[k], x[k + 1], c, m, e0, e1);
      } else {
#pragma unroll
        for (int k = 0; k < E::kVec; ++k) add(x[k]);
      }
    }
  };
  // elements up to a 16-byte boundary, whole pieces, the elements behind them
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
  const int head = min(a.vocab, (16 - off) % 16 / static_cast<int>(sizeof(T)));
  const int n_vec = (a.vocab - head) / E::kVec, behind = head + n_vec * E::kVec;
  const uint4* const v = reinterpret_cast<const uint4*>(src + head);
  int j = t;
  const auto batches = [&](auto n) {
    for (; j + (n.value - 1) * NT < n_vec; j += n.value * NT) {
      uint4 w[n.value];
#pragma unroll
      for (int i = 0; i < n.value; ++i) w[i] = __ldg(v + j + i * NT);
      batch(w, n);
    }
  };
  batches(std::integral_constant<int, kBatch>{});
  batches(std::integral_constant<int, kBatch / 2>{});
  batches(std::integral_constant<int, 1>{});
  if (t < head + a.vocab - behind) {
    const float x = E::load(src + (t < head ? t : behind + t - head));
    meet(x, x);
    add(x);
  }
  Stat st = {m, s.x + s.y, u.x + u.y};
#pragma unroll
  for (int d = 16; d > 0; d /= 2)
    st = join(st, {__shfl_xor_sync(0xffffffffu, st.m, d), __shfl_xor_sync(0xffffffffu, st.s, d),
                   __shfl_xor_sync(0xffffffffu, st.u, d)});
  if (NT > 32) {
    if (t % 32 == 0) sh[t / 32] = st;
    __syncthreads();
    if (t >= 32) return;
    if (t == 0)
      for (int w = 1; w < NT / 32; ++w) st = join(st, sh[w]);
  }
  if (is_far(__shfl_sync(0xffffffffu, st.m, 0))) {
    st = far_stat<T, 32>(src, a.vocab, a.inv_temperature, t, nullptr);
    if (t == 0) store_row<true>(a, row, st, target, x_target);
  } else if (t == 0) {
    store_row<false>(a, row, st, target, x_target);
  }
}

struct BwdArgs {
  const void* logits;
  void* d_logits;
  int64_t ld, ldd;
  int vocab, slice;
  const int32_t* targets;
  float inv_temperature;
  const float *lse, *entropy, *d_logprob, *d_entropy;
};

// From here on lse, in fp32, tells p to 2^-10 of itself or less (2^-24 |lse|), which a bf16 result shows; at
// 1e38 it does not tell a row's sum from its maximum.  The row is then summed again, and its
// gradient taken by distances from its maximum: by one team, as another slice's CTA may have
// overwritten the logits (d_logits may be the logits) before they are read.
constexpr float kFarLse = 16384.0f;
template <typename T, int NT>
__device__ __noinline__ void far_gradient(const T* src, T* dst, int vocab, float inv_t, int t, float* place, int target,
                                          float g, float gh, float entropy) {
  const Stat st = far_stat<T, NT>(src, vocab, inv_t, t, place);
  const float log_sum = log2f(st.s) * kLn2, base = fmaf(gh, entropy, g);
  each_of_row<T, NT>(src, vocab, t, [&](float x, int i) {
    const float logp = __fmul_rn(x, inv_t) - st.m - log_sum, p = ex2(logp * kLog2e);
    float d = p == 0.0f ? 0.0f : -p * fmaf(gh, logp, base);
    if (i == target) d += g;
    dst[i] = Elem<T>::store(d);
  });
}

// NT threads, a CTA or a warp of it, write one slice of a row.  Reads and writes every
// element once: HBM bounds it.  The row's four numbers are loaded once by each thread.
template <typename T, int NT>
__global__ void __launch_bounds__(kBwdThreads) logprobs_bwd_kernel(const BwdArgs a, int n_rows) {
  using E = Elem<T>;
  __shared__ float place[kBwdThreads / 32];
  grid_dependency_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kBwdThreads / NT) + threadIdx.x / NT;
  if (row >= n_rows) return;
  const int tid = threadIdx.x % NT;
  const T* const src = static_cast<const T*>(a.logits) + row * a.ld;
  T* const dst = static_cast<T*>(a.d_logits) + row * a.ldd;
  const int beg = blockIdx.y * a.slice, n = min(a.slice, a.vocab - beg);
  const float lse = a.lse[row], inv_t = a.inv_temperature;
  int target = a.targets ? a.targets[row] : -1;
  if (target < 0 || target >= a.vocab) target = -1;
  const float g = target >= 0 ? a.d_logprob[row] * inv_t : 0.0f;
  const float gh = a.entropy ? a.d_entropy[row] * inv_t : 0.0f;
  // -p (g + gh (log p + H)) + g [j = t], all times 1 / T
  const float base = a.entropy ? fmaf(gh, a.entropy[row], g) : g;
  const bool empty = lse == -INFINITY;
  if (fabsf(lse) >= kFarLse && fabsf(lse) < INFINITY) {
    if (blockIdx.y == 0)
      far_gradient<T, NT>(src, dst, a.vocab, inv_t, tid, place, target, g, gh, a.entropy ? a.entropy[row] : 0.0f);
    return;
  }
  target -= beg;
  const auto grad = [&](float x, int at) {
    const float logp = __fmul_rn(x, inv_t) - lse;
    const float p = ex2(logp * kLog2e);
    float d = p == 0.0f ? 0.0f : -p * fmaf(gh, logp, base);
    if (at == target) d += g;
    return empty ? 0.0f : d;
  };
  const T* const from = src + beg;
  T* const to = dst + beg;
  // both rows at the same place within 16 bytes: a scalar head up to the
  // boundary, whole vectors, a scalar tail
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(from) & 15);
  const bool together = off == (reinterpret_cast<uintptr_t>(to) & 15);
  const int head = together ? min(n, static_cast<int>((16 - off) % 16 / sizeof(T))) : n;
  for (int i = tid; i < head; i += NT) to[i] = E::store(grad(E::load(from + i), i));
  const int n_vec = (n - head) / E::kVec;
  const uint4* const v = reinterpret_cast<const uint4*>(from + head);
  uint4* const w = reinterpret_cast<uint4*>(to + head);
#pragma unroll 4
  for (int j = tid; j < n_vec; j += NT) {
    float x[E::kVec];
    E::unpack(v[j], x);
#pragma unroll
    for (int i = 0; i < E::kVec; ++i) x[i] = grad(x[i], head + j * E::kVec + i);
    w[j] = E::pack(x);
  }
  for (int i = head + n_vec * E::kVec + tid; i < n; i += NT) to[i] = E::store(grad(E::load(from + i), i));
}

// Cluster width and slice of the forward pass.  A slice above 72 KB would leave
// room for two CTAs on an SM only, too few copies in flight; with few rows the
// slices are halved until two CTAs an SM have work or 16 KB is reached, where
// the join costs as much as the slice.
int choose_cluster(int n_rows, int64_t row_bytes) {
  int c = 1;
  while (c < kMaxCluster && (row_bytes / c > 72 * 1024 ||
                             (static_cast<int64_t>(n_rows) * c < 2 * sm_count() && row_bytes / c > 16 * 1024)))
    c *= 2;
  return c;
}

// A warp a row for short rows, if every SM gets 8 of them (bf16, 8192 rows of 1000: 7.4 us, with a
// CTA a row 16.6; of 8000: 29.4 and 36.4; 1400 of 8000: 8.1 and 7.1; 700 of 3000: 4.2 and 3.3).
template <typename T>
bool warp_rows(int n_rows, int vocab) {
  return vocab * sizeof(T) <= 16384 && n_rows >= 8 * sm_count();
}

template <typename T, int NT>
int launch_rows(const LogprobsArgs& a, int n_rows, int cluster, cudaStream_t s) {
  const size_t smem = (static_cast<size_t>(a.slice) * sizeof(T) + 15) / 16 * 16 + 16;
  constexpr int kMaxSlice = ((kMaxVocab + kMaxCluster - 1) / kMaxCluster + 7) / 8 * 8;
  KV_TRY(set_max_dynamic_smem(reinterpret_cast<const void*>(logprobs_kernel<T, NT>),
                              static_cast<int>(kMaxSlice * sizeof(T) + 32)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n_rows) * cluster);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  LaunchScope scope(TWELL_KERNEL_LOGPROBS, s);
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, NT>, a) == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

template <typename T>
int launch_logprobs(LogprobsArgs a, int n_rows, cudaStream_t s) {
  const bool warps = warp_rows<T>(n_rows, a.vocab);
  if (a.top_k == 0 && (warps || n_rows >= kManyRows * sm_count())) {
    LaunchScope scope(TWELL_KERNEL_LOGPROBS, s);
    const int grid = warps ? (n_rows + kRowsThreads / 32 - 1) / (kRowsThreads / 32) : n_rows;
    return launch_pdl(warps ? logprobs_rows_kernel<T, 32> : logprobs_rows_kernel<T, kRowsThreads>, dim3(grid),
                      dim3(kRowsThreads), 0, s, a, n_rows) == cudaSuccess
               ? TWELL_OK
               : TWELL_ERR_CUDA;
  }
  const int c = choose_cluster(n_rows, static_cast<int64_t>(a.vocab) * sizeof(T));
  a.slice = ((a.vocab + c - 1) / c + 7) / 8 * 8;
  // One CTA or less an SM: its threads are all there are to hide the latencies, but two must fit, as the
  // SMs of a GPC need not be a multiple of a cluster (16 x 131072 fp32 with 20 alternatives: 9.0 us;
  // with 1024 threads, one of 16 clusters late, 15.6; with 256 9.1.  1 row: 7.3, 8.3 and 7.9).
  if (static_cast<int64_t>(n_rows) * c <= sm_count() && static_cast<int64_t>(a.slice) * sizeof(T) > 16 * 1024)
    return launch_rows<T, 512>(a, n_rows, c, s);
  // A slice's 16-byte pieces go to the threads in turn, and a group's maximum needs a piece: with
  // few pieces a group has to be one thread for enough groups to have one (6614 rows of 500 bf16 with 20 alternatives:
  // 33 us, with 256 threads and no bound 382).  Fewer pieces than alternatives give no bound either way.
  const int chunks = a.slice / Elem<T>::kVec;
  if (chunks >= a.top_k && chunks < 6 * a.top_k) return launch_rows<T, 64>(a, n_rows, c, s);
  return launch_rows<T, 256>(a, n_rows, c, s);
}

template <typename T>
int launch_logprobs_bwd(BwdArgs a, int n_rows, cudaStream_t s) {
  // slices of 32768 elements where there is work for all SMs several times over,
  // down to 2048 where there is not
  const int64_t share = static_cast<int64_t>(n_rows) * a.vocab / (8 * sm_count());
  a.slice = static_cast<int>(share > 32768 ? 32768 : share < 2048 ? 2048 : share) / 8 * 8;
  if (a.slice > a.vocab) a.slice = (a.vocab + 7) / 8 * 8;
  // a warp a row where that is 4 KB or less and every SM gets 16 (bf16, 8192 rows of 1000: 12.5 us,
  // with a CTA a row 14.9; 100000 of 100: 41 and 140)
  const bool warps = a.vocab * sizeof(T) <= 4096 && n_rows >= 16 * sm_count();
  if (warps) a.slice = a.vocab;
  const dim3 grid(warps ? (n_rows + kBwdThreads / 32 - 1) / (kBwdThreads / 32) : n_rows,
                  (a.vocab + a.slice - 1) / a.slice);
  LaunchScope scope(TWELL_KERNEL_LOGPROBS_BWD, s);
  return launch_pdl(warps ? logprobs_bwd_kernel<T, 32> : logprobs_bwd_kernel<T, kBwdThreads>, grid,
                    dim3(kBwdThreads), 0, s, a, n_rows) == cudaSuccess
             ? TWELL_OK
             : TWELL_ERR_CUDA;
}

int check_logits(const void* logits, int dtype, int64_t ld, int n_rows, int vocab, float inv_temperature) {
  if (n_rows < 0 || vocab < 1 || ld < vocab) return TWELL_ERR_INVALID_ARG;
  if (dtype != TWELL_BF16 && dtype != TWELL_F32) return TWELL_ERR_INVALID_ARG;
  if (!(inv_temperature > 0.0f) || inv_temperature > 3.0e38f) return TWELL_ERR_INVALID_ARG;
  if (vocab > kMaxVocab || n_rows > INT_MAX / kMaxCluster) return TWELL_ERR_UNSUPPORTED;
  return n_rows > 0 ? check_array(logits, 16) : TWELL_OK;
}

}  // namespace
}  // namespace twell

using namespace twell;

extern "C" TWELL_API int twell_logprobs(const void* logits, int32_t dtype, int64_t ld, int32_t n_rows, int32_t vocab,
                                        const int32_t* targets, float inv_temperature, float* logprob,
                                        float* entropy, float* lse, int32_t top_k, float* top_logprob,
                                        int32_t* top_index, twell_stream_t stream) {
  KV_TRY(check_logits(logits, dtype, ld, n_rows, vocab, inv_temperature));
  if (top_k < 0) return TWELL_ERR_INVALID_ARG;
  if (top_k > kMaxTop || top_k > vocab) return TWELL_ERR_UNSUPPORTED;
  if (n_rows > 0) {
    if (!targets != !logprob) return TWELL_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(targets), static_cast<const void*>(logprob),
                          static_cast<const void*>(entropy), static_cast<const void*>(lse)})
      if (!aligned_to(p, 4)) return TWELL_ERR_MISALIGNED;
    if (top_k > 0) {
      KV_TRY(check_array(top_logprob, 4));
      KV_TRY(check_array(top_index, 4));
    }
  }
  if (!device_is_sm103()) return TWELL_ERR_NO_DEVICE;
  if (n_rows == 0) return TWELL_OK;
  const LogprobsArgs a{logits, ld, vocab, 0, targets, inv_temperature, logprob, entropy, lse,
                       top_k, top_logprob, top_index};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == TWELL_BF16 ? launch_logprobs<uint16_t>(a, n_rows, s) : launch_logprobs<float>(a, n_rows, s);
}

extern "C" TWELL_API int twell_logprobs_bwd(const void* logits, int32_t dtype, int64_t ld, int32_t n_rows,
                                            int32_t vocab, const int32_t* targets, float inv_temperature,
                                            const float* lse, const float* entropy, const float* d_logprob,
                                            const float* d_entropy, void* d_logits, int64_t ldd,
                                            twell_stream_t stream) {
  KV_TRY(check_logits(logits, dtype, ld, n_rows, vocab, inv_temperature));
  if (ldd < vocab) return TWELL_ERR_INVALID_ARG;
  if (n_rows > 0) {
    KV_TRY(check_array(lse, 4));
    KV_TRY(check_array(d_logits, 16));
    if (!targets != !d_logprob || !entropy != !d_entropy) return TWELL_ERR_INVALID_ARG;
    if (d_logits == logits && ldd != ld) return TWELL_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(targets), static_cast<const void*>(d_logprob),
                          static_cast<const void*>(entropy), static_cast<const void*>(d_entropy)})
      if (!aligned_to(p, 4)) return TWELL_ERR_MISALIGNED;
  }
  if (!device_is_sm103()) return TWELL_ERR_NO_DEVICE;
  if (n_rows == 0) return TWELL_OK;
  const BwdArgs a{logits, d_logits, ld, ldd, vocab, 0, targets, inv_temperature, lse, entropy, d_logprob, d_entropy};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == TWELL_BF16 ? launch_logprobs_bwd<uint16_t>(a, n_rows, s) : launch_logprobs_bwd<float>(a, n_rows, s);
}
