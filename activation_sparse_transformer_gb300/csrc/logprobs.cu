// Log probabilities of given tokens with entropy and best alternatives
// (twell_logprobs) and their gradient (twell_logprobs_bwd).
//
// With x = logits / T, m = max x, S = sum exp(x - m), U = sum exp(x - m) (x - m):
//   lse = m + log S,  logprob = (x_t - m) - log S,  entropy = log S - U / S.
// A row is read from memory once: a CTA (or a cluster of 2 to 8 for long rows
// and few of them) copies its slice to shared memory with asynchronous 16-byte
// copies, finds the maximum there and then sums with it, so no running maximum has
// to be corrected; slices are joined through distributed shared memory.  HBM
// bounds many rows; few rows are bound by the latency of one slice.
//
// The k largest: the k-th largest of the 256 threads' own maxima is a lower bound
// of the k-th largest value, and hardly more than k values reach it.  Those are
// collected and ranked by counting.  Keys are (value, index) pairs in one
// 64-bit word, so equal values go by index and no two keys are equal.
#include <cooperative_groups.h>

#include <cfloat>
#include <climits>

#include "kv_internal.h"

namespace cg = cooperative_groups;

namespace twell {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr int kCandidates = 1024;
constexpr int kMaxVocab = 400000;
constexpr float kLog2e = 1.4426950408889634f;

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
  static __device__ __forceinline__ float lowest() { return -INFINITY; }
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
  static __device__ __forceinline__ uint16_t lowest() { return 0xFF80u; }
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

// Stats relative to a common maximum; an empty part has s = u = 0.
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b) {
  const float m = fmaxf(a.m, b.m);
  const float ea = ex2((a.m - m) * kLog2e), eb = ex2((b.m - m) * kLog2e);
  return {m, a.s * ea + b.s * eb, ea * (a.u + a.s * (a.m - m)) + eb * (b.u + b.s * (b.m - m))};
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

struct LpShared {
  uint64_t thread_key[kLpThreads];   // then: the cluster's lists
  uint64_t candidates[kCandidates];
  uint64_t best[kMaxTop];
  uint64_t bound;
  Stat stat;
  float warp_m[kLpWarps];
  Stat warp_stat[kLpWarps];
  uint64_t warp_key[kLpWarps];
  int count;
};

// The top_k best keys of the CTA's slice to sh.best, in order, 0 behind the last.
template <typename T>
__device__ void slice_top(LpShared& sh, const uint4* chunks, int n_chunks, int index0, int slice_n, float inv_t, int k,
                          uint64_t mine) {
  using E = Elem<T>;
  const int tid = threadIdx.x;
  sh.thread_key[tid] = mine;
  if (tid < kMaxTop) sh.best[tid] = 0;
  if (tid == 0) {
    sh.count = 0;
    sh.bound = 1;  // every key is larger: fewer than k threads have one
  }
  __syncthreads();
  int better = 0;
  for (int i = 0; i < kLpThreads; ++i) better += sh.thread_key[i] > mine;
  if (better == k - 1 && mine) sh.bound = mine;
  __syncthreads();
  const uint64_t bound = sh.bound;
  const auto each = [&](auto&& f) {
    for (int j = tid; j < n_chunks; j += kLpThreads) {
      float x[E::kVec];
      E::unpack(chunks[j], x);
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) {
        const int at = j * E::kVec + i - index0;
        if (at >= 0 && at < slice_n) f(key_of(x[i] * inv_t, at));
      }
    }
  };
  each([&](uint64_t key) {
    if (key >= bound) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kCandidates) sh.candidates[at] = key;
    }
  });
  __syncthreads();
  if (sh.count <= kCandidates) {
    const int n = sh.count;
    for (int c = tid; c < n; c += kLpThreads) {
      const uint64_t key = sh.candidates[c];
      int rank = 0;
      for (int i = 0; i < n; ++i) rank += sh.candidates[i] > key;
      if (rank < k) sh.best[rank] = key;
    }
  } else {
    // rare: a few threads own most of the largest values; take them one by one
    uint64_t last = ~0ull;
    for (int i = 0; i < k; ++i) {
      uint64_t top = 0;
      each([&](uint64_t key) {
        if (key < last && key > top) top = key;
      });
#pragma unroll
      for (int d = 16; d > 0; d /= 2) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, top, d);
        top = o > top ? o : top;
      }
      if ((tid & 31) == 0) sh.warp_key[tid / 32] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kLpWarps; ++w) top = sh.warp_key[w] > top ? sh.warp_key[w] : top;
      if (tid == 0) sh.best[i] = top;
      last = top;
      __syncthreads();
    }
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const LogprobsArgs a) {
  using E = Elem<T>;
  extern __shared__ uint4 chunks[];
  __shared__ LpShared sh;
  grid_dependency_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int64_t row = blockIdx.x / ranks;
  const T* const src = static_cast<const T*>(a.logits) + row * a.ld;
  const int beg = min(rank * a.slice, a.vocab), n = min(a.slice, a.vocab - beg);
  // the slice with the 16-byte pieces it touches; the pieces' other elements
  // are replaced by -inf, and the last, cut piece comes in by elements
  const T* const from = src + beg;
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(from) & 15) / sizeof(T));
  const int n_chunks = n > 0 ? (lead + n + E::kVec - 1) / E::kVec : 0, whole = (lead + n) / E::kVec;
  const uint4* const g = reinterpret_cast<const uint4*>(from - lead);
  for (int j = tid; j < whole && n > 0; j += kLpThreads)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(chunks + j)), "l"(g + j) : "memory");
  T* const elems = reinterpret_cast<T*>(chunks);
  for (int i = whole * E::kVec + tid; i < n_chunks * E::kVec; i += kLpThreads)
    elems[i] = i >= lead && i < lead + n ? from[i - lead] : E::lowest();
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if (whole > 0 && tid < lead) elems[tid] = E::lowest();
  if (lead) __syncthreads();

  float m = -FLT_MAX;
  uint64_t mine = 0;
  if (a.top_k > 0) {
    float best = -INFINITY;
    int at = INT_MAX;
    for (int j = tid; j < n_chunks; j += kLpThreads) {
      float x[E::kVec];
      E::unpack(chunks[j], x);
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) {
        const float v = x[i] * a.inv_temperature;
        const int index = j * E::kVec + i - lead;
        if (v > best || (at == INT_MAX && index >= 0 && index < n)) best = v, at = index;
      }
    }
    if (at != INT_MAX) mine = key_of(best, at);
    m = fmaxf(m, best);
  } else {
    float best = -INFINITY;
    for (int j = tid; j < n_chunks; j += kLpThreads) {
      float x[E::kVec];
      E::unpack(chunks[j], x);
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) best = fmaxf(best, x[i]);
    }
    m = fmaxf(m, best * a.inv_temperature);
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((tid & 31) == 0) sh.warp_m[tid / 32] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) m = fmaxf(m, sh.warp_m[w]);

  float s = 0.0f, u = 0.0f;
  for (int j = tid; j < n_chunks; j += kLpThreads) {
    float x[E::kVec];
    E::unpack(chunks[j], x);
#pragma unroll
    for (int i = 0; i < E::kVec; ++i) {
      // the product rounded as m's was: fused, a row of -1e30 would be far from its own maximum
      const float d = __fmul_rn(x[i], a.inv_temperature) - m;
      const float e = ex2(d * kLog2e);
      s += e;
      u = fmaf(e, fmaxf(d, -1000.0f), u);  // a masked token adds 0, not 0 * inf
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    s += __shfl_xor_sync(0xffffffffu, s, d);
    u += __shfl_xor_sync(0xffffffffu, u, d);
  }
  if ((tid & 31) == 0) sh.warp_stat[tid / 32] = {m, s, u};
  __syncthreads();
  if (tid == 0) {
    Stat all = {m, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kLpWarps; ++w) all.s += sh.warp_stat[w].s, all.u += sh.warp_stat[w].u;
    sh.stat = all;
  }
  if (a.top_k > 0) slice_top<T>(sh, chunks, n_chunks, lead, n, a.inv_temperature, a.top_k, mine);
  if (ranks > 1) {
    cluster.sync();
    if (rank == 0) {
      if (tid == 0) {
        Stat all = sh.stat;
        for (int i = 1; i < ranks; ++i) all = join(all, *cluster.map_shared_rank(&sh.stat, i));
        sh.stat = all;
      }
      // the ranks' lists, indexes made those of the row, ranked together
      const int of = tid / kMaxTop, i = tid % kMaxTop;
      uint64_t key = 0;
      if (of < ranks && i < a.top_k) {
        key = cluster.map_shared_rank(&sh, of)->best[i];
        if (key) key -= static_cast<uint64_t>(of) * a.slice;
      }
      if (a.top_k > 0) {
        sh.thread_key[tid] = key;
        __syncthreads();
        int better = 0;
        for (int j = 0; j < kLpThreads; ++j) better += sh.thread_key[j] > key;
        __syncthreads();
        if (key && better < a.top_k) sh.best[better] = key;
      }
    }
    cluster.sync();  // the other ranks' shared memory is read above
  }
  if (rank != 0) return;
  __syncthreads();
  const Stat st = sh.stat;
  const bool broken = isnan(st.s), empty = !broken && st.s == 0.0f;
  const float log_s = logf(st.s);
  const float nan = __int_as_float(0x7FC00000);
  if (tid == 0) {
    if (a.lse) a.lse[row] = broken ? nan : empty ? -INFINITY : st.m + log_s;
    if (a.entropy) a.entropy[row] = broken ? nan : empty ? 0.0f : log_s - st.u / st.s;
    if (a.targets) {
      const int t = a.targets[row];
      float lp = 0.0f;
      if (t >= 0 && t < a.vocab) {
        const float x = E::load(src + t) * a.inv_temperature;
        lp = broken ? nan : empty ? -INFINITY : (x - st.m) - log_s;
      }
      a.logprob[row] = lp;
    }
  }
  if (tid < a.top_k) {
    const uint64_t key = sh.best[tid];
    const float x = key_value(key);
    a.top_logprob[row * a.top_k + tid] = broken ? nan : empty ? -INFINITY : (x - st.m) - log_s;
    a.top_index[row * a.top_k + tid] = broken ? -1 : key_index(key);
  }
}

struct BwdArgs {
  const void* logits;
  void* d_logits;
  int64_t ld, ldd;
  int vocab, slice, slices;
  const int32_t* targets;
  float inv_temperature;
  const float *lse, *entropy, *d_logprob, *d_entropy;
};

// One CTA writes one slice of a row.  Reads and writes every element once:
// HBM bounds it.  The row's four numbers are loaded once per CTA.
template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_bwd_kernel(const BwdArgs a) {
  using E = Elem<T>;
  grid_dependency_wait();
  const int64_t row = blockIdx.x / a.slices;
  const int tid = threadIdx.x;
  const T* const src = static_cast<const T*>(a.logits) + row * a.ld;
  T* const dst = static_cast<T*>(a.d_logits) + row * a.ldd;
  const int beg = (blockIdx.x % a.slices) * a.slice, n = min(a.slice, a.vocab - beg);
  const float lse = a.lse[row], inv_t = a.inv_temperature;
  int target = a.targets ? a.targets[row] : -1;
  if (target < 0 || target >= a.vocab) target = -1;
  const float g = target >= 0 ? a.d_logprob[row] * inv_t : 0.0f;
  const float gh = a.entropy ? a.d_entropy[row] * inv_t : 0.0f;
  // -p (g + gh (log p + H)) + g [j = t], all times 1 / T
  const float base = a.entropy ? fmaf(gh, a.entropy[row], g) : g;
  const bool empty = lse == -INFINITY;
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
  for (int i = tid; i < head; i += kLpThreads) to[i] = E::store(grad(E::load(from + i), i));
  const int n_vec = (n - head) / E::kVec;
  const uint4* const v = reinterpret_cast<const uint4*>(from + head);
  uint4* const w = reinterpret_cast<uint4*>(to + head);
#pragma unroll 4
  for (int j = tid; j < n_vec; j += kLpThreads) {
    float x[E::kVec];
    E::unpack(v[j], x);
#pragma unroll
    for (int i = 0; i < E::kVec; ++i) x[i] = grad(x[i], head + j * E::kVec + i);
    w[j] = E::pack(x);
  }
  for (int i = head + n_vec * E::kVec + tid; i < n; i += kLpThreads) to[i] = E::store(grad(E::load(from + i), i));
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

template <typename T>
int launch_logprobs(LogprobsArgs a, int n_rows, cudaStream_t s) {
  const int c = choose_cluster(n_rows, static_cast<int64_t>(a.vocab) * sizeof(T));
  a.slice = ((a.vocab + c - 1) / c + 7) / 8 * 8;
  const size_t smem = (static_cast<size_t>(a.slice) * sizeof(T) + 15) / 16 * 16 + 16;
  constexpr int kMaxSlice = ((kMaxVocab + kMaxCluster - 1) / kMaxCluster + 7) / 8 * 8;
  KV_TRY(set_max_dynamic_smem(reinterpret_cast<const void*>(logprobs_kernel<T>),
                              static_cast<int>(kMaxSlice * sizeof(T) + 32)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n_rows) * c);
  cfg.blockDim = dim3(kLpThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  LaunchScope scope(TWELL_KERNEL_LOGPROBS, s);
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, a) == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

template <typename T>
int launch_logprobs_bwd(BwdArgs a, int n_rows, cudaStream_t s) {
  // whole rows of up to 32768 elements; longer ones, or few, in slices of 8192
  a.slice = a.vocab <= 32768 && n_rows >= 4 * sm_count() ? (a.vocab + 7) / 8 * 8 : 8192;
  a.slices = (a.vocab + a.slice - 1) / a.slice;
  if (static_cast<int64_t>(n_rows) * a.slices > INT_MAX) return TWELL_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(n_rows) * a.slices);
  LaunchScope scope(TWELL_KERNEL_LOGPROBS_BWD, s);
  return launch_pdl(logprobs_bwd_kernel<T>, grid, dim3(kLpThreads), 0, s, a) == cudaSuccess ? TWELL_OK
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
  const BwdArgs a{logits, d_logits, ld, ldd, vocab, 0, 0, targets, inv_temperature, lse, entropy, d_logprob, d_entropy};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == TWELL_BF16 ? launch_logprobs_bwd<uint16_t>(a, n_rows, s) : launch_logprobs_bwd<float>(a, n_rows, s);
}
