// The norms before and after a block, its gate and the residual sum in one
// pass (twell_block_norm), and their gradient (twell_block_norm_bwd).
//
//   r1 = (mean y^2 + eps)^-1/2,  u = y r1 w_post  (or u = y)
//   z = skip x + branch row_gate gate u
//   r2 = (mean z^2 + eps)^-1/2,  h = z r2 w_pre
//
// Backward, with v = z r2, a = dh w_pre and s = y r1 (or y):
//   dz = d_out + r2 (a - v mean(a v)),  dx = skip dz,  dw_pre = sum_n dh v
//   P = sum_n branch row_gate dz s:  dw_post = gate P,  dgate = w_post P
//   t = branch row_gate gate w_post dz:  dy = r1 (t - s mean(t s))  (or t)
//   drow_gate = sum_c branch gate w_post dz s
// so the two vectors of the branch share one sum over the rows.
//
// A row is taken by a group of threads, 16 elements a thread, and is read from memory once; up to 256
// columns several rows share a warp.  One CTA an SM stays and takes rows in turn, several groups side by
// side; each thread copies its own elements of the next rows into its own shared memory
// asynchronously, which keeps enough bytes on the way without a barrier or a register, and reads
// them from there once for each pass over the row.  Arithmetic goes two fp32 lanes an
// instruction: with one, instructions bound it (8192 x 2048 bf16: 31 us forward, 54 backward).  The
// gradient's three sums of a row are taken together:
//   sum t s / scale = sum w (d_out + r2 a) s - r2 c2 sum w v s,  c2 = mean(a v), w = gate w_post.
// HBM bounds long calls (16384 x 2048 bf16: 48 us, 5.6 TB/s; gradient 71 us, 5.7 TB/s; 8192 rows 26 and 41, where
// starting and the sum over the CTAs are 5 and 8 of it), the launch and a row's chain of two sums short
// ones (16 x 4096: 2.8 us).  The gradient keeps its sums over the rows in registers, so its CTAs have 512
// threads (with 640 or 768 they spill: 54 and 65 us), and rows of 4104 to 8191 columns leave it one group
// an SM (8000 x 4104: 116 us, 3.4 TB/s; forward, 1024 threads, 53).  Above 8192 columns two CTAs share a row
// and its sums, through each other's shared memory (2048 x 16384: 80 us, gradient 108).
// All sums are fp32: a thread's own elements in order, then a tree over the group; sums over the
// rows by groups, CTAs and then runs of CTAs in order, so equal calls give equal bits.
#include <algorithm>

#include "kv_internal.h"

namespace twell {
namespace {

constexpr int kMaxDim = 16384;
constexpr int kMaxParts = 160;      // CTAs that leave sums of their rows
constexpr int kMaxBarriers = 15;    // groups of more than a warp in a CTA
constexpr int kMaxStages = 4;       // rows on the way to a thread
constexpr int kSharedBytes = 208 * 1024;  // beside 12 KB for the sums
constexpr int kV = 2;               // pieces of 8 elements a thread
constexpr int kThreads = 1024, kBwdThreads = 512;  // of a CTA: what registers allow
// Above, two CTAs share a row, so that its weights and the sums over the rows stay where they are (read anew for
// each row and with spills, 2048 x 16384 took 88 us, the gradient 206; now 80 and 108).  A barrier of the pair is
// dearer than one of a CTA's, so narrower rows stay in one (4096 x 8192: 49 us, in two 77; gradient 81 and 101; 8176 x 4104 53
// and 92; 119 and 127).
constexpr int kWide = 8192;

struct NormArgs {
  const void* x;
  const uint16_t* y;
  void* x_out;
  uint16_t* h;
  int64_t ldx, ldy, ldo, ldh;
  int n_rows, dim, group, stages;  // group: threads of a row
  const void *w_post, *gate, *w_pre;
  bool w_f32;
  const float* row_gate;
  float skip, branch, eps;
  float *rstd_post, *rstd_pre;
};

struct NormBwdArgs {
  const uint16_t* dh;
  const void* d_out;
  const void* z;
  const uint16_t* y;
  void* dx;
  uint16_t* dy;
  int64_t lddh, lddo, ldz, ldy, lddx, lddy;
  int n_rows, dim, group, stages;
  const void *w_post, *gate, *w_pre;
  bool w_f32;
  const float* row_gate;
  float skip, branch;
  const float *rstd_post, *rstd_pre;
  float* drow_gate;
  bool want_pre, want_branch;  // sums over the rows that are asked for
  float* part;                 // [parts][2][dim]: sum dh v, then P
};

// Two fp32 lanes, one instruction an operation.
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
__device__ __forceinline__ float both(F2 a) {
  const float2 f = lanes(a);
  return f.x + f.y;
}

// A thread's 8 elements of a piece.
struct Oct {
  F2 v[4];
};
__device__ __forceinline__ Oct from_bf16(const uint4& w) {
  return Oct{{pair(bf16_lo(w.x), bf16_hi(w.x)), pair(bf16_lo(w.y), bf16_hi(w.y)), pair(bf16_lo(w.z), bf16_hi(w.z)),
              pair(bf16_lo(w.w), bf16_hi(w.w))}};
}
__device__ __forceinline__ Oct from_f32(const float4& a, const float4& b) {
  return Oct{{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
}
__device__ __forceinline__ uint32_t bf16_word(F2 a) {
  const float2 f = lanes(a);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(f.y), "f"(f.x));
  return r;
}
__device__ __forceinline__ float weight1(const void* p, bool f32, int c) {
  return f32 ? static_cast<const float*>(p)[c] : bf16_bits_to_float(static_cast<const uint16_t*>(p)[c]);
}

// The sum of the warps' sums (zero past the group's warps).
__device__ __forceinline__ float warp_sums(const float* scratch, int group) {
  const float4* const at = reinterpret_cast<const float4*>(scratch);
  float4 a = at[0];
  if (group > 128) {  // more than 4 warps
    const float4 b = at[1];
    a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
    for (int k = 2; k * 128 < group; ++k) {
      const float4 c = at[k];
      a.x += c.x, a.y += c.y, a.z += c.z, a.w += c.w;
    }
  }
  return (a.x + a.y) + (a.z + a.w);
}

// How a row's threads lie: in a part of a warp, in whole warps of a CTA, or in both CTAs of a cluster.
enum Span { kSub, kCta, kPair };

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// A barrier of the cluster's threads; what was written to either shared memory is there after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// A warp's sum to its place in the shared memory of both CTAs.
__device__ __forceinline__ void tell_both(float* at, float v) {
  *at = v;
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, %1;\n\tst.shared::cluster.f32 [r], %2;\n\t}" ::"r"(smem_u32(at)),
      "r"(cluster_rank() ^ 1), "f"(v)
      : "memory");
}

// K sums over the group's threads at once, in every thread of it.  scratch: [K][32] floats of the group's own, zero past its
// warps; free again once the group has passed another such barrier.
template <Span SPAN, int K>
__device__ __forceinline__ void group_sums(float (&v)[K], int group, int id, int thread, float* scratch) {
  for (int o = SPAN == kSub ? group >> 1 : 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (SPAN == kSub || (SPAN == kCta && group == 32)) return;
  if ((thread & 31) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float* const at = scratch + k * 32 + (thread >> 5);
      if constexpr (SPAN == kPair)
        tell_both(at, v[k]);
      else
        *at = v[k];
    }
  }
  if constexpr (SPAN == kPair)
    cluster_sync();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(group) : "memory");
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sums(scratch + k * 32, group);
}

__device__ __forceinline__ void copy16(uint8_t* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint8_t* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest `stages - 1` groups of this thread's copies have landed.
__device__ __forceinline__ void copies_wait(int stages) {
  if (stages == 1)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (stages == 2)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (stages == 3)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// Which columns a thread has.  A piece is 8 elements a thread: with a bf16 stream 8 in a
// row, with fp32 two runs of 4, `group` runs apart, so that every access of a warp is one run of whole lines
// (8 in a row of fp32 are two accesses of half of every line: 8192 x 2048, 42 us).
// In shared memory a piece is 16 bytes a thread, or two planes of them in fp32, those of a CTA's threads side by
// side (`pitch` bytes together).  Columns past the row are zero there and in the weights, so they add nothing.
template <typename T>
struct Layout {
  static constexpr int kRuns = sizeof(T) / 2, kRun = 8 / kRuns;
  static constexpr int kPieces = kRuns;  // 16-byte pieces of the stream's 8 elements
  int dim, first, step;  // a run's column is first + its number * step

  __device__ __forceinline__ int column(int i, int q) const { return first + (i * kRuns + q) * step; }
  __device__ __forceinline__ bool on(int i, int q) const { return column(i, q) < dim; }

  __device__ __forceinline__ void copy(uint8_t* at, int pitch, const T* row, int i) const {
#pragma unroll
    for (int q = 0; q < kRuns; ++q)
      if (on(i, q)) copy16(at + q * pitch, row + column(i, q));
  }
  __device__ __forceinline__ void copy_bf16(uint8_t* at, const uint16_t* row, int i) const {
    if constexpr (kRuns == 1) {
      if (on(i, 0)) copy16(at, row + column(i, 0));
    } else {
#pragma unroll
      for (int q = 0; q < kRuns; ++q)
        if (on(i, q)) copy8(at + 8 * q, row + column(i, q));
    }
  }
  static __device__ __forceinline__ Oct read(const uint8_t* at, int pitch) {
    if constexpr (kRuns == 1)
      return read_bf16(at);
    else
      return from_f32(*reinterpret_cast<const float4*>(at), *reinterpret_cast<const float4*>(at + pitch));
  }
  static __device__ __forceinline__ Oct read_bf16(const uint8_t* at) {
    return from_bf16(*reinterpret_cast<const uint4*>(at));
  }
  __device__ __forceinline__ void write(T* row, int i, const Oct& o) const {
    if constexpr (kRuns == 1)
      write_bf16(row, i, o);
    else
      write_f32(row, i, o);
  }
  __device__ __forceinline__ void write_bf16(uint16_t* row, int i, const Oct& o) const {
    const uint4 w = make_uint4(bf16_word(o.v[0]), bf16_word(o.v[1]), bf16_word(o.v[2]), bf16_word(o.v[3]));
    if constexpr (kRuns == 1) {
      if (on(i, 0)) *reinterpret_cast<uint4*>(row + column(i, 0)) = w;
    } else {
      if (on(i, 0)) *reinterpret_cast<uint2*>(row + column(i, 0)) = make_uint2(w.x, w.y);
      if (on(i, 1)) *reinterpret_cast<uint2*>(row + column(i, 1)) = make_uint2(w.z, w.w);
    }
  }
  // fp32, wherever the runs are
  __device__ __forceinline__ void write_f32(float* row, int i, const Oct& o) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 a = lanes(o.v[2 * h]), b = lanes(o.v[2 * h + 1]);
      const int c = kRuns == 1 ? column(i, 0) + 4 * h : column(i, h);
      if (c < dim) *reinterpret_cast<float4*>(row + c) = make_float4(a.x, a.y, b.x, b.y);
    }
  }
  __device__ __forceinline__ Oct read_f32(const float* row, int i) const {  // of columns that are on, else 0
    float4 f[2] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = kRuns == 1 ? column(i, 0) + 4 * h : column(i, h);
      if (c < dim) f[h] = *reinterpret_cast<const float4*>(row + c);
    }
    return from_f32(f[0], f[1]);
  }
};

// The product of the branch's weights, and the next norm's weight, as fp32 in shared memory: [2]
// planes of a thread's 16-byte pieces, read without conflicts.
template <typename T>
struct Weights {
  static constexpr int V = kV;
  uint8_t* base;  // [branch, pre][piece][2][group] of 16 bytes; group: of this CTA
  const void *post, *gate, *pre;
  bool f32;
  int group, thread;
  Layout<T> at;

  // a run of a vector as fp32 (1 without one)
  __device__ __forceinline__ void run(const void* p, int c, float (&f)[Layout<T>::kRun]) const {
    constexpr int R = Layout<T>::kRun;
#pragma unroll
    for (int e = 0; e < R; e += 4) {
      float4 v = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
      if (p && f32) {
        v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + e);
      } else if (p) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + c + e);
        v = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
      }
      f[e] = v.x, f[e + 1] = v.y, f[e + 2] = v.z, f[e + 3] = v.w;
    }
  }
  __device__ __forceinline__ Oct make(bool branch, int i) const {
    constexpr int R = Layout<T>::kRun;
    float f[8] = {};
#pragma unroll
    for (int q = 0; q < Layout<T>::kRuns; ++q) {
      if (!at.on(i, q)) continue;
      float x[R], y[R];
      run(branch ? post : pre, at.column(i, q), x);
      run(branch ? gate : nullptr, at.column(i, q), y);
#pragma unroll
      for (int e = 0; e < R; ++e) f[q * R + e] = x[e] * y[e];
    }
    return Oct{{pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7])}};
  }
  __device__ __forceinline__ ulonglong2* slot(bool branch, int i, int h) const {
    return reinterpret_cast<ulonglong2*>(base) + (((branch ? 0 : V) + i) * 2 + h) * group + thread;
  }
  // by the first group's threads, a barrier before the first use
  __device__ __forceinline__ void fill() const {
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) {
      const Oct w = make(i < V, i % V);
      *slot(i < V, i % V, 0) = make_ulonglong2(w.v[0], w.v[1]);
      *slot(i < V, i % V, 1) = make_ulonglong2(w.v[2], w.v[3]);
    }
  }
  __device__ __forceinline__ Oct get(bool branch, int i) const {
    const ulonglong2 a = *slot(branch, i, 0), b = *slot(branch, i, 1);
    return Oct{{a.x, a.y, b.x, b.y}};
  }
};

// What the two kernels set up alike.
template <typename T, Span SPAN>
struct Setup {
  static constexpr int V = kV;
  int groups, id, thread, pitch, rows;  // rows: of a warp
  int team, teams;                      // CTAs that deal with rows, alone or as pairs
  Layout<T> at;
  Weights<T> weights;
  uint8_t *ring, *mine;
  __device__ __forceinline__ Setup(uint8_t* smem, int group, int dim, const void* post, const void* gate,
                                   const void* pre, bool f32) {
    constexpr int kCtas = SPAN == kPair ? 2 : 1;
    const int here = group / kCtas;  // threads of a row in this CTA
    groups = blockDim.x / here, id = threadIdx.x / here, thread = threadIdx.x % here;
    team = blockIdx.x / kCtas, teams = gridDim.x / kCtas;
    pitch = blockDim.x * 16, rows = SPAN == kSub ? 32 / group : 1;
    weights = Weights<T>{smem, post, gate, pre, f32, here, thread};
    if constexpr (SPAN == kPair) thread += cluster_rank() * here;
    weights.at = at = Layout<T>{dim, thread * Layout<T>::kRun, group * Layout<T>::kRun};
    ring = smem + 2 * V * 2 * 16 * here;
    mine = ring + threadIdx.x * 16;
  }
  // The first row of those that stay together, which loops go by: a warp's, or (their barrier is one) a pair's.
  __device__ __forceinline__ int64_t first_row(int64_t row) const {
    return SPAN == kSub ? row - id % rows : SPAN == kPair ? row - id : row;
  }
  // Zeros where no copy goes.
  __device__ __forceinline__ void clear(int pieces) const {
    if (at.on(V - 1, Layout<T>::kRuns - 1)) return;
    for (int p = 0; p < pieces; ++p) *reinterpret_cast<uint4*>(mine + p * pitch) = make_uint4(0, 0, 0, 0);
  }
  // All that was set up is there: the weights, and in a pair the other CTA with its scratch.
  __device__ __forceinline__ void ready() const {
    if (id == 0) weights.fill();
    if constexpr (SPAN == kPair)
      cluster_sync();
    else
      __syncthreads();
  }
};

// A row for each group of threads in turn; Y: there is a block's output.
template <typename T, int NT, Span SPAN, bool Y>
__global__ void __launch_bounds__(NT, 1) block_norm_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float scratch[kMaxBarriers][2][2][32];  // two sums of a row, rows in turn
  for (int i = threadIdx.x; i < kMaxBarriers * 128; i += blockDim.x) (&scratch[0][0][0][0])[i] = 0.0f;
  grid_dependency_wait();
  constexpr int V = kV;
  const Setup<T, SPAN> g(smem, a.group, a.dim, a.w_post, a.gate, a.w_pre, a.w_f32);
  const Layout<T>& at = g.at;
  constexpr int kX = Layout<T>::kPieces, kPieces = kX + (Y ? 1 : 0);  // of x, of y
  const int pitch = g.pitch, step = g.teams * g.groups;
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  g.clear(a.stages * V * kPieces);
  int64_t row = static_cast<int64_t>(g.team) * g.groups + g.id, next = row;
  auto copy = [&](uint8_t* to) {
    if (next < a.n_rows) {
      const T* const x = static_cast<const T*>(a.x) + next * a.ldx;
      const uint16_t* const y = Y ? a.y + next * a.ldy : nullptr;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        at.copy(to + i * kPieces * pitch, pitch, x, i);
        if (Y) at.copy_bf16(to + (i * kPieces + kX) * pitch, y, i);
      }
    }
    copies_commit();
    next += step;
  };
#pragma unroll 1
  for (int s = 0; s < a.stages; ++s) copy(g.mine + s * V * kPieces * pitch);
  float gate = a.branch;  // of a row, read a row ahead
  if (Y && a.row_gate && row < a.n_rows) gate *= a.row_gate[row];
  g.ready();
  const F2 skip = pair(a.skip, a.skip);
  uint8_t* from = g.mine;
  int stage = 0, turn = 0;
  const int own = a.group > 32 ? g.id : 0;  // smaller groups use no scratch
#pragma unroll 1
  for (; g.first_row(row) < a.n_rows; row += step, turn ^= 1) {
    const bool live = SPAN == kCta || row < a.n_rows;
    float scale = gate;
    if (Y && a.row_gate && row + step < a.n_rows) gate = a.branch * a.row_gate[row + step];
    copies_wait(a.stages);
    F2 sum = 0;
    if (Y && a.w_post) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const Oct y = at.read_bf16(from + (i * kPieces + kX) * pitch);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum = fma2(y.v[k], y.v[k], sum);
      }
      float s[1] = {both(sum)};
      group_sums<SPAN>(s, a.group, g.id, g.thread, scratch[own][0][turn]);
      const float r1 = rsqrtf(fmaf(s[0], inv_dim, a.eps));
      if (live && g.thread == 0 && a.rstd_post) a.rstd_post[row] = r1;
      scale *= r1;
    }
    Oct z[V];
    const F2 scale2 = pair(scale, scale);
    sum = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const Oct x = at.read(from + i * kPieces * pitch, pitch);
      Oct y, w;
      if (Y) y = at.read_bf16(from + (i * kPieces + kX) * pitch), w = g.weights.get(true, i);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const F2 xs = mul2(x.v[k], skip);
        z[i].v[k] = Y ? fma2(mul2(y.v[k], w.v[k]), scale2, xs) : xs;
        sum = fma2(z[i].v[k], z[i].v[k], sum);
      }
    }
    copy(from);  // into what has just been read
    from += V * kPieces * pitch;
    if (++stage == a.stages) stage = 0, from = g.mine;
    if (a.x_out && live) {
      T* const to = static_cast<T*>(a.x_out) + row * a.ldo;
#pragma unroll
      for (int i = 0; i < V; ++i) at.write(to, i, z[i]);
    }
    if (!a.h) continue;
    float s[1] = {both(sum)};
    group_sums<SPAN>(s, a.group, g.id, g.thread, scratch[own][1][turn]);
    const float r2 = rsqrtf(fmaf(s[0], inv_dim, a.eps));
    if (live && g.thread == 0 && a.rstd_pre) a.rstd_pre[row] = r2;
    const F2 r22 = pair(r2, r2);
    uint16_t* const to = a.h + row * a.ldh;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const Oct w = g.weights.get(false, i);
#pragma unroll
      for (int k = 0; k < 4; ++k) z[i].v[k] = mul2(mul2(z[i].v[k], w.v[k]), r22);
      if (live) at.write_bf16(to, i, z[i]);
    }
  }
  copies_wait(1);
}

// Its gradient, dealt the same.  NORM: there is a norm behind (dh); Y: there is a block's output.
template <typename T, int NT, Span SPAN, bool NORM, bool Y>
__global__ void __launch_bounds__(NT, 1) block_norm_bwd_kernel(const NormBwdArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float scratch[kMaxBarriers][2][3][32];  // three sums of a row, rows in turn
  for (int i = threadIdx.x; i < kMaxBarriers * 192; i += blockDim.x) (&scratch[0][0][0][0])[i] = 0.0f;
  grid_dependency_wait();
  constexpr int V = kV;
  const Setup<T, SPAN> g(smem, a.group, a.dim, a.w_post, a.gate, a.w_pre, a.w_f32);
  const Layout<T>& at = g.at;
  // of x_out, dh, y, d_out
  constexpr int kP = Layout<T>::kPieces, kDh = NORM ? kP : 0, kY = kDh + (NORM ? 1 : 0);
  constexpr int kUp = kY + (Y ? 1 : 0), kPieces = kUp + kP;
  const int pitch = g.pitch, step = g.teams * g.groups;
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  g.clear(a.stages * V * kPieces);
  int64_t row = static_cast<int64_t>(g.team) * g.groups + g.id, next = row;
  auto copy = [&](uint8_t* slot) {
    if (next < a.n_rows) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        uint8_t* const to = slot + i * kPieces * pitch;
        if (NORM) {
          at.copy(to, pitch, static_cast<const T*>(a.z) + next * a.ldz, i);
          at.copy_bf16(to + kDh * pitch, a.dh + next * a.lddh, i);
        }
        if (Y) at.copy_bf16(to + kY * pitch, a.y + next * a.ldy, i);
        if (a.d_out) at.copy(to + kUp * pitch, pitch, static_cast<const T*>(a.d_out) + next * a.lddo, i);
      }
    }
    copies_commit();
    next += step;
  };
#pragma unroll 1
  for (int s = 0; s < a.stages; ++s) copy(g.mine + s * V * kPieces * pitch);
  // a row's factors, read a row ahead
  float r1 = 1.0f, r2 = 0.0f, scale = a.branch;
  auto factors = [&](int64_t of) {
    if (of >= a.n_rows) return;
    if (NORM) r2 = a.rstd_pre[of];
    if (Y && a.rstd_post) r1 = a.rstd_post[of];
    if (Y && a.row_gate) scale = a.branch * a.row_gate[of];
  };
  factors(row);
  g.ready();
  Oct sum_pre[V] = {}, sum_branch[V] = {};
  const F2 skip = pair(a.skip, a.skip);
  uint8_t* slot = g.mine;
  int stage = 0, turn = 0;
  const int own = a.group > 32 ? g.id : 0;  // smaller groups use no scratch
#pragma unroll 1
  for (; g.first_row(row) < a.n_rows; row += step, turn ^= 1) {
    const bool live = SPAN == kCta || row < a.n_rows;
    const float now_r1 = r1, now_r2 = r2, now_scale = scale;
    factors(row + step);
    copies_wait(a.stages);
    if (SPAN != kCta && !live) {  // past the last row: zeros, which add nothing to the sums over the rows
      for (int p = 0; p < V * kPieces; ++p) *reinterpret_cast<uint4*>(slot + p * pitch) = make_uint4(0, 0, 0, 0);
    }
    // e = d_out + r2 a, so that dz = e - r2 c2 v; the three sums of the row
    Oct e[V], v[V];
    F2 sum_av = 0, sum_es = 0, sum_vs = 0;
    const F2 r12 = pair(now_r1, now_r1), r22 = pair(now_r2, now_r2);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint8_t* const from = slot + i * kPieces * pitch;
      if (a.d_out) {
        e[i] = at.read(from + kUp * pitch, pitch);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) e[i].v[k] = 0;
      }
      if (NORM) {
        v[i] = at.read(from, pitch);
        const Oct dh = at.read_bf16(from + kDh * pitch), w = g.weights.get(false, i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[i].v[k] = mul2(v[i].v[k], r22);
          sum_pre[i].v[k] = fma2(dh.v[k], v[i].v[k], sum_pre[i].v[k]);
          const F2 up = mul2(dh.v[k], w.v[k]);
          sum_av = fma2(up, v[i].v[k], sum_av);
          e[i].v[k] = fma2(up, r22, e[i].v[k]);
        }
      }
      if (Y) {
        const Oct y = at.read_bf16(from + kY * pitch), w = g.weights.get(true, i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const F2 ws = mul2(mul2(y.v[k], r12), w.v[k]);
          sum_es = fma2(e[i].v[k], ws, sum_es);
          if (NORM) sum_vs = fma2(v[i].v[k], ws, sum_vs);
        }
      }
    }
    float c2 = 0.0f, c1 = 0.0f;
    if (NORM || (Y && (a.w_post || a.drow_gate))) {
      float sums[3] = {both(sum_av), both(sum_es), both(sum_vs)};
      group_sums<SPAN>(sums, a.group, g.id, g.thread, scratch[own][turn][0]);
      c2 = now_r2 * (inv_dim * sums[0]);
      c1 = fmaf(-c2, sums[2], sums[1]);  // sum of gate w_post dz s
      if (Y && live && g.thread == 0 && a.drow_gate) a.drow_gate[row] = a.branch * c1;
      c1 = Y && a.w_post ? inv_dim * c1 : 0.0f;
    }
    const F2 minus_c2 = pair(-c2, -c2), minus_c1 = pair(-c1, -c1), scale2 = pair(now_scale, now_scale);
    const F2 factor = pair(now_r1 * now_scale, now_r1 * now_scale);
    T* const to_x = a.dx ? static_cast<T*>(a.dx) + row * a.lddx : nullptr;
    uint16_t* const to_y = Y && a.dy ? a.dy + row * a.lddy : nullptr;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (NORM) {
#pragma unroll
        for (int k = 0; k < 4; ++k) e[i].v[k] = fma2(v[i].v[k], minus_c2, e[i].v[k]);  // dz
      }
      if (a.dx) {
        Oct dx;
#pragma unroll
        for (int k = 0; k < 4; ++k) dx.v[k] = mul2(e[i].v[k], skip);
        if (live) at.write(to_x, i, dx);
      }
      if (!Y) continue;
      const Oct y = at.read_bf16(slot + (i * kPieces + kY) * pitch), w = g.weights.get(true, i);
      Oct dy;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const F2 s = mul2(y.v[k], r12);
        sum_branch[i].v[k] = fma2(mul2(e[i].v[k], scale2), s, sum_branch[i].v[k]);
        dy.v[k] = mul2(fma2(s, minus_c1, mul2(e[i].v[k], w.v[k])), factor);
      }
      if (a.dy && live) at.write_bf16(to_y, i, dy);
    }
    copy(slot);  // into what has just been read
    slot += V * kPieces * pitch;
    if (++stage == a.stages) stage = 0, slot = g.mine;
  }
  copies_wait(1);
  if (!a.want_pre && !a.want_branch) return;
  // the groups of a warp, then the groups (or warps) in order through shared memory, then the CTA's to the workspace
  for (int o = a.group; SPAN == kSub && o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        sum_pre[i].v[m] = add2(sum_pre[i].v[m], __shfl_xor_sync(0xffffffffu, sum_pre[i].v[m], o));
        sum_branch[i].v[m] = add2(sum_branch[i].v[m], __shfl_xor_sync(0xffffffffu, sum_branch[i].v[m], o));
      }
  }
  const int parts = g.groups / g.rows, part_id = g.id / g.rows;
  const bool writes = g.id % g.rows == 0;
  float* const sums = reinterpret_cast<float*>(g.ring);
  float* const part = a.part + static_cast<int64_t>(g.team) * 2 * a.dim;
  for (int k = 0; k < parts; ++k) {
    __syncthreads();  // also: every thread is through with the ring
    if (part_id != k || !writes) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (k > 0) {
        const Oct p = at.read_f32(sums, i), q = at.read_f32(sums + a.dim, i);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          sum_pre[i].v[m] = add2(sum_pre[i].v[m], p.v[m]);
          sum_branch[i].v[m] = add2(sum_branch[i].v[m], q.v[m]);
        }
      }
      float* const to = k + 1 < parts ? sums : part;
      if (NORM) at.write_f32(to, i, sum_pre[i]);
      if (Y) at.write_f32(to + a.dim, i, sum_branch[i]);
    }
  }
}

struct NormSumArgs {
  const float* part;
  int parts, dim;
  const void *w_post, *gate;
  bool w_f32;
  float *dw_pre, *dw_post, *dgate;
};

// The CTAs' sums of 32 columns: a lane a column, 32 warps with 5 CTAs each (all their
// loads at once: this kernel is one latency), joined in order.
constexpr int kRun = kMaxParts / 32;
__global__ void __launch_bounds__(1024) block_norm_sum_kernel(const NormSumArgs a) {
  __shared__ float s[2][32][32];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const bool want_branch = a.dw_post || a.dgate;
  float pre[kRun], branch[kRun];
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    const int p = run * kRun + k;
    const bool there = c < a.dim && p < a.parts;
    const float* const at = a.part + static_cast<int64_t>(p) * 2 * a.dim + c;
    pre[k] = there && a.dw_pre ? at[0] : 0.0f;
    branch[k] = there && want_branch ? at[a.dim] : 0.0f;
  }
#pragma unroll
  for (int k = 1; k < kRun; ++k) pre[0] += pre[k], branch[0] += branch[k];
  s[0][run][lane] = pre[0], s[1][run][lane] = branch[0];
  __syncthreads();
  if (run > 0 || c >= a.dim) return;
  for (int r = 1; r < 32; ++r) pre[0] += s[0][r][lane], branch[0] += s[1][r][lane];
  if (a.dw_pre) a.dw_pre[c] = pre[0];
  if (a.dw_post) a.dw_post[c] = a.gate ? branch[0] * weight1(a.gate, a.w_f32, c) : branch[0];
  if (a.dgate) a.dgate[c] = a.w_post ? branch[0] * weight1(a.w_post, a.w_f32, c) : branch[0];
}

// How a call's rows are dealt: threads of a row, rows and CTAs of a cluster, clusters, and rows on the way.
struct Deal {
  int group, groups, ctas, grid, stages, smem;
};
Deal deal(int64_t n_rows, int dim, int threads, int pieces, bool sums) {
  Deal d;
  const int need = (dim + 8 * kV - 1) / (8 * kV);
  d.ctas = dim > kWide ? 2 : 1;
  d.group = need > 32 ? (need + 32 * d.ctas - 1) / (32 * d.ctas) * (32 * d.ctas) : 1;
  while (d.group < need) d.group *= 2;  // within a warp: a power of two
  const int teams = sm_count() / d.ctas, here = std::max(1, d.group / d.ctas);
  // few rows are spread over the SMs, one to a CTA (or a warp's)
  d.groups = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(threads / here, (n_rows + teams - 1) / teams)));
  if (d.group < 32) d.groups = (d.groups + 32 / d.group - 1) / (32 / d.group) * (32 / d.group);
  if (d.group > 32) d.groups = std::min(d.groups, kMaxBarriers);
  d.grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({(n_rows + d.groups - 1) / d.groups, teams, kMaxParts})));
  const int row = d.groups * here * kV * pieces * 16, weights = 2 * kV * 2 * 16 * here;
  d.stages = std::max(1, std::min(kMaxStages, (kSharedBytes - weights) / row));
  // the groups' sums over the rows meet where the rows were
  d.smem = weights + std::max(d.stages * row, sums && d.groups > 1 ? 2 * dim * 4 : 0);
  return d;
}

template <typename Args>
int launch(void (*kernel)(Args), const Deal& d, const Args& a, int id, cudaStream_t s) {
  KV_TRY(set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), kSharedBytes));
  LaunchScope scope(id, s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(d.grid * d.ctas);
  cfg.blockDim = dim3(d.groups * d.group / d.ctas);
  cfg.dynamicSmemBytes = d.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = d.ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = d.ctas == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

template <typename T, int NT, Span SPAN>
auto fwd_kernel(const NormArgs& a) {
  return a.y ? block_norm_kernel<T, NT, SPAN, true> : block_norm_kernel<T, NT, SPAN, false>;
}

template <typename T>
int launch_norm(NormArgs a, cudaStream_t s) {
  const Deal d = deal(a.n_rows, a.dim, kThreads, Layout<T>::kPieces + (a.y ? 1 : 0), false);
  a.group = d.group, a.stages = d.stages;
  return launch(d.ctas == 2 ? fwd_kernel<T, kThreads, kPair>(a)
                : d.group < 32 ? fwd_kernel<T, kThreads, kSub>(a) : fwd_kernel<T, kThreads, kCta>(a),
                d, a, TWELL_KERNEL_BLOCK_NORM, s);
}

template <typename T, int NT, Span SPAN>
auto bwd_kernel(const NormBwdArgs& a) {
  if (a.dh) return a.y ? block_norm_bwd_kernel<T, NT, SPAN, true, true> : block_norm_bwd_kernel<T, NT, SPAN, true, false>;
  return a.y ? block_norm_bwd_kernel<T, NT, SPAN, false, true> : block_norm_bwd_kernel<T, NT, SPAN, false, false>;
}

template <typename T>
int launch_norm_bwd(NormBwdArgs a, int* parts, cudaStream_t s) {
  const Deal d = deal(a.n_rows, a.dim, kBwdThreads,
                      Layout<T>::kPieces * (a.dh ? 2 : 1) + (a.dh ? 1 : 0) + (a.y ? 1 : 0), true);
  a.group = d.group, a.stages = d.stages, *parts = d.grid;
  return launch(d.ctas == 2 ? bwd_kernel<T, kBwdThreads, kPair>(a)
                : d.group < 32 ? bwd_kernel<T, kBwdThreads, kSub>(a) : bwd_kernel<T, kBwdThreads, kCta>(a),
                d, a, TWELL_KERNEL_BLOCK_NORM_BWD, s);
}

bool finite(float x) { return x - x == 0.0f; }

// A row matrix that must be there (or may be null), ld elements between rows.
int check_matrix(const void* p, int64_t ld, int dim, bool needed) {
  if (!p) return needed ? TWELL_ERR_INVALID_ARG : TWELL_OK;
  if (!aligned_to(p, 16)) return TWELL_ERR_MISALIGNED;
  return ld >= dim && ld % 8 == 0 ? TWELL_OK : TWELL_ERR_INVALID_ARG;
}

// No output lies where an input or another output does (null: none).
bool apart(std::initializer_list<const void*> outputs, std::initializer_list<const void*> inputs) {
  for (const void* const* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const void* const* p = outputs.begin(); p != o; ++p)
      if (*o && *o == *p) return false;
    for (const void* p : inputs)
      if (*o && *o == p) return false;
  }
  return true;
}

int check_sizes(int n_rows, int dim, int dtype, int w_dtype) {
  if (n_rows < 0 || dim < 1) return TWELL_ERR_INVALID_ARG;
  if (dtype != TWELL_BF16 && dtype != TWELL_F32) return TWELL_ERR_INVALID_ARG;
  if (w_dtype != TWELL_BF16 && w_dtype != TWELL_F32) return TWELL_ERR_INVALID_ARG;
  return dim % 8 == 0 && dim <= kMaxDim ? TWELL_OK : TWELL_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace twell

using namespace twell;

extern "C" TWELL_API int twell_block_norm(const void* x, int32_t dtype, int64_t ldx, const uint16_t* y, int64_t ldy,
                                          int32_t n_rows, int32_t d_model, const void* w_post, const void* gate,
                                          const void* w_pre, int32_t w_dtype, const float* row_gate, float skip_scale,
                                          float branch_scale, float eps, void* x_out, int64_t ldo, uint16_t* h,
                                          int64_t ldh, float* rstd_post, float* rstd_pre, twell_stream_t stream) {
  KV_TRY(check_sizes(n_rows, d_model, dtype, w_dtype));
  if (!finite(skip_scale) || !finite(branch_scale) || !finite(eps) || !(eps > 0.0f)) return TWELL_ERR_INVALID_ARG;
  if (n_rows > 0) {  // matrices of no rows may be null
    if (!y && (w_post || gate || row_gate)) return TWELL_ERR_INVALID_ARG;
    if (!h != !w_pre || (rstd_post && !w_post) || (rstd_pre && !w_pre)) return TWELL_ERR_INVALID_ARG;
    if (!x_out && !h) return TWELL_ERR_INVALID_ARG;
    KV_TRY(check_matrix(x, ldx, d_model, true));
    KV_TRY(check_matrix(y, ldy, d_model, false));
    KV_TRY(check_matrix(x_out, ldo, d_model, false));
    KV_TRY(check_matrix(h, ldh, d_model, false));
    if (x_out == x && ldo != ldx) return TWELL_ERR_INVALID_ARG;
    if (!apart({x_out, h}, {y}) || h == x) return TWELL_ERR_INVALID_ARG;
    for (const void* p : {w_post, gate, w_pre})
      if (!aligned_to(p, 16)) return TWELL_ERR_MISALIGNED;
    for (const float* p : {row_gate, static_cast<const float*>(rstd_post), static_cast<const float*>(rstd_pre)})
      if (!aligned_to(p, 4)) return TWELL_ERR_MISALIGNED;
  }
  if (!device_is_sm103()) return TWELL_ERR_NO_DEVICE;
  if (n_rows == 0) return TWELL_OK;
  const NormArgs a{x,    y,      x_out, h,     ldx,  ldy,    ldo,   ldh, n_rows,    d_model, 0, 0, w_post,
                   gate, w_pre,  w_dtype == TWELL_F32, row_gate, skip_scale, branch_scale, eps, rstd_post, rstd_pre};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == TWELL_BF16 ? launch_norm<uint16_t>(a, s) : launch_norm<float>(a, s);
}

extern "C" TWELL_API size_t twell_block_norm_bwd_workspace_bytes(int32_t n_rows, int32_t d_model) {
  if (n_rows < 0 || d_model < 8 || d_model % 8 != 0 || d_model > kMaxDim) return 0;
  return static_cast<size_t>(kMaxParts) * 2 * d_model * sizeof(float);
}

extern "C" TWELL_API int twell_block_norm_bwd(const uint16_t* dh, int64_t lddh, const void* d_out, int32_t dtype,
                                              int64_t lddo, const void* x_out, int64_t ldo, const uint16_t* y,
                                              int64_t ldy, int32_t n_rows, int32_t d_model, const void* w_post,
                                              const void* gate, const void* w_pre, int32_t w_dtype,
                                              const float* row_gate, float skip_scale, float branch_scale,
                                              const float* rstd_post, const float* rstd_pre, void* dx, int64_t lddx,
                                              uint16_t* dy, int64_t lddy, float* dw_post, float* dgate, float* dw_pre,
                                              float* drow_gate, void* workspace, size_t workspace_bytes,
                                              twell_stream_t stream) {
  KV_TRY(check_sizes(n_rows, d_model, dtype, w_dtype));
  if (!finite(skip_scale) || !finite(branch_scale)) return TWELL_ERR_INVALID_ARG;
  if ((dw_post && !w_post) || (dgate && !gate) || (dw_pre && !w_pre)) return TWELL_ERR_INVALID_ARG;
  for (const void* p : {w_post, gate, w_pre})
    if (!aligned_to(p, 16)) return TWELL_ERR_MISALIGNED;
  for (const float* p : {row_gate, rstd_post, rstd_pre, static_cast<const float*>(dw_post),
                         static_cast<const float*>(dgate), static_cast<const float*>(dw_pre),
                         static_cast<const float*>(drow_gate)})
    if (!aligned_to(p, 4)) return TWELL_ERR_MISALIGNED;
  if (n_rows > 0) {
    if (!y && (w_post || gate || row_gate || dy)) return TWELL_ERR_INVALID_ARG;
    if (!dh != !w_pre || !dh != !rstd_pre || !w_post != !rstd_post) return TWELL_ERR_INVALID_ARG;
    if (drow_gate && !row_gate) return TWELL_ERR_INVALID_ARG;
    if (!dh && !d_out) return TWELL_ERR_INVALID_ARG;
    KV_TRY(check_matrix(dh, lddh, d_model, false));
    KV_TRY(check_matrix(d_out, lddo, d_model, false));
    KV_TRY(check_matrix(x_out, ldo, d_model, dh != nullptr));
    KV_TRY(check_matrix(y, ldy, d_model, false));
    KV_TRY(check_matrix(dx, lddx, d_model, false));
    KV_TRY(check_matrix(dy, lddy, d_model, false));
    if (dx && dx == d_out && lddx != lddo) return TWELL_ERR_INVALID_ARG;
    if (!apart({dx, dy}, {dh, x_out, y}) || (dy && dy == d_out)) return TWELL_ERR_INVALID_ARG;
  }
  const bool sums = dw_post || dgate || dw_pre;
  if (sums) {
    if (!workspace || workspace_bytes < twell_block_norm_bwd_workspace_bytes(n_rows, d_model))
      return TWELL_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return TWELL_ERR_MISALIGNED;
  }
  if (!device_is_sm103()) return TWELL_ERR_NO_DEVICE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int parts = 0;
  if (n_rows > 0) {
    const NormBwdArgs a{dh,     d_out,   x_out, y,      dx,   dy,    lddh,  lddo,
                        ldo,    ldy,     lddx,  lddy,   n_rows, d_model, 0, 0, w_post, gate, w_pre,
                        w_dtype == TWELL_F32, row_gate, skip_scale, branch_scale, rstd_post, rstd_pre,
                        drow_gate, dw_pre != nullptr, dw_post || dgate, static_cast<float*>(workspace)};
    KV_TRY(dtype == TWELL_BF16 ? launch_norm_bwd<uint16_t>(a, &parts, s) : launch_norm_bwd<float>(a, &parts, s));
  }
  if (!sums) return TWELL_OK;
  const NormSumArgs a{static_cast<const float*>(workspace), parts, d_model, w_post, gate, w_dtype == TWELL_F32,
                      dw_pre, dw_post, dgate};
  LaunchScope scope(TWELL_KERNEL_BLOCK_NORM_BWD, s);
  return launch_pdl(block_norm_sum_kernel, dim3((d_model + 31) / 32), dim3(1024), 0, s, a) == cudaSuccess
             ? TWELL_OK
             : TWELL_ERR_CUDA;
}
