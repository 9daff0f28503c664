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
// A row is held in registers by a group of threads, 8 elements a 16-byte load,
// and is read once.  All sums are fp32: a thread's own elements in order, then
// a tree over the group, so results do not depend on the launch.
#include <algorithm>

#include "kv_internal.h"

namespace twell {
namespace {

constexpr int kMaxDim = 16384;
constexpr int kMaxParts = 1024;  // partial sums of the weights' gradients

struct NormArgs {
  const void* x;
  const uint16_t* y;
  void* x_out;
  uint16_t* h;
  int64_t ldx, ldy, ldo, ldh;
  int n_rows, dim, group;  // group: threads of a row
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
  int n_rows, dim, group;
  const void *w_post, *gate, *w_pre;
  bool w_f32;
  const float* row_gate;
  float skip, branch;
  const float *rstd_post, *rstd_pre;
  float* drow_gate;
  bool want_pre, want_branch;  // sums over the rows that are asked for
  float* part;                 // [parts][2][dim]: sum dh v, then P
};

// 8 elements of a row at p + 8 i.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]);
template <>
__device__ __forceinline__ void load8<uint16_t>(const uint16_t* p, float (&f)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
  f[4] = bf16_lo(w.z), f[5] = bf16_hi(w.z), f[6] = bf16_lo(w.w), f[7] = bf16_hi(w.w);
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void weight8(const void* p, bool f32, int at, float (&f)[8]) {
  if (f32)
    load8(static_cast<const float*>(p) + at, f);
  else
    load8(static_cast<const uint16_t*>(p) + at, f);
}

// The sum over the group's threads, in every thread of it.  scratch: 32 floats of
// the group's own, free again once the group has passed another such barrier.
__device__ __forceinline__ float group_sum(float v, int group, int id, int thread, float* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (group == 32) return v;
  const int lane = thread & 31;
  if (lane == 0) scratch[thread >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(group) : "memory");
  v = lane < (group >> 5) ? scratch[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int kMaxGroups = 8;  // rows of a CTA at a time (named barriers 1 to 8)

template <typename T, int V>
__global__ void __launch_bounds__(1024) block_norm_kernel(const NormArgs a) {
  __shared__ float scratch[kMaxGroups][2][32];
  grid_dependency_wait();
  const int id = threadIdx.x / a.group, t = threadIdx.x % a.group;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / a.group) + id;
  if (row >= a.n_rows) return;  // whole groups leave: barriers are a group's own
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  float z[V][8];
  float scale = a.branch;
  if (a.row_gate) scale *= a.row_gate[row];
  if (a.y) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (t + i * a.group) * 8;
      if (c < a.dim) {
        load8(a.y + row * a.ldy + c, z[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(z[i][e], z[i][e], s);
      }
    }
    if (a.w_post) {
      s = group_sum(s, a.group, id, t, scratch[id][0]);
      const float r1 = 1.0f / sqrtf(fmaf(s, inv_dim, a.eps));
      if (t == 0 && a.rstd_post) a.rstd_post[row] = r1;
      scale *= r1;
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (t + i * a.group) * 8;
    if (c >= a.dim) continue;
    float x[8];
    load8(static_cast<const T*>(a.x) + row * a.ldx + c, x);
    if (a.y) {
      float w[8];
      if (a.w_post) {
        weight8(a.w_post, a.w_f32, c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[i][e] *= w[e];
      }
      if (a.gate) {
        weight8(a.gate, a.w_f32, c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[i][e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i][e] = fmaf(scale, z[i][e], a.skip * x[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i][e] = a.skip * x[e];
    }
    if (a.x_out) store8(static_cast<T*>(a.x_out) + row * a.ldo + c, z[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(z[i][e], z[i][e], s);
  }
  if (!a.h) return;
  s = group_sum(s, a.group, id, t, scratch[id][1]);
  const float r2 = 1.0f / sqrtf(fmaf(s, inv_dim, a.eps));
  if (t == 0 && a.rstd_pre) a.rstd_pre[row] = r2;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (t + i * a.group) * 8;
    if (c >= a.dim) continue;
    float w[8];
    weight8(a.w_pre, a.w_f32, c, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[i][e] *= r2 * w[e];
    store8(a.h + row * a.ldh + c, z[i]);
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(1024) block_norm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float scratch[kMaxGroups][2][2][32];  // two sums of a row, rows in turn
  grid_dependency_wait();
  const int id = threadIdx.x / a.group, t = threadIdx.x % a.group, groups = blockDim.x / a.group;
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  float sum_pre[V][8] = {}, sum_branch[V][8] = {};
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * groups + id; row < a.n_rows;
       row += static_cast<int64_t>(gridDim.x) * groups, turn ^= 1) {
    float dz[V][8], v[V][8];
    float r2 = 0.0f, c2 = 0.0f;
    if (a.dh) {
      r2 = a.rstd_pre[row];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (t + i * a.group) * 8;
        if (c >= a.dim) continue;
        float w[8];
        load8(a.dh + row * a.lddh + c, dz[i]);
        load8(static_cast<const T*>(a.z) + row * a.ldz + c, v[i]);
        weight8(a.w_pre, a.w_f32, c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[i][e] *= r2;
          sum_pre[i][e] = fmaf(dz[i][e], v[i][e], sum_pre[i][e]);
          dz[i][e] *= w[e];
          c2 = fmaf(dz[i][e], v[i][e], c2);
        }
      }
      c2 = group_sum(c2, a.group, id, t, scratch[id][0][turn]) * inv_dim;
    }
    const float scale = a.row_gate ? a.branch * a.row_gate[row] : a.branch;
    const float r1 = a.rstd_post ? a.rstd_post[row] : 1.0f;
    float c1 = 0.0f;  // sum t s / scale
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (t + i * a.group) * 8;
      if (c >= a.dim) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) dz[i][e] = a.dh ? r2 * (dz[i][e] - v[i][e] * c2) : 0.0f;
      float w[8];
      if (a.d_out) {
        load8(static_cast<const T*>(a.d_out) + row * a.lddo + c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) dz[i][e] += w[e];
      }
      if (a.dx) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = a.skip * dz[i][e];
        store8(static_cast<T*>(a.dx) + row * a.lddx + c, w);
      }
      if (!a.y) continue;
      load8(a.y + row * a.ldy + c, v[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i][e] *= r1;
        sum_branch[i][e] = fmaf(scale * dz[i][e], v[i][e], sum_branch[i][e]);
      }
      if (a.w_post) {
        weight8(a.w_post, a.w_f32, c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) dz[i][e] *= w[e];
      }
      if (a.gate) {
        weight8(a.gate, a.w_f32, c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) dz[i][e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) c1 = fmaf(dz[i][e], v[i][e], c1);
    }
    if (!a.y) continue;
    if (a.w_post || a.drow_gate) {
      c1 = group_sum(c1, a.group, id, t, scratch[id][1][turn]);
      if (t == 0 && a.drow_gate) a.drow_gate[row] = a.branch * c1;
    }
    c1 = a.w_post ? c1 * inv_dim : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (t + i * a.group) * 8;
      if (c >= a.dim) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) dz[i][e] = scale * (r1 * (dz[i][e] - v[i][e] * c1));
      if (a.dy) store8(a.dy + row * a.lddy + c, dz[i]);
    }
  }
  float* const part = a.part + static_cast<int64_t>(blockIdx.x * groups + id) * 2 * a.dim;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (t + i * a.group) * 8;
    if (c >= a.dim) continue;
    if (a.want_pre) store8(part + c, sum_pre[i]);
    if (a.want_branch) store8(part + a.dim + c, sum_branch[i]);
  }
}

struct NormSumArgs {
  const float* part;
  int parts, dim;
  const void *w_post, *gate;
  bool w_f32;
  float *dw_pre, *dw_post, *dgate;
};

__device__ __forceinline__ float weight1(const void* p, bool f32, int c) {
  return f32 ? static_cast<const float*>(p)[c] : bf16_bits_to_float(static_cast<const uint16_t*>(p)[c]);
}

// The partial sums of 32 columns in order: 32 threads of columns by 8 runs of parts.
__global__ void __launch_bounds__(256) block_norm_sum_kernel(const NormSumArgs a) {
  __shared__ float s[2][8][32];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float pre = 0.0f, branch = 0.0f;
  if (c < a.dim)
    for (int p = run * a.parts / 8; p < (run + 1) * a.parts / 8; ++p) {
      const float* const at = a.part + static_cast<int64_t>(p) * 2 * a.dim + c;
      if (a.dw_pre) pre += at[0];
      if (a.dw_post || a.dgate) branch += at[a.dim];
    }
  s[0][run][lane] = pre, s[1][run][lane] = branch;
  __syncthreads();
  if (run > 0 || c >= a.dim) return;
  for (int r = 1; r < 8; ++r) pre += s[0][r][lane], branch += s[1][r][lane];
  if (a.dw_pre) a.dw_pre[c] = pre;
  if (a.dw_post) a.dw_post[c] = a.gate ? branch * weight1(a.gate, a.w_f32, c) : branch;
  if (a.dgate) a.dgate[c] = a.w_post ? branch * weight1(a.w_post, a.w_f32, c) : branch;
}

// Threads of a row: 8 V elements a thread, whole warps.
int group_of(int dim, int v) { return ((dim + 8 * v - 1) / (8 * v) + 31) / 32 * 32; }
int groups_of(int group) { return std::max(1, std::min(kMaxGroups, 256 / group)); }

int bwd_parts(int n_rows, int dim) {
  const int groups = groups_of(group_of(dim, 2));
  return std::max(1, std::min({(n_rows + groups - 1) / groups, 2 * sm_count(), kMaxParts / groups})) * groups;
}

template <typename T>
int launch_norm(NormArgs a, cudaStream_t s) {
  a.group = group_of(a.dim, 2);
  const int groups = groups_of(a.group);
  LaunchScope scope(TWELL_KERNEL_BLOCK_NORM, s);
  return launch_pdl(block_norm_kernel<T, 2>, dim3((a.n_rows + groups - 1) / groups), dim3(groups * a.group), 0, s,
                    a) == cudaSuccess
             ? TWELL_OK
             : TWELL_ERR_CUDA;
}

template <typename T>
int launch_norm_bwd(NormBwdArgs a, int parts, cudaStream_t s) {
  a.group = group_of(a.dim, 2);
  const int groups = groups_of(a.group);
  LaunchScope scope(TWELL_KERNEL_BLOCK_NORM_BWD, s);
  return launch_pdl(block_norm_bwd_kernel<T, 2>, dim3(parts / groups), dim3(groups * a.group), 0, s, a) == cudaSuccess
             ? TWELL_OK
             : TWELL_ERR_CUDA;
}

bool finite(float x) { return x - x == 0.0f; }

// A row matrix that must be there (or may be null), ld elements between rows.
int check_matrix(const void* p, int64_t ld, int dim, bool needed) {
  if (!p) return needed ? TWELL_ERR_INVALID_ARG : TWELL_OK;
  if (!aligned_to(p, 16)) return TWELL_ERR_MISALIGNED;
  return ld >= dim && ld % 8 == 0 ? TWELL_OK : TWELL_ERR_INVALID_ARG;
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
    for (const void* p : {w_post, gate, w_pre})
      if (!aligned_to(p, 16)) return TWELL_ERR_MISALIGNED;
    for (const float* p : {row_gate, static_cast<const float*>(rstd_post), static_cast<const float*>(rstd_pre)})
      if (!aligned_to(p, 4)) return TWELL_ERR_MISALIGNED;
  }
  if (!device_is_sm103()) return TWELL_ERR_NO_DEVICE;
  if (n_rows == 0) return TWELL_OK;
  const NormArgs a{x,    y,      x_out, h,     ldx,  ldy,    ldo,   ldh, n_rows,    d_model, 0, w_post,
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
  }
  const bool sums = dw_post || dgate || dw_pre;
  if (sums) {
    if (!workspace || workspace_bytes < twell_block_norm_bwd_workspace_bytes(n_rows, d_model))
      return TWELL_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return TWELL_ERR_MISALIGNED;
  }
  if (!device_is_sm103()) return TWELL_ERR_NO_DEVICE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int parts = n_rows > 0 ? bwd_parts(n_rows, d_model) : 0;
  if (n_rows > 0) {
    const NormBwdArgs a{dh,     d_out,   x_out, y,      dx,   dy,    lddh,  lddo,
                        ldo,    ldy,     lddx,  lddy,   n_rows, d_model, 0, w_post, gate, w_pre,
                        w_dtype == TWELL_F32, row_gate, skip_scale, branch_scale, rstd_post, rstd_pre,
                        drow_gate, dw_pre != nullptr, dw_post || dgate, static_cast<float*>(workspace)};
    KV_TRY(dtype == TWELL_BF16 ? launch_norm_bwd<uint16_t>(a, parts, s) : launch_norm_bwd<float>(a, parts, s));
  }
  if (!sums) return TWELL_OK;
  const NormSumArgs a{static_cast<const float*>(workspace), parts, d_model, w_post, gate, w_dtype == TWELL_F32,
                      dw_pre, dw_post, dgate};
  LaunchScope scope(TWELL_KERNEL_BLOCK_NORM_BWD, s);
  return launch_pdl(block_norm_sum_kernel, dim3((d_model + 31) / 32), dim3(256), 0, s, a) == cudaSuccess
             ? TWELL_OK
             : TWELL_ERR_CUDA;
}
