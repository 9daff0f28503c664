// Block tables and slot maps of a decode step (twell_kv_plan).
//
// With l_r the old and n_r the new tokens of request r and P the page size,
//   have_r = ceil(l_r / P),  need_r = ceil((l_r + n_r) / P) - have_r,
//   a_r = sum of need over the requests before r,
// the j-th new page of r is ring[(head + a_r + j) mod n_pages].  Everything is
// a prefix sum over the requests followed by independent writes, a few
// kilobytes: the launch and three dependent memory latencies bound it, not
// bytes.  So there is one launch and no exchange between CTAs: every CTA sums
// over all requests itself (a few loads a thread, from L2) into shared memory and
// then serves its own share of the tokens by binary search there.  A token
// whose page is new takes it from the ring, not from the block table that the
// same launch is writing.
// 16 requests: 3.6 us; 1000 requests with prompts among them 6.5; 4000 of them 17.
#include "kv_internal.h"

namespace twell {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxRequests = 16384;

struct PlanArgs {
  const int32_t* kv_lens;
  const int32_t* new_tokens;
  int n_requests, page_shift, n_pages, max_blocks;
  int32_t* block_table;
  int32_t* ring;
  const int32_t* pool;
  int32_t* pool_out;
  int32_t* kv_lens_out;
  int32_t* cu_q;
  int64_t* slots;
  int32_t* positions;
  int n_tokens;
  int32_t* status;
};

struct Sums {
  int64_t tokens, need, back;
};

__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.tokens + b.tokens, a.need + b.need, a.back + b.back};
}

__device__ __forceinline__ Sums shfl_up(const Sums& a, int d) {
  return {__shfl_up_sync(0xffffffffu, a.tokens, d), __shfl_up_sync(0xffffffffu, a.need, d),
          __shfl_up_sync(0xffffffffu, a.back, d)};
}

__device__ __forceinline__ int blocks_of(int64_t tokens, int page_shift) {
  return static_cast<int>((tokens + (1 << page_shift) - 1) >> page_shift);
}

// i mod n for 0 <= i < 2 n, without a division.
__device__ __forceinline__ int wrap(int64_t i, int n) {
  if (i >= n) i -= n;
  return static_cast<int>(i);
}

// What one request asks for.  One that wants more blocks than its table has
// is refused whatever is free, so it asks for no pages.  Of the others, once
// the running sum passes the free pages (or the tokens' capacity) every later
// one with a need is refused too: the accepted ones' pages are one run.
__device__ __forceinline__ Sums asks(const PlanArgs& a, int len, int add) {
  const int have = blocks_of(len, a.page_shift);
  if (add < 0) return {0, 0, min(have, a.max_blocks)};
  const int upto = blocks_of(static_cast<int64_t>(len) + add, a.page_shift);
  return {add, upto > a.max_blocks ? 0 : upto - have, 0};
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  // cu[r]: first token, base[r]: first new page (>= 0), or -1 refused, or
  // -2 - f finished with f pages given back before its own
  extern __shared__ int32_t dyn[];
  int32_t* const cu = dyn;
  int32_t* const base = dyn + a.n_requests + 1;
  __shared__ Sums warp_sum[kPlanThreads / 32];
  __shared__ int taken_all, refused_any;
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = a.n_requests, cap = a.n_tokens;
  const bool first_cta = blockIdx.x == 0;
  // whatever the pool words hold, ring indexes stay inside the ring
  const int head = static_cast<int>(static_cast<uint32_t>(a.pool[0]) % static_cast<uint32_t>(a.n_pages));
  const int free_pages = min(max(a.pool[1], 0), a.n_pages);
  if (tid == 0) taken_all = refused_any = 0;
  // each thread sums a run of requests, then the CTA scans the runs' sums
  const int per = (R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  Sums mine = {0, 0, 0};
  for (int r = r0; r < r1; ++r) mine = mine + asks(a, max(a.kv_lens[r], 0), a.new_tokens[r]);
  Sums inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const Sums o = shfl_up(inc, d);
    if (lane >= d) inc = inc + o;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  Sums run = {inc.tokens - mine.tokens, inc.need - mine.need, inc.back - mine.back};
  Sums all = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) run = run + warp_sum[w];
    all = all + warp_sum[w];
  }
  int taken = 0, refused = 0;
  for (int r = r0; r < r1; ++r) {
    const int len = max(a.kv_lens[r], 0), add = a.new_tokens[r];
    const Sums s = asks(a, len, add), upto = run + s;
    const bool no = add > 0 && ((s.need > 0 && upto.need > free_pages) ||
                                blocks_of(static_cast<int64_t>(len) + add, a.page_shift) > a.max_blocks ||
                                upto.tokens > cap);
    cu[r] = static_cast<int32_t>(min(run.tokens, static_cast<int64_t>(cap)));
    base[r] = add < 0 ? -2 - static_cast<int>(run.back) : no ? -1 : static_cast<int>(run.need);
    if (!no && s.need > 0) taken = static_cast<int>(upto.need);
    refused |= no;
    if (first_cta) {
      a.cu_q[r] = cu[r];
      a.kv_lens_out[r] = add < 0 ? 0 : no ? len : len + add;
    }
    run = upto;
  }
  if (tid == 0) cu[R] = static_cast<int32_t>(min(all.tokens, static_cast<int64_t>(cap)));
  if (first_cta) {
    atomicMax(&taken_all, taken);
    if (refused) refused_any = 1;
  }
  __syncthreads();
  if (first_cta && tid == 0) {
    a.cu_q[R] = cu[R];
    a.pool_out[0] = wrap(static_cast<int64_t>(head) + taken_all, a.n_pages);
    a.pool_out[1] = free_pages - taken_all + static_cast<int32_t>(all.back);
    *a.status = refused_any ? TWELL_ERR_CACHE_FULL : TWELL_OK;
  }
  // slots and positions; the token at a new page's first place (or a request's
  // first token) enters the page in the block table
  for (int t = blockIdx.x * kPlanThreads + tid; t < cap; t += gridDim.x * kPlanThreads) {
    int64_t slot = -1;
    int32_t pos = -1;
    if (t < cu[R]) {
      int lo = 0, hi = R - 1;  // the last request with cu <= t (those behind it start later)
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (cu[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      if (base[lo] >= 0) {
        const int len = max(a.kv_lens[lo], 0), have = blocks_of(len, a.page_shift);
        pos = len + (t - cu[lo]);
        const int block = pos >> a.page_shift, in = pos & ((1 << a.page_shift) - 1);
        int32_t* const entry = a.block_table + static_cast<int64_t>(lo) * a.max_blocks + block;
        int page;
        if (block < have) {
          page = *entry;
        } else {
          page = a.ring[wrap(static_cast<int64_t>(head) + base[lo] + (block - have), a.n_pages)];
          if (in == 0) *entry = page;
        }
        slot = static_cast<int64_t>(page) * (1 << a.page_shift) + in;
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
  // pages of finished requests, a CTA per request
  for (int r = blockIdx.x; r < R; r += gridDim.x) {
    if (base[r] > -2) continue;
    const int back = min(blocks_of(max(a.kv_lens[r], 0), a.page_shift), a.max_blocks);
    const int64_t to = static_cast<int64_t>(head) + free_pages + (-2 - base[r]);
    for (int j = tid; j < back; j += kPlanThreads)
      a.ring[(to + j) % a.n_pages] = a.block_table[static_cast<int64_t>(r) * a.max_blocks + j];
  }
}

}  // namespace
}  // namespace twell

using namespace twell;

extern "C" TWELL_API int twell_kv_plan(const int32_t* kv_lens, const int32_t* new_tokens, int32_t n_requests,
                                       int32_t page_size, int32_t n_pages, int32_t max_blocks, int32_t* block_table,
                                       int32_t* ring, const int32_t* pool, int32_t* pool_out, int32_t* kv_lens_out,
                                       int32_t* cu_q, int64_t* slots, int32_t* positions, int32_t n_tokens,
                                       int32_t* status, twell_stream_t stream) {
  if (n_requests < 0 || n_pages < 1 || max_blocks < 0 || n_tokens < 0) return TWELL_ERR_INVALID_ARG;
  if (!valid_page_size(page_size) || n_requests > kPlanMaxRequests) return TWELL_ERR_UNSUPPORTED;
  if (n_requests > 0) {
    KV_TRY(check_array(kv_lens, 4));
    KV_TRY(check_array(new_tokens, 4));
    KV_TRY(check_array(kv_lens_out, 4));
    if (max_blocks > 0) KV_TRY(check_array(block_table, 4));
    if (kv_lens == kv_lens_out) return TWELL_ERR_INVALID_ARG;
  }
  KV_TRY(check_array(ring, 4));
  KV_TRY(check_array(pool, 4));
  KV_TRY(check_array(pool_out, 4));
  KV_TRY(check_array(cu_q, 4));
  KV_TRY(check_array(status, 4));
  if (pool == pool_out) return TWELL_ERR_INVALID_ARG;
  if (n_tokens > 0) {
    KV_TRY(check_array(slots, 8));
    KV_TRY(check_array(positions, 4));
  }
  if (!device_is_sm103()) return TWELL_ERR_NO_DEVICE;
  const PlanArgs a{kv_lens, new_tokens, n_requests, __builtin_ctz(page_size), n_pages, max_blocks, block_table, ring, pool,
                   pool_out, kv_lens_out, cu_q, slots, positions, n_tokens, status};
  const size_t smem = sizeof(int32_t) * (2 * static_cast<size_t>(n_requests) + 1);
  KV_TRY(set_max_dynamic_smem(reinterpret_cast<const void*>(plan_kernel),
                              sizeof(int32_t) * (2 * kPlanMaxRequests + 1)));
  // every CTA repeats the sums, so no more CTAs than one wave
  // (finished requests take a CTA each in turn, so some for those too)
  const int tokens = (n_tokens + kPlanThreads - 1) / kPlanThreads, requests = (n_requests + 15) / 16;
  const int want = tokens > requests ? tokens : requests;
  const int grid = want < 1 ? 1 : want < 2 * sm_count() ? want : 2 * sm_count();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  LaunchScope scope(TWELL_KERNEL_KV_PLAN, s);
  return launch_pdl(plan_kernel, dim3(grid), dim3(kPlanThreads), smem, s, a) == cudaSuccess ? TWELL_OK
                                                                                           : TWELL_ERR_CUDA;
}
