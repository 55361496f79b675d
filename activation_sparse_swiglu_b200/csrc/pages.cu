// Block tables, slots and positions from request lengths: what a batch's
// scheduler would otherwise read back to the host every step.
//
// With have_i = ceil(len_i / page) and need_i = ceil((len_i + delta_i) / page):
// rows that shrink push their table entries [need_i, have_i) onto the free
// list, in request order; rows that grow take entries off its end, in request
// order; token n of the step belongs to the request whose range of the running
// sum of positive deltas holds n.  All of it follows from three prefix sums
// over the requests, so one cluster does the whole plan: every CTA forms the
// sums of all requests in its own shared memory (a few KB of reads) and the
// CTAs share out the pages and the tokens.  Nothing is written until every
// CTA knows that the plan fits.  Bound: launch and dependent-access latency
// (16 bytes per request and 12 per token are read and written in all).
#include "decode4.h"
#include "prox_device.cuh"

namespace prox {
namespace {

constexpr int kMaxPlanCtas = 8;

__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Largest i in [0, n) with pre[i] <= v (pre ascending, pre[0] = 0 <= v).
__device__ __forceinline__ int find_row(const int* pre, int n, int v) {
  int lo = 0, hi = n;  // pre[lo] <= v < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= v)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(1024) page_plan_kernel(PagePlan p, int ctas) {
  extern __shared__ int smem[];
  int* s_new = smem;                 // [B + 1] first new token of each request
  int* s_gain = s_new + p.B + 1;     // [B + 1] first page each request takes
  int* s_drop = s_gain + p.B + 1;    // [B + 1] first page each request returns
  int* s_len = s_drop + p.B + 1;     // [B]
  __shared__ long long scratch[33];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, per = (p.B + blockDim.x - 1) / blockDim.x;
  const int lo = min(tid * per, p.B), hi = min(lo + per, p.B);
  const int c0 = *p.count;
  bool bad = false;
  long long n_new = 0, n_page = 0;  // new tokens; pages taken << 32 | pages returned
  for (int i = lo; i < hi; ++i) {
    const long long len = p.lens[i], to = len + p.delta[i];
    s_len[i] = (int)len;
    if (len < 0 || to < 0 || (to + p.page - 1) / p.page > p.cols || (len + p.page - 1) / p.page > p.cols) {
      bad = true;
      continue;
    }
    const int have = (int)((len + p.page - 1) / p.page), need = (int)((to + p.page - 1) / p.page);
    n_new += to > len ? to - len : 0;
    n_page += need > have ? (long long)(need - have) << 32 : (long long)(have - need);
  }
  long long all_new, all_page;
  long long at_new = block_exclusive_scan(n_new, scratch, &all_new);
  long long at_page = block_exclusive_scan(n_page, scratch, &all_page);
  const int taken = (int)(all_page >> 32), returned = (int)(all_page & 0xffffffffLL);
  const long long c1 = (long long)c0 + returned;
  bad |= c0 < 0 || c1 > p.free_cap || taken > c1 || all_new > p.max_new;
  bad = __syncthreads_or(bad);
  if (!bad) {
    for (int i = lo; i < hi; ++i) {
      const int len = s_len[i], to = len + p.delta[i];
      const int have = (len + p.page - 1) / p.page, need = (to + p.page - 1) / p.page;
      s_new[i] = (int)at_new;
      s_gain[i] = (int)(at_page >> 32);
      s_drop[i] = (int)(at_page & 0xffffffffLL);
      at_new += to > len ? to - len : 0;
      at_page += need > have ? (long long)(need - have) << 32 : (long long)(have - need);
    }
    if (tid == 0) s_new[p.B] = (int)all_new, s_gain[p.B] = taken, s_drop[p.B] = returned;
  }
  __syncthreads();
  const int total = bad ? 0 : (int)all_new;
  int top_step = 1;
  while (2 * top_step < p.B) top_step *= 2;
  const int all = gridDim.x * blockDim.x, at = blockIdx.x * blockDim.x + tid;
  if (!bad) {
    for (int n = at; n < returned; n += all) {
      const int i = find_row(s_drop, p.B, n);
      const int need = (s_len[i] + p.delta[i] + p.page - 1) / p.page;
      p.free_pages[c0 + n] = p.table[(size_t)i * p.table_stride + need + (n - s_drop[i])];
    }
    // returned pages are on the list before any is taken
    if (returned > 0) ctas > 1 ? cluster_sync_all() : __syncthreads();
    for (int n = at; n < taken; n += all) {
      const int i = find_row(s_gain, p.B, n);
      const int have = (s_len[i] + p.page - 1) / p.page;
      p.table[(size_t)i * p.table_stride + have + (n - s_gain[i])] = __ldcg(p.free_pages + (c1 - 1 - n));
    }
  }
  // the table is complete, and every CTA has read lens, delta and count
  if (ctas > 1)
    cluster_sync_all();
  else
    __syncthreads();
  // four tokens of a thread at once: their searches and page loads overlap
  for (int n0 = at; n0 < p.max_new; n0 += 4 * all) {
    int row[4], pos[4], id[4], col[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) row[k] = 0;
    for (int step = top_step; step > 0; step >>= 1)  // the largest i with s_new[i] <= n
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (row[k] + step < p.B && s_new[row[k] + step] <= n0 + k * all) row[k] += step;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = n0 + k * all;
      pos[k] = -1;
      if (n < total) {
        pos[k] = s_len[row[k]] + (n - s_new[row[k]]);
        col[k] = pos[k] / p.page;
        id[k] = __ldcg(p.table + (size_t)row[k] * p.table_stride + col[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = n0 + k * all;
      if (n >= p.max_new) break;
      p.slots[n] = pos[k] < 0 ? -1 : (long long)id[k] * p.page + (pos[k] - col[k] * p.page);
      p.positions[n] = pos[k];
    }
  }
  for (int i = at; i <= p.B; i += all) p.cu[i] = bad ? 0 : s_new[i];
  // delta is still read here, so lens_out may be lens but not delta
  for (int i = at; i < p.B; i += all) p.lens_out[i] = bad ? s_len[i] : s_len[i] + p.delta[i];
  if (at == 0) {
    *p.count_out = bad ? c0 : (int)(c1 - taken);
    *p.status = bad;
  }
}

}  // namespace

cudaError_t setup_page_plan() {
  return cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (4 * kPlanMaxRequests + 3) * 4);
}

cudaError_t launch_page_plan(const PagePlan& p, cudaStream_t s) {
  int ctas = 1;
  while (ctas < kMaxPlanCtas && (p.max_new > 2048 * ctas || p.B > 2048 * ctas)) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(p.max_new <= 256 && p.B <= 256 ? 256 : 1024, 1, 1);
  cfg.dynamicSmemBytes = (size_t)(4 * p.B + 3) * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, page_plan_kernel, p, ctas);
}

}  // namespace prox
