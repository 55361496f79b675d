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
// CTA knows that the plan fits.
//
// Which page a row gains is read off the prefix sums and what was there before
// the call (the free list, or the row that returns it), so pages are returned
// and taken without a barrier between; one barrier stands before the tokens,
// which read the finished table.  A warp takes 128 tokens in a row: one search
// for the first, then steps from request to request, and four page loads of a
// lane at once.  (With a search per token 1021 requests gaining 86000 tokens
// took 21 us, bound by issue on the cluster's eight SMs.)
//
// Bound: launch and dependent-access latency (16 bytes per request and 12 per
// token are read and written in all).
#include <climits>

#include "decode4.h"
#include "prox_device.cuh"

namespace prox {
namespace {

constexpr int kMaxPlanCtas = 16;  // beyond 8 a cluster needs the kernel's consent

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

// Exclusive prefix sums of two values over the threads of the block, and their
// totals.
__device__ __forceinline__ void scan2(long long a, long long b, longlong2* scratch, long long* at_a, long long* at_b,
                                      long long* all_a, long long* all_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  long long x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += u, y += v;
  }
  if (lane == 31) scratch[warp] = make_longlong2(x, y);
  __syncthreads();
  // every warp sums the warps before it
  longlong2 w = lane < warps ? scratch[lane] : make_longlong2(0, 0);
  long long before_x = lane < warp ? w.x : 0, before_y = lane < warp ? w.y : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before_x += __shfl_xor_sync(0xffffffffu, before_x, o);
    before_y += __shfl_xor_sync(0xffffffffu, before_y, o);
    w.x += __shfl_xor_sync(0xffffffffu, w.x, o);
    w.y += __shfl_xor_sync(0xffffffffu, w.y, o);
  }
  *at_a = before_x + x - a;
  *at_b = before_y + y - b;
  *all_a = w.x;
  *all_b = w.y;
}

__global__ void __launch_bounds__(1024, 1) page_plan_kernel(PagePlan p, int ctas, int shift) {
  extern __shared__ int smem[];
  int* s_new = smem;                 // [B + 1] first new token of each request
  int* s_gain = s_new + p.B + 1;     // [B + 1] first page each request takes
  int* s_drop = s_gain + p.B + 1;    // [B + 1] first page each request returns
  int* s_len = s_drop + p.B + 1;     // [B] before
  int* s_to = s_len + p.B;           // [B] after
  __shared__ longlong2 scratch[33];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, per = (p.B + blockDim.x - 1) / blockDim.x;
  const int lo = min(tid * per, p.B), hi = min(lo + per, p.B);
  const int c0 = *p.count;
  const unsigned page = p.page;  // a power of two if shift >= 0
  auto over_page = [&](unsigned v) { return shift >= 0 ? v >> shift : v / page; };
  auto pages = [&](int tokens) { return (int)over_page((unsigned)tokens + page - 1); };  // tokens >= 0, page <= 2^30
  bool bad = false;
  long long n_new = 0, n_page = 0;  // new tokens; pages taken << 32 | pages returned
  for (int i = lo; i < hi; ++i) {
    const long long len = p.lens[i], to = len + p.delta[i];
    s_len[i] = (int)len;
    s_to[i] = (int)to;
    if (len < 0 || to < 0 || to > INT_MAX || pages((int)to) > p.cols || pages((int)len) > p.cols) {
      bad = true;
      continue;
    }
    const int have = pages((int)len), need = pages((int)to);
    n_new += to > len ? to - len : 0;
    n_page += need > have ? (long long)(need - have) << 32 : (long long)(have - need);
  }
  long long all_new, all_page, at_new, at_page;
  scan2(n_new, n_page, scratch, &at_new, &at_page, &all_new, &all_page);
  const int taken = (int)(all_page >> 32), returned = (int)(all_page & 0xffffffffLL);
  const long long c1 = (long long)c0 + returned;
  bad |= c0 < 0 || c1 > p.free_cap || taken > c1 || all_new > p.max_new;
  bad = __syncthreads_or(bad);
  if (!bad) {
    for (int i = lo; i < hi; ++i) {
      const int have = pages(s_len[i]), need = pages(s_to[i]);
      s_new[i] = (int)at_new;
      s_gain[i] = (int)(at_page >> 32);
      s_drop[i] = (int)(at_page & 0xffffffffLL);
      at_new += max(0, s_to[i] - s_len[i]);
      at_page += need > have ? (long long)(need - have) << 32 : (long long)(have - need);
    }
    if (tid == 0) s_new[p.B] = (int)all_new, s_gain[p.B] = taken, s_drop[p.B] = returned;
  }
  __syncthreads();
  const int total = bad ? 0 : (int)all_new;
  const int all = gridDim.x * blockDim.x, at = blockIdx.x * blockDim.x + tid;
  auto entry = [&](int i, int col) { return p.table + (size_t)i * p.table_stride + col; };
  // returned page n, of those before any is taken
  auto returned_page = [&](int n) {
    const int i = find_row(s_drop, p.B, n);
    return *entry(i, pages(s_to[i]) + (n - s_drop[i]));
  };
  // the n-th page taken: from the end of the free list with the returned pages on it
  auto taken_page = [&](int n) {
    const long long j = c1 - 1 - n;
    return j < c0 ? p.free_pages[j] : returned_page((int)(j - c0));
  };
  if (!bad) {
    const unsigned moved = max(returned, taken);  // (up to 2^31: n may pass it by the CTAs' threads)
    for (unsigned u = at; u < moved; u += all) {  // both lookups before either write
      const int n = (int)u;
      const int back = n < returned ? returned_page(n) : 0;
      if (n < taken) {
        const int i = find_row(s_gain, p.B, n), id = taken_page(n);
        *entry(i, pages(s_len[i]) + (n - s_gain[i])) = id;
      }
      if (n < returned) p.free_pages[c0 + n] = back;
    }
  }
  // The table is complete, and what lens_out and count_out may replace is read.
  if (ctas > 1)
    cluster_sync_all();
  else
    __syncthreads();
  const int lane = tid & 31;
  const bool sparse = total < 4 * p.B;  // few tokens a request: a search each beats the steps
  const int per_lane = p.max_new <= all ? 1 : 4;  // (n0 stays below kPlanMaxNew + 4 all)
  for (int n0 = (at >> 5) * (32 * per_lane); n0 < p.max_new; n0 += all * per_lane) {
    int i = !sparse && n0 < total ? find_row(s_new, p.B, n0) : 0;
    int pos[4], id[4];
    unsigned off[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = n0 + 32 * k + lane;
      pos[k] = -1;
      id[k] = 0;
      off[k] = 0;
      if (k < per_lane && n < total) {
        if (sparse)
          i = find_row(s_new, p.B, n);
        else
          while (s_new[i + 1] <= n) ++i;
        pos[k] = s_len[i] + (n - s_new[i]);
        const unsigned col = over_page(pos[k]);
        off[k] = pos[k] - col * page;
        id[k] = __ldcg(entry(i, col));
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = n0 + 32 * k + lane;
      if (k >= per_lane || n >= p.max_new) break;
      p.slots[n] = pos[k] < 0 ? -1 : (long long)id[k] * page + off[k];
      p.positions[n] = pos[k];
    }
  }
  for (int i = at; i <= p.B; i += all) p.cu[i] = bad ? 0 : s_new[i];
  for (int i = at; i < p.B; i += all) p.lens_out[i] = bad ? s_len[i] : s_to[i];
  if (at == 0) {
    *p.count_out = bad ? c0 : (int)(c1 - taken);
    *p.status = bad;
  }
}

}  // namespace

cudaError_t setup_page_plan(int* max_ctas) {
  const size_t smem = (5 * kPlanMaxRequests + 3) * 4;
  cudaError_t e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kMaxPlanCtas, 1, 1);
  cfg.blockDim = dim3(1024, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kMaxPlanCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, page_plan_kernel, &cfg) != cudaSuccess) cudaGetLastError(), n = 0;
  *max_ctas = n > 0 ? kMaxPlanCtas : 8;  // eight are portable
  return cudaSuccess;
}

cudaError_t launch_page_plan(const PagePlan& p, int max_ctas, cudaStream_t s) {
  int ctas = 1;
  while (ctas < max_ctas && (p.max_new > 4096 * ctas || p.B > 2048 * ctas)) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(p.max_new <= 256 && p.B <= 256 ? 256 : 1024, 1, 1);
  cfg.dynamicSmemBytes = (size_t)(5 * p.B + 3) * 4;
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
  int shift = -1;
  if ((p.page & (p.page - 1)) == 0)
    while ((1 << ++shift) < p.page) {
    }
  return cudaLaunchKernelEx(&cfg, page_plan_kernel, p, ctas, shift);
}

}  // namespace prox
