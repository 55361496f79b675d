// C ABI of the 4-bit operators: argument checks, the linear4 and kv4 handles,
// and their launches.
#include <atomic>
#include <climits>
#include <cmath>
#include <new>

#include "api_util.h"
#include "decode4.h"
#include "prox_internal.h"

using namespace prox::api;

namespace {

constexpr int kMaxIn = 65536;
constexpr int kMaxOut = 1 << 20;
constexpr int kMaxDevices = 64;

bool good_dtype(int dtype) { return dtype == PROX_F32 || dtype == PROX_F16 || dtype == PROX_BF16; }
size_t dtype_size(int dtype) { return dtype == PROX_F32 ? 4 : 2; }

prox_status on_device(int device, const char* what) {
  int dev = -1;
  PROX_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev != device) return fail(PROX_EINVAL, "%s lives on device %d but device %d is current", what, device, dev);
  return PROX_OK;
}

prox_status linear4_shape(int d_in, int d_out) {
  if (d_in <= 0 || d_in % prox::kGroupRows != 0 || d_in > kMaxIn)
    return fail(PROX_EINVAL, "d_in=%d must be a positive multiple of 128 and <= %d", d_in, kMaxIn);
  if (d_out <= 0 || d_out % 2 != 0 || d_out > kMaxOut)
    return fail(PROX_EINVAL, "d_out=%d must be positive, even and <= %d", d_out, kMaxOut);
  return PROX_OK;
}

// Whether B rows of n_a values at a share memory with B rows of n_b values at
// b.  Rows of one stride may interleave (column ranges of one buffer); rows of
// two strides may not even share a range.
bool rows_overlap(const void* a, int64_t n_a, int64_t s_a, const void* b, int64_t n_b, int64_t s_b, int B,
                  size_t size) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  const uintptr_t ea = pa + ((B - 1) * s_a + n_a) * size, eb = pb + ((B - 1) * s_b + n_b) * size;
  if (ea <= pb || eb <= pa) return false;
  if (B == 1 || s_a != s_b) return true;
  const uintptr_t stride = s_a * size;
  const uintptr_t d = pb >= pa ? (pb - pa) % stride : (stride - (pa - pb) % stride) % stride;
  return d < n_a * size || d + n_b * size > stride;
}

struct Span {
  uintptr_t lo, hi;
  bool meets(const Span& o) const { return lo < o.hi && o.lo < hi; }
};
Span span_of(const void* p, int64_t n, size_t size) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return {at, at + n * size};
}

// Whether `w` meets the queries of any request.  (Between requests there may
// be anything: q may be a column range of wider rows.)
bool meets_queries(const Span& w, const prox::Attend4Call& c, int D) {
  const size_t size = dtype_size(c.dtype);
  auto queries = [&](int b0, int b1) {  // of requests [b0, b1]
    int64_t lo = 0, hi = D;
    auto along = [&](int64_t stride, int64_t first, int64_t last) {
      lo += stride < 0 ? stride * last : stride * first;
      hi += stride < 0 ? stride * first : stride * last;
    };
    along(c.q_req, b0, b1);
    along(c.q_tok, 0, c.Tq - 1);
    along(c.q_head, 0, c.Hq - 1);
    return span_of(static_cast<const char*>(c.q) + lo * (int64_t)size, hi - lo, size);
  };
  if (!w.meets(queries(0, c.B - 1))) return false;
  for (int b = 0; b < c.B; ++b)
    if (w.meets(queries(b, b))) return true;
  return false;
}

// Allocates the handle and its buffers for a checked shape.
prox_status linear4_new(int d_in, int d_out, prox_linear4** out) {
  int dev, sms;
  prox_status st = check_device(&dev, &sms);
  if (st != PROX_OK) return st;
  prox_linear4* L = new (std::nothrow) prox_linear4();
  if (!L) return fail(PROX_ENOMEM, "host allocation failed");
  L->K = d_in;
  L->N = d_out;
  L->G = d_in / prox::kGroupRows;
  L->strips = (d_out + 31) / 32;
  L->device = dev;
  L->num_sms = sms;
  const size_t units = (size_t)L->strips * L->G, code_bytes = units * 2048, scale_bytes = units * 64;
  cudaError_t e = prox::setup_linear4(L);
  if (e == cudaSuccess) e = dev_alloc(&L->codes, code_bytes + scale_bytes);
  if (e != cudaSuccess) {
    delete L;
    return cuda_fail(e, "prox_linear4_create");
  }
  L->scales = reinterpret_cast<uint16_t*>(L->codes + code_bytes);
  L->bytes = code_bytes + scale_bytes;
  *out = L;
  return PROX_OK;
}

void linear4_free(prox_linear4* L) {
  int cur = 0;
  cudaGetDevice(&cur);
  if (cur != L->device) cudaSetDevice(L->device);
  if (L->codes) cudaFree(L->codes);
  if (cur != L->device) cudaSetDevice(cur);
  delete L;
}

}  // namespace

extern "C" {

prox_status prox_linear4_create(const uint8_t* codes, const uint16_t* scales, int d_in, int d_out, void* stream,
                                prox_linear4** out_host) {
  if (!out_host) return fail(PROX_EINVAL, "out_host is NULL");
  *out_host = nullptr;
  prox_status st = linear4_shape(d_in, d_out);
  if (st != PROX_OK) return st;
  if (!codes || !scales || !aligned(scales, 2))
    return fail(PROX_EINVAL, "codes and scales must be non-NULL, scales 2-byte aligned");
  prox_linear4* L = nullptr;
  if ((st = linear4_new(d_in, d_out, &L)) != PROX_OK) return st;
  cudaStream_t s = as_stream(stream);
  cudaError_t e = prox::launch_linear4_pack(codes, scales, L, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) {
    linear4_free(L);
    return cuda_fail(e, "prox_linear4_create");
  }
  *out_host = L;
  return PROX_OK;
}

prox_status prox_linear4_create_bf16(const uint16_t* W, int d_in, int d_out, void* stream, prox_linear4** out_host) {
  if (!out_host) return fail(PROX_EINVAL, "out_host is NULL");
  *out_host = nullptr;
  prox_status st = linear4_shape(d_in, d_out);
  if (st != PROX_OK) return st;
  if (!W || !aligned4(W)) return fail(PROX_EINVAL, "W must be a 4-byte aligned pointer");
  prox_linear4* L = nullptr;
  if ((st = linear4_new(d_in, d_out, &L)) != PROX_OK) return st;
  cudaStream_t s = as_stream(stream);
  const size_t n_codes = (size_t)d_in * d_out / 2;
  uint8_t* tmp = nullptr;
  cudaError_t e = dev_alloc(&tmp, align256(n_codes) + (size_t)L->G * d_out * 2);
  if (e == cudaSuccess) {
    uint16_t* sc = reinterpret_cast<uint16_t*>(tmp + align256(n_codes));
    e = prox::launch_pack_proxy(W, d_in, d_out, tmp, sc, s);
    if (e == cudaSuccess) e = prox::launch_linear4_pack(tmp, sc, L, s);
    const cudaError_t sync = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = sync;
    cudaFree(tmp);
  }
  if (e != cudaSuccess) {
    linear4_free(L);
    return cuda_fail(e, "prox_linear4_create_bf16");
  }
  *out_host = L;
  return PROX_OK;
}

prox_status prox_linear4_destroy(prox_linear4* L) {
  if (L) linear4_free(L);
  return PROX_OK;
}

prox_status prox_linear4_forward(const prox_linear4* L, const void* x, int64_t x_stride, void* out,
                                 int64_t out_stride, int B, int dtype, void* stream) {
  if (!L) return fail(PROX_EINVAL, "linear4 handle is NULL");
  if (!good_dtype(dtype)) return fail(PROX_EINVAL, "dtype %d is not one of PROX_F32, PROX_F16, PROX_BF16", dtype);
  if (B < 1 || B > prox::kLinear4MaxTokens)
    return fail(PROX_EINVAL, "B=%d must be in [1, %d]", B, prox::kLinear4MaxTokens);
  if (!x || !out || !aligned(x, dtype_size(dtype)) || !aligned(out, dtype_size(dtype)))
    return fail(PROX_EINVAL, "x and out must be non-NULL and aligned to their type");
  if (B > 1 && (x_stride < L->K || out_stride < L->N))
    return fail(PROX_EINVAL, "x_stride=%lld and out_stride=%lld must be at least d_in=%d and d_out=%d",
                (long long)x_stride, (long long)out_stride, L->K, L->N);
  if (rows_overlap(x, L->K, x_stride, out, L->N, out_stride, B, dtype_size(dtype)))
    return fail(PROX_EINVAL, "out may not overlap x");
  prox_status st = on_device(L->device, "linear4");
  if (st != PROX_OK) return st;
  PROX_CUDA(prox::launch_linear4(L, x, x_stride, out, out_stride, B, dtype, as_stream(stream)),
            "prox_linear4_forward launch");
  return PROX_OK;
}

prox_status prox_kv4_create(uint8_t* k_codes, uint16_t* k_scales, uint8_t* v_codes, uint16_t* v_scales,
                            int num_pages, int n_heads, int page_size, int head_dim, prox_kv4** out_host) {
  if (!out_host) return fail(PROX_EINVAL, "out_host is NULL");
  *out_host = nullptr;
  if (num_pages < 1 || n_heads < 1 || n_heads > 1024)
    return fail(PROX_EINVAL, "num_pages=%d must be positive and n_heads=%d in [1, 1024]", num_pages, n_heads);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(PROX_EINVAL, "head_dim=%d must be 64, 128 or 256", head_dim);
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return fail(PROX_EINVAL, "page_size=%d must be 16, 32, 64, 128 or 256", page_size);
  if (!k_codes || !v_codes || !aligned16(k_codes) || !aligned16(v_codes))
    return fail(PROX_EINVAL, "k_codes and v_codes must be non-NULL 16-byte aligned pointers");
  if (!k_scales || !v_scales || !aligned(k_scales, 32) || !aligned(v_scales, 32))
    return fail(PROX_EINVAL, "k_scales and v_scales must be non-NULL 32-byte aligned pointers");
  int dev, sms;
  prox_status st = check_device(&dev, &sms);
  if (st != PROX_OK) return st;
  prox_kv4* C = new (std::nothrow) prox_kv4();
  if (!C) return fail(PROX_ENOMEM, "host allocation failed");
  C->k = k_codes;
  C->ks = k_scales;
  C->v = v_codes;
  C->vs = v_scales;
  C->pages = num_pages;
  C->heads = n_heads;
  C->page = page_size;
  C->D = head_dim;
  C->device = dev;
  C->num_sms = sms;
  const size_t one = prox::attend4_part_floats(head_dim) * 4;
  const size_t warp_part = align256((size_t)sms * prox::attend4_warps() * one);
  const size_t part = align256(2 * (size_t)sms * one) + warp_part;
  const size_t arrived = align256((size_t)sms * 4);
  C->bytes = part + arrived + 256;
  cudaError_t e = prox::setup_attend4();
  if (e == cudaSuccess) e = dev_alloc(&C->base, C->bytes);
  if (e == cudaSuccess) {
    e = cudaMemset(static_cast<char*>(C->base) + part, 0, arrived + 256);
    // the legacy stream's clear is done before any other stream uses it
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  }
  if (e != cudaSuccess) {
    if (C->base) cudaFree(C->base);
    delete C;
    return cuda_fail(e, "prox_kv4_create");
  }
  char* b = static_cast<char*>(C->base);
  C->warp_part = reinterpret_cast<float*>(b);
  C->part = reinterpret_cast<float*>(b + warp_part);
  C->arrived = reinterpret_cast<int*>(b + part);
  C->err = reinterpret_cast<int*>(b + part + arrived);
  *out_host = C;
  return PROX_OK;
}

prox_status prox_kv4_destroy(prox_kv4* C) {
  if (!C) return PROX_OK;
  int cur = 0;
  cudaGetDevice(&cur);
  if (cur != C->device) cudaSetDevice(C->device);
  cudaFree(C->base);
  if (cur != C->device) cudaSetDevice(cur);
  delete C;
  return PROX_OK;
}

prox_status prox_kv4_error(prox_kv4* C, int32_t* word_host, void* stream) {
  if (!C || !word_host) return fail(PROX_EINVAL, "NULL argument");
  prox_status st = on_device(C->device, "kv4 cache");
  if (st != PROX_OK) return st;
  cudaStream_t s = as_stream(stream);
  int32_t v = 0;
  PROX_CUDA(cudaMemcpyAsync(&v, C->err, 4, cudaMemcpyDeviceToHost, s), "read error word");
  PROX_CUDA(cudaMemsetAsync(C->err, 0, 4, s), "clear error word");
  PROX_CUDA(cudaStreamSynchronize(s), "cudaStreamSynchronize");
  *word_host = v;
  return PROX_OK;
}

// Rows of one append or read fit the grid.
static prox_status check_rows(const prox_kv4* C, const int64_t* slots, int T, int dtype) {
  if (!C) return fail(PROX_EINVAL, "kv4 handle is NULL");
  if (!good_dtype(dtype)) return fail(PROX_EINVAL, "dtype %d is not one of PROX_F32, PROX_F16, PROX_BF16", dtype);
  if (T < 0 || (int64_t)T * C->heads > INT_MAX)
    return fail(PROX_EINVAL, "T=%d must be >= 0 and T * n_heads below 2^31", T);
  if (T > 0 && (!slots || !aligned(slots, 8))) return fail(PROX_EINVAL, "slots must be an 8-byte aligned pointer");
  return on_device(C->device, "kv4 cache");
}

prox_status prox_kv4_append(const prox_kv4* C, const void* k, const void* v, int64_t k_token, int64_t k_head,
                            int64_t v_token, int64_t v_head, const int64_t* slots, int T, int dtype, void* stream) {
  prox_status st = check_rows(C, slots, T, dtype);
  if (st != PROX_OK) return st;
  if (T == 0) return PROX_OK;
  if (!k || !v || !aligned(k, dtype_size(dtype)) || !aligned(v, dtype_size(dtype)))
    return fail(PROX_EINVAL, "k and v must be non-NULL and aligned to their type");
  PROX_CUDA(prox::launch_kv4_append(C, k, v, k_token, k_head, v_token, v_head, slots, T, dtype, as_stream(stream)),
            "prox_kv4_append launch");
  return PROX_OK;
}

prox_status prox_kv4_read(const prox_kv4* C, const int64_t* slots, int T, void* k_out, void* v_out, int dtype,
                          void* stream) {
  prox_status st = check_rows(C, slots, T, dtype);
  if (st != PROX_OK) return st;
  if (T == 0) return PROX_OK;
  if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out))
    return fail(PROX_EINVAL, "k_out and v_out must be non-NULL 16-byte aligned pointers");
  PROX_CUDA(prox::launch_kv4_read(C, slots, T, k_out, v_out, dtype, as_stream(stream)), "prox_kv4_read launch");
  return PROX_OK;
}

prox_status prox_kv4_attend(const prox_kv4* C, const void* q, int64_t q_req, int64_t q_tok, int64_t q_head,
                            int n_q_heads, int B, int Tq, const int32_t* table, int64_t table_stride, int cols,
                            const int32_t* lens, float scale, void* out, float* lse, int dtype, void* stream) {
  if (!C) return fail(PROX_EINVAL, "kv4 handle is NULL");
  if (!good_dtype(dtype)) return fail(PROX_EINVAL, "dtype %d is not one of PROX_F32, PROX_F16, PROX_BF16", dtype);
  if (B < 1 || B > prox::kAttendMaxRequests)
    return fail(PROX_EINVAL, "B=%d must be in [1, %d]", B, prox::kAttendMaxRequests);
  if (n_q_heads < 1 || n_q_heads % C->heads != 0)
    return fail(PROX_EINVAL, "n_q_heads=%d must be a positive multiple of the cache's %d heads", n_q_heads, C->heads);
  if (Tq < 1 || (int64_t)Tq * n_q_heads > (1 << 20))
    return fail(PROX_EINVAL, "Tq=%d must be positive and Tq * n_q_heads at most 2^20", Tq);
  if (cols < 0 || table_stride < cols) return fail(PROX_EINVAL, "cols=%d must be >= 0 and table_stride >= cols", cols);
  if (((int64_t)cols * C->page / 32 + 3) * Tq * n_q_heads >= (int64_t)1 << 32)
    return fail(PROX_EINVAL, "cols * page_size * Tq * n_q_heads must stay below 2^36");
  // (units of 32 rows, 2 for a start and 1 for a ragged end, of all requests: see attend4.cu)
  if (((int64_t)cols * C->page / 32 + 3) * B > INT_MAX)
    return fail(PROX_EINVAL, "B * cols * page_size must stay below 2^36 (with 96 tokens more a request)");
  if (!std::isfinite(scale)) return fail(PROX_EINVAL, "scale must be finite");
  if (!q || !aligned(q, dtype_size(dtype)) || !out || !aligned16(out))
    return fail(PROX_EINVAL, "q must be aligned to its type and out a 16-byte aligned pointer");
  if (!lens || !aligned4(lens) || (cols > 0 && (!table || !aligned4(table))) || !aligned4(lse))
    return fail(PROX_EINVAL, "lens, table and lse must be 4-byte aligned pointers");
  prox::Attend4Call c;
  c.q = q;
  c.q_req = q_req;
  c.q_tok = q_tok;
  c.q_head = q_head;
  c.out = out;
  c.lse = lse;
  c.table = table;
  c.table_stride = table_stride;
  c.cols = cols;
  c.lens = lens;
  c.B = B;
  c.Tq = Tq;
  c.Hq = n_q_heads;
  c.dtype = dtype;
  c.scale = scale;
  // A request's queries are read when its turn comes, other requests' results
  // are written by then.  Results in the queries' own places are fine: a row is
  // written after all that read it.
  const int64_t rows = (int64_t)B * Tq * n_q_heads;
  const Span to = span_of(out, rows * C->D, dtype_size(dtype)), lse_to = span_of(lse, lse ? rows : 0, 4);
  const Span in_lens = span_of(lens, B, 4), in_table = span_of(table, cols ? (B - 1) * table_stride + cols : 0, 4);
  const bool in_place = out == q && (n_q_heads == 1 || q_head == C->D) &&
                        (Tq == 1 || q_tok == (int64_t)n_q_heads * C->D) &&
                        (B == 1 || q_req == (int64_t)Tq * n_q_heads * C->D);
  if ((!in_place && meets_queries(to, c, C->D)) || (lse && meets_queries(lse_to, c, C->D)))
    return fail(PROX_EINVAL, "out and lse may not overlap q (unless out is q, contiguous)");
  if (to.meets(lse_to) || to.meets(in_lens) || to.meets(in_table) || lse_to.meets(in_lens) || lse_to.meets(in_table))
    return fail(PROX_EINVAL, "out and lse may not overlap each other, lens or table");
  prox_status st = on_device(C->device, "kv4 cache");
  if (st != PROX_OK) return st;
  PROX_CUDA(prox::launch_attend4(C, c, as_stream(stream)), "prox_kv4_attend launch");
  return PROX_OK;
}

prox_status prox_plan_pages(const int32_t* lens, const int32_t* delta, int B, int page_size, int32_t* table,
                            int64_t table_stride, int cols, int32_t* free_pages, int free_cap,
                            const int32_t* free_count, int32_t* lens_out, int32_t* free_count_out, int32_t* cu,
                            int64_t* slots, int32_t* positions, int max_new, int32_t* status, void* stream) {
  if (B < 1 || B > prox::kPlanMaxRequests)
    return fail(PROX_EINVAL, "B=%d must be in [1, %d]", B, prox::kPlanMaxRequests);
  if (page_size < 1 || page_size > 1 << 30) return fail(PROX_EINVAL, "page_size=%d must be in [1, 2^30]", page_size);
  if (cols < 0 || table_stride < cols || (int64_t)B * cols > INT_MAX)
    return fail(PROX_EINVAL, "cols=%d must be >= 0, table_stride >= cols and B * cols < 2^31", cols);
  if (free_cap < 0 || max_new < 0) return fail(PROX_EINVAL, "free_cap and max_new must be >= 0");
  if (max_new > prox::kPlanMaxNew) return fail(PROX_EINVAL, "max_new=%d must be at most 2^30", max_new);
  const void* words[] = {lens, delta, free_count, lens_out, free_count_out, cu, status};
  for (const void* w : words)
    if (!w || !aligned4(w)) return fail(PROX_EINVAL, "pointers must be non-NULL and 4-byte aligned");
  if ((cols > 0 && (!table || !aligned4(table))) || (free_cap > 0 && (!free_pages || !aligned4(free_pages))) ||
      (max_new > 0 && (!slots || !aligned(slots, 8) || !positions || !aligned4(positions))))
    return fail(PROX_EINVAL, "table, free_pages, positions (4-byte) and slots (8-byte aligned) must be non-NULL");
  if (lens_out == delta) return fail(PROX_EINVAL, "lens_out may not alias delta");
  int dev, sms;
  prox_status st = check_device(&dev, &sms);
  if (st != PROX_OK) return st;
  if (dev >= kMaxDevices) return fail(PROX_EUNSUPPORTED, "device ordinal %d out of range", dev);
  static std::atomic<int> ctas_of[kMaxDevices];  // largest cluster, 0: not set up yet
  int ctas = ctas_of[dev].load(std::memory_order_acquire);
  if (ctas == 0) {
    PROX_CUDA(prox::setup_page_plan(&ctas), "prox_plan_pages set-up");
    ctas_of[dev].store(ctas, std::memory_order_release);
  }
  prox::PagePlan p;
  p.lens = lens;
  p.delta = delta;
  p.B = B;
  p.page = page_size;
  p.table = table;
  p.table_stride = table_stride;
  p.cols = cols;
  p.free_pages = free_pages;
  p.free_cap = free_cap;
  p.count = free_count;
  p.lens_out = lens_out;
  p.count_out = free_count_out;
  p.cu = cu;
  p.slots = slots;
  p.positions = positions;
  p.max_new = max_new;
  p.status = status;
  PROX_CUDA(prox::launch_page_plan(p, ctas, as_stream(stream)), "prox_plan_pages launch");
  return PROX_OK;
}

}  // extern "C"
