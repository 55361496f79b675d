// Host-side internals of the 4-bit operators of the decode step: the linear4
// and kv4 handles and the kernel launchers that decode4_api.cu calls.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "prox.h"

namespace prox {

constexpr int kGroupRows = 128;  // input rows of one weight scale
constexpr int kLinear4MaxTokens = 16;
constexpr int kPlanMaxRequests = 8192;    // bounds the page plan's shared memory
constexpr int kPlanMaxNew = 1 << 30;      // token numbers plus a grid's stride stay in 32 bits
constexpr int kAttendMaxRequests = 8192;  // bounds the attention's table of chunk counts

}  // namespace prox

// INT4 weights [K, N] in the order the product's fragments need:
// by strips of 32 channels and groups of 128 input rows, 2 KB of codes and 64
// bytes of scales each (linear4.cu has the order inside).
struct prox_linear4 {
  int K = 0, N = 0, G = 0, strips = 0;
  int device = 0, num_sms = 0;
  int clusters[4] = {0, 0, 0, 0};  // clusters of 1, 2, 4, 8 CTAs that are resident at once
  uint8_t* codes = nullptr;
  uint16_t* scales = nullptr;
  size_t bytes = 0;
};

// A paged 4-bit cache (caller-owned tensors) and the attention's workspace.
struct prox_kv4 {
  uint8_t* k = nullptr;
  uint16_t* ks = nullptr;
  uint8_t* v = nullptr;
  uint16_t* vs = nullptr;
  int pages = 0, heads = 0, page = 0, D = 0;
  int device = 0, num_sms = 0;
  int* err = nullptr;
  float* part = nullptr;       // [2 * num_sms] partial results of contexts that CTAs share
  float* warp_part = nullptr;  // [num_sms * warps] ... that warps share
  int* arrived = nullptr;   // [num_sms] CTAs that left a part, zero between calls
  void* base = nullptr;
  size_t bytes = 0;
};

namespace prox {

cudaError_t launch_linear4_pack(const uint8_t* codes, const uint16_t* scales, const prox_linear4* L, cudaStream_t s);
// Loads the kernels and counts the clusters of each size that fit at once.
cudaError_t setup_linear4(prox_linear4* L);
cudaError_t launch_linear4(const prox_linear4* L, const void* x, int64_t x_stride, void* out, int64_t out_stride,
                           int B, int dtype, cudaStream_t s);

cudaError_t launch_kv4_append(const prox_kv4* C, const void* k, const void* v, int64_t k_token, int64_t k_head,
                              int64_t v_token, int64_t v_head, const int64_t* slots, int T, int dtype, cudaStream_t s);
cudaError_t launch_kv4_read(const prox_kv4* C, const int64_t* slots, int T, void* k, void* v, int dtype,
                            cudaStream_t s);

cudaError_t setup_attend4();
size_t attend4_part_floats(int D);  // one partial result
int attend4_warps();                // of a CTA, at most
struct Attend4Call {
  const void* q = nullptr;
  int64_t q_req = 0, q_tok = 0, q_head = 0;  // strides in elements
  void* out = nullptr;                       // [B, Tq, Hq, D] contiguous
  float* lse = nullptr;                      // [B, Tq, Hq] or NULL
  const int32_t* table = nullptr;
  int64_t table_stride = 0;
  int cols = 0;
  const int32_t* lens = nullptr;
  int B = 0, Tq = 0, Hq = 0, dtype = 0;
  float scale = 0.f;
};
cudaError_t launch_attend4(const prox_kv4* C, const Attend4Call& c, cudaStream_t s);

struct PagePlan {
  const int32_t* lens = nullptr;
  const int32_t* delta = nullptr;
  int B = 0, page = 0;
  int32_t* table = nullptr;
  int64_t table_stride = 0;
  int cols = 0;
  int32_t* free_pages = nullptr;
  int free_cap = 0;
  const int32_t* count = nullptr;
  int32_t* lens_out = nullptr;
  int32_t* count_out = nullptr;
  int32_t* cu = nullptr;
  int64_t* slots = nullptr;
  int32_t* positions = nullptr;
  int max_new = 0;
  int32_t* status = nullptr;
};
// Loads the kernel and finds the largest cluster (CTAs) the device can hold.
cudaError_t setup_page_plan(int* max_ctas);
cudaError_t launch_page_plan(const PagePlan& p, int max_ctas, cudaStream_t s);

}  // namespace prox
