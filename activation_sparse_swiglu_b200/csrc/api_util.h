// What the C ABI's translation units share: the calling thread's error
// message, device checks and the allocation that fault injection can fail.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "prox.h"

namespace prox {
namespace api {

// Stores the formatted message for prox_last_error and returns `st`.
prox_status fail(prox_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// The status and message of a failed CUDA call; clears the runtime's error.
prox_status cuda_fail(cudaError_t e, const char* what);
// cudaMalloc, or the failure that prox_debug_fail_alloc asked for.
cudaError_t dev_alloc(void** p, size_t bytes);
template <typename T>
cudaError_t dev_alloc(T** p, size_t bytes) {
  void* v = nullptr;
  const cudaError_t e = dev_alloc(&v, bytes);
  *p = static_cast<T*>(v);
  return e;
}
// The current device and its SM count; PROX_EUNSUPPORTED unless it is sm_100.
prox_status check_device(int* dev, int* sms);

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }
inline bool aligned4(const void* p) { return aligned(p, 4); }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace api
}  // namespace prox

#define PROX_CUDA(call, what)                                   \
  do {                                                          \
    cudaError_t e_ = (call);                                    \
    if (e_ != cudaSuccess) return prox::api::cuda_fail(e_, what); \
  } while (0)
