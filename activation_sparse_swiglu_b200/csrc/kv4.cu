// The paged 4-bit cache's rows: quantised at their slots, and read back.
//
// One row is the D values of one token and head.  D / 16 lanes share a row,
// 16 values each as two runs of 8 (so that every load and store of the row is
// contiguous over its lanes): the largest magnitude by shuffles, the scale
// S = fp16(amax / 7), and the codes.
//
// The code of x is x / S rounded half to even, exactly: n = rint(x * (1 / S))
// is off by at most one, and e = x - n S is exact in one fused multiply-add
// (n S has at most 15 significant bits, and |e| < S is a multiple of both
// numbers' units), so comparing |e| with S / 2 settles n, ties included.
//
// Bound: HBM for prompts (16000 tokens x 8 heads of 128: 65 MB in, 17 MB
// out); launch latency for the rows of a decode step.
#include <type_traits>

#include "decode4.h"
#include "quant4.cuh"

namespace prox {
namespace {

using namespace q4;

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t code8(const float (&x)[8], float s) {
  const float half = 0.5f * s, rs = 1.0f / s;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float n = rintf(x[i] * rs);
    const float e = fmaf(-n, s, x[i]), a = fabsf(e);
    if (a >= half && (a > half || (((int)n) & 1))) n += copysignf(1.f, e);
    // s > 0 and finite: n is finite; a NaN or infinity in x gave s = NaN or inf
    const int q = s > 0.f ? (int)fminf(fmaxf(n, -7.f), 7.f) : 0;
    w |= (uint32_t)(q + 8) << (4 * i);
  }
  return w;
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(prox_kv4 C, const void* k_in, const void* v_in,
                                                          int64_t k_token, int64_t k_head, int64_t v_token,
                                                          int64_t v_head, const int64_t* slots, int T, bool vec) {
  using T_ = typename Act<DT>::T;
  constexpr int LPR = D / 16;  // lanes of one row
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % LPR;
  const int64_t row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / LPR;
  const bool is_v = blockIdx.y;
  if (row / C.heads >= T) return;  // a whole row's lanes leave together
  const int t = (int)(row / C.heads), h = (int)(row % C.heads);
  const int64_t slot = slots[t];
  if (slot < 0) return;
  if (slot >= (int64_t)C.pages * C.page) {
    if (lane == 0) atomicOr(C.err, PROX_DEVERR_SLOT);
    return;
  }
  const T_* x = static_cast<const T_*>(is_v ? v_in : k_in) + t * (is_v ? v_token : k_token) +
                h * (is_v ? v_head : k_head);
  float a[8], b[8];
  load_vals<DT, 8>(x + 8 * lane, vec, a);
  load_vals<DT, 8>(x + D / 2 + 8 * lane, vec, b);
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = max_nan(mx, max_nan(fabsf(a[i]), fabsf(b[i])));
  const unsigned mask = (LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1)) << ((threadIdx.x & 31) / LPR * LPR);
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(mask, mx, o));
  const __half sh = __float2half_rn(mx / 7.0f);
  const float s = __half2float(sh);
  const int64_t page = slot / C.page, r = slot % C.page;
  const int64_t at = (page * C.heads + h) * C.page + r;
  uint8_t* dst = (is_v ? C.v : C.k) + at * (D / 2);
  *reinterpret_cast<uint32_t*>(dst + 4 * lane) = code8(a, s);
  *reinterpret_cast<uint32_t*>(dst + D / 4 + 4 * lane) = code8(b, s);
  if (lane == 0) reinterpret_cast<__half*>(is_v ? C.vs : C.ks)[at] = sh;
}

__device__ __forceinline__ void value8(uint32_t w, float s, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)((int)((w >> (4 * i)) & 15u) - 8) * s;
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(prox_kv4 C, const int64_t* slots, int T, void* k_out,
                                                        void* v_out) {
  using T_ = typename Act<DT>::T;
  constexpr int LPR = D / 16;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % LPR;
  const int64_t row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / LPR;
  const bool is_v = blockIdx.y;
  if (row / C.heads >= T) return;
  const int t = (int)(row / C.heads), h = (int)(row % C.heads);
  const int64_t slot = slots[t];
  float a[8] = {}, b[8] = {};
  if (slot >= (int64_t)C.pages * C.page) {
    if (lane == 0) atomicOr(C.err, PROX_DEVERR_SLOT);
  } else if (slot >= 0) {
    const int64_t at = ((slot / C.page) * C.heads + h) * C.page + slot % C.page;
    const uint8_t* src = (is_v ? C.v : C.k) + at * (D / 2);
    const float s = __half2float(reinterpret_cast<const __half*>(is_v ? C.vs : C.ks)[at]);
    value8(*reinterpret_cast<const uint32_t*>(src + 4 * lane), s, a);
    value8(*reinterpret_cast<const uint32_t*>(src + D / 4 + 4 * lane), s, b);
  }
  T_* y = static_cast<T_*>(is_v ? v_out : k_out) + row * D;
  store_vals<DT, 8>(y + 8 * lane, true, a);
  store_vals<DT, 8>(y + D / 2 + 8 * lane, true, b);
}

cudaLaunchConfig_t rows_config(int64_t rows, int lanes, cudaStream_t s, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows * lanes + kThreads - 1) / kThreads), 2, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename F>
cudaError_t by_shape(int dtype, int D, F&& f) {
  auto with = [&](auto dt) -> cudaError_t {
    switch (D) {
      case 64: return f(dt, std::integral_constant<int, 64>());
      case 128: return f(dt, std::integral_constant<int, 128>());
      default: return f(dt, std::integral_constant<int, 256>());
    }
  };
  switch (dtype) {
    case PROX_F32: return with(std::integral_constant<int, PROX_F32>());
    case PROX_F16: return with(std::integral_constant<int, PROX_F16>());
    default: return with(std::integral_constant<int, PROX_BF16>());
  }
}

}  // namespace

cudaError_t launch_kv4_append(const prox_kv4* C, const void* k, const void* v, int64_t k_token, int64_t k_head,
                              int64_t v_token, int64_t v_head, const int64_t* slots, int T, int dtype,
                              cudaStream_t s) {
  // 16-byte loads where every row starts on 16 bytes
  const int per16 = dtype == PROX_F32 ? 4 : 8;
  const bool vec = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) == 0 &&
                   k_token % per16 == 0 && k_head % per16 == 0 && v_token % per16 == 0 && v_head % per16 == 0;
  return by_shape(dtype, C->D, [&](auto dt, auto d) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = rows_config((int64_t)T * C->heads, C->D / 16, s, attr);
    return cudaLaunchKernelEx(&cfg, append_kernel<decltype(dt)::value, decltype(d)::value>, *C, k, v, k_token, k_head,
                              v_token, v_head, slots, T, vec);
  });
}

cudaError_t launch_kv4_read(const prox_kv4* C, const int64_t* slots, int T, void* k, void* v, int dtype,
                            cudaStream_t s) {
  return by_shape(dtype, C->D, [&](auto dt, auto d) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = rows_config((int64_t)T * C->heads, C->D / 16, s, attr);
    return cudaLaunchKernelEx(&cfg, read_kernel<decltype(dt)::value, decltype(d)::value>, *C, slots, T, k, v);
  });
}

}  // namespace prox
