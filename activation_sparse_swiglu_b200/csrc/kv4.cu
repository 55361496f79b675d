// The paged 4-bit cache's rows: quantised at their slots, and read back.
//
// One row is the D values of one token and head.  D / 16 lanes share a row,
// 16 values each as two runs of 8 (so that every load and store of the row is
// contiguous over its lanes): the largest magnitude by shuffles, the scale
// S = fp16(amax / 7), and the codes.
//
// The code of x is x / S rounded half to even, exactly.  The quotient q is
// corrected once by its exact remainder, so it is right where it is a number of
// 24 bits, ties n + 1/2 among them.  For 16-bit x nothing else can go wrong: x / S
// off a tie is off it by 2^-12 at least (both are integers of 11 bits times
// powers of two).  For fp32 x a quotient next to a tie may have been rounded
// onto it: e = x - n S, exact in one fused multiply-add, then exceeds S / 2.
// Adding 1.5 2^23 + 8 rounds q and leaves the code in the low bits.
//
// Bound: HBM for prompts (16000 tokens x 8 heads of 128: 65 MB in, 17 MB out),
// with issue close behind; launch latency for the rows of a decode step.
#include <type_traits>

#include "decode4.h"
#include "quant4.cuh"

namespace prox {
namespace {

using namespace q4;

constexpr int kThreads = 256;

// Eight codes of x under a scale s whose quotients all lie within 7.5.
template <int DT>
__device__ __forceinline__ uint32_t code8(const float (&x)[8], float s, float rs, float half) {
  constexpr float kMagic = 12582912.f + 8.f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float q0 = x[i] * rs;
    const float q = fmaf(fmaf(-q0, s, x[i]), rs, q0);
    float t = q + kMagic;
    if (DT == PROX_F32) {
      const float e = fmaf(-(t - kMagic), s, x[i]);
      if (fabsf(e) > half) t += copysignf(1.f, e);
    }
    w = w * 16 + (__float_as_uint(t) & 15u);
  }
  return w;
}
// The same for any scale: 0 (codes 0), infinite or NaN (codes 0; the row reads
// as NaN), and fp16's subnormals, whose coarse steps leave quotients past 7.
__device__ uint32_t code8_any(const float (&x)[8], float s) {
  uint32_t w = 0;
  for (int i = 7; i >= 0; --i) {
    int n = 0;
    if (s > 0.f && s <= 65504.f) {
      const float q = x[i] / s;
      n = (int)rintf(q);
      const float e = fmaf(-(float)n, s, x[i]);
      if (fabsf(e) > 0.5f * s) n += e > 0.f ? 1 : -1;
      n = min(7, max(-7, n));
    }
    w = w * 16 + (uint32_t)(n + 8);
  }
  return w;
}

// One row quantised into slot row `at` of codes and scales, by its LPR lanes.
template <int DT, int D>
__device__ __forceinline__ void put_row(const float (&a)[8], const float (&b)[8], int lane, unsigned mask,
                                        uint8_t* codes, uint16_t* scales, int64_t at) {
  constexpr int LPR = D / 16;
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = max_nan(mx, max_nan(fabsf(a[i]), fabsf(b[i])));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(mask, mx, o));
  const __half sh = __float2half_rn(mx / 7.0f);
  const float s = __half2float(sh);
  uint32_t ca, cb;
  if (s >= 0x1p-14f && s <= 65504.f) {
    const float rs = 1.0f / s, half = 0.5f * s;
    ca = code8<DT>(a, s, rs, half);
    cb = code8<DT>(b, s, rs, half);
  } else {
    ca = code8_any(a, s);
    cb = code8_any(b, s);
  }
  uint8_t* dst = codes + at * (D / 2) + 4 * lane;
  *reinterpret_cast<uint32_t*>(dst) = ca;
  *reinterpret_cast<uint32_t*>(dst + D / 4) = cb;
  if (lane == 0) reinterpret_cast<__half*>(scales)[at] = sh;
}

// Each group of lanes takes a row of K and the same of V: one slot, one place.
template <int DT, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(prox_kv4 C, const void* k_in, const void* v_in,
                                                          int64_t k_token, int64_t k_head, int64_t v_token,
                                                          int64_t v_head, const int64_t* slots, int T, int shift,
                                                          bool vec) {
  using T_ = typename Act<DT>::T;
  constexpr int LPR = D / 16;  // lanes of one row
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % LPR;
  const unsigned row = (unsigned)(((int64_t)blockIdx.x * kThreads + threadIdx.x) / LPR);
  const unsigned t = row / (unsigned)C.heads, h = row - t * C.heads;
  if (t >= (unsigned)T) return;  // a whole row's lanes leave together
  const int64_t slot = slots[t];
  const T_* k = static_cast<const T_*>(k_in) + (int64_t)t * k_token + (int64_t)h * k_head + 8 * lane;
  const T_* v = static_cast<const T_*>(v_in) + (int64_t)t * v_token + (int64_t)h * v_head + 8 * lane;
  float ka[8], kb[8], va[8], vb[8];
  if (slot < 0) return;
  if (slot >= (int64_t)C.pages * C.page) {
    if (lane == 0) atomicOr(C.err, PROX_DEVERR_SLOT);
    return;
  }
  load_vals<DT, 8>(k, vec, ka);
  load_vals<DT, 8>(k + D / 2, vec, kb);
  load_vals<DT, 8>(v, vec, va);
  load_vals<DT, 8>(v + D / 2, vec, vb);
  const unsigned mask = ((1u << LPR) - 1) << ((threadIdx.x & 31) / LPR * LPR);
  const int64_t at = (((slot >> shift) * C.heads + h) << shift) + (slot & (C.page - 1));
  put_row<DT, D>(ka, kb, lane, mask, C.k, C.ks, at);
  put_row<DT, D>(va, vb, lane, mask, C.v, C.vs, at);
}

// The eight values of a word under scale s, rounded once and stored.  (A code
// times an fp16 scale has 15 significant bits: one rounding in any type.)
template <int DT>
__device__ __forceinline__ void store8(typename Act<DT>::T* y, uint32_t w, __half s) {
  uint32_t r[4];  // nibbles (0, 4), (1, 5), (2, 6), (3, 7)
  widen8(w, r);
  if constexpr (DT == PROX_F16) {
    const __half2 s2 = __half2half2(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = h2_bits(__hmul2(bits_h2(r[i]), s2));
    *reinterpret_cast<uint4*>(y) =
        make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410), __byte_perm(r[0], r[1], 0x7632),
                   __byte_perm(r[2], r[3], 0x7632));
  } else {
    const float f = __half2float(s);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = __half22float2(bits_h2(r[i]));
      v[i] = q.x * f, v[4 + i] = q.y * f;
    }
    store_vals<DT, 8>(y, true, v);
  }
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(prox_kv4 C, const int64_t* slots, int T, int shift,
                                                        void* k_out, void* v_out) {
  using T_ = typename Act<DT>::T;
  constexpr int LPR = D / 16;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % LPR;
  const unsigned row = (unsigned)(((int64_t)blockIdx.x * kThreads + threadIdx.x) / LPR);
  const unsigned t = row / (unsigned)C.heads, h = row - t * C.heads;
  if (t >= (unsigned)T) return;
  const int64_t slot = slots[t];
  uint32_t w[4] = {0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
  __half ks = __half(0.f), vs = __half(0.f);
  if (slot >= (int64_t)C.pages * C.page) {
    if (lane == 0) atomicOr(C.err, PROX_DEVERR_SLOT);
  } else if (slot >= 0) {
    const int64_t at = (((slot >> shift) * C.heads + h) << shift) + (slot & (C.page - 1));
    const uint8_t* k = C.k + at * (D / 2) + 4 * lane;
    const uint8_t* v = C.v + at * (D / 2) + 4 * lane;
    ks = reinterpret_cast<const __half*>(C.ks)[at];
    vs = reinterpret_cast<const __half*>(C.vs)[at];
    w[0] = *reinterpret_cast<const uint32_t*>(k);
    w[1] = *reinterpret_cast<const uint32_t*>(k + D / 4);
    w[2] = *reinterpret_cast<const uint32_t*>(v);
    w[3] = *reinterpret_cast<const uint32_t*>(v + D / 4);
  }
  T_* ko = static_cast<T_*>(k_out) + (int64_t)row * D + 8 * lane;
  T_* vo = static_cast<T_*>(v_out) + (int64_t)row * D + 8 * lane;
  store8<DT>(ko, w[0], ks);
  store8<DT>(ko + D / 2, w[1], ks);
  store8<DT>(vo, w[2], vs);
  store8<DT>(vo + D / 2, w[3], vs);
}

int shift_of(int page) {
  int s = 0;
  while ((1 << s) < page) ++s;
  return s;
}

cudaLaunchConfig_t rows_config(int64_t rows, int lanes, cudaStream_t s, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows * lanes + kThreads - 1) / kThreads), 1, 1);
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
                              v_token, v_head, slots, T, shift_of(C->page), vec);
  });
}

cudaError_t launch_kv4_read(const prox_kv4* C, const int64_t* slots, int T, void* k, void* v, int dtype,
                            cudaStream_t s) {
  return by_shape(dtype, C->D, [&](auto dt, auto d) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = rows_config((int64_t)T * C->heads, C->D / 16, s, attr);
    return cudaLaunchKernelEx(&cfg, read_kernel<decltype(dt)::value, decltype(d)::value>, *C, slots, T,
                              shift_of(C->page), k, v);
  });
}

}  // namespace prox
