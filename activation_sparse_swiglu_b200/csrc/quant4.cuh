// Device-side helpers of the 4-bit operators (linear4.cu, kv4.cu, attend4.cu):
// activations in three types, codes widened to fp16, and the warp's tensor
// product on them.
//
// Codes are held as q + 8 in a nibble.  A nibble ORed into the mantissa of
// 1024.0 (0x6400) is the fp16 number 1024 + n, and 4 bits higher in that of 64.0
// (0x5400) it is 64 + n, so one fp16 subtraction gives the exact integer q for
// two codes at once.  |q| <= 8 is
// exact in fp16, products with fp16 operands are exact in the tensor core's
// fp32 sum, and the scales are applied to sums in fp32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "prox_device.cuh"

namespace prox {
namespace q4 {

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }

// (w & mask) | bits, as one instruction (left to the compiler it may become two).
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
  return r;
}

// The codes at nibbles 0 and 4 (SHIFTED = false) or 1 and 5 (true) of w, as
// two fp16 integers in [-8, 7].
template <bool SHIFTED>
__device__ __forceinline__ uint32_t widen(uint32_t w) {
  if (SHIFTED) {
    const uint32_t m = and_or(w, 0x00F000F0u, 0x54005400u);  // 64 + n
    return h2_bits(__hsub2(bits_h2(m), bits_h2(0x54805480u)));  // m - 72
  }
  const uint32_t m = and_or(w, 0x000F000Fu, 0x64006400u);  // 1024 + n
  return h2_bits(__hsub2(bits_h2(m), bits_h2(0x64086408u)));  // m - 1032
}

// The word's codes as four fp16 pairs: r[0] = nibbles (0, 4), r[1] = (1, 5),
// r[2] = (2, 6), r[3] = (3, 7).
__device__ __forceinline__ void widen8(uint32_t w, uint32_t (&r)[4]) {
  r[0] = widen<false>(w);
  r[1] = widen<true>(w);
  w >>= 8;
  r[2] = widen<false>(w);
  r[3] = widen<true>(w);
}

// D[16 x 8] += A[16 x 16] B[16 x 8], fp16 operands, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B + C.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// The transpose of an 8 x 8 matrix of 16-bit values held as fragments.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max that returns NaN when either side is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// ---- shared memory by 32-bit address -----------------------------------------
// (A generic pointer costs 64-bit additions and a conversion per access; these
// fold a constant into the instruction.)
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- activations: PROX_F32, PROX_F16 or PROX_BF16 --------------------------
template <int DT>
struct Act;
template <>
struct Act<PROX_F32> {
  using T = float;
  __device__ static float get(const float* p) { return *p; }
  __device__ static float from(float v) { return v; }
};
template <>
struct Act<PROX_F16> {
  using T = __half;
  __device__ static float get(const __half* p) { return __half2float(*p); }
  __device__ static __half from(float v) { return __float2half_rn(v); }
};
template <>
struct Act<PROX_BF16> {
  using T = __nv_bfloat16;
  __device__ static float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};

// N consecutive values as fp32 (N a multiple of 4); `vec`: p is aligned to
// min(16, N * sizeof(T)) bytes.
template <int DT, int N>
__device__ __forceinline__ void load_vals(const typename Act<DT>::T* p, bool vec, float (&v)[N]) {
  if (!vec) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = Act<DT>::get(p + i);
    return;
  }
  if constexpr (DT == PROX_F32) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + i);
      v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
    }
  } else {
    uint32_t w[N / 2];
    if constexpr (N % 8 == 0) {
#pragma unroll
      for (int i = 0; i < N / 8; ++i) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const uint2 u = reinterpret_cast<const uint2*>(p)[i];
        w[2 * i] = u.x, w[2 * i + 1] = u.y;
      }
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      float2 f;
      if constexpr (DT == PROX_F16)
        f = __half22float2(bits_h2(w[i]));
      else
        f = bf16x2_to_f2(w[i]);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}

// N consecutive values rounded once and stored (N a multiple of 4).
template <int DT, int N>
__device__ __forceinline__ void store_vals(typename Act<DT>::T* p, bool vec, const float (&v)[N]) {
  if (!vec) {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = Act<DT>::from(v[i]);
    return;
  }
  if constexpr (DT == PROX_F32) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (DT == PROX_F16) {
        w[i] = h2_bits(__floats2half2_rn(v[2 * i], v[2 * i + 1]));
      } else {
        __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&b);
      }
    }
    if constexpr (N % 8 == 0) {
#pragma unroll
      for (int i = 0; i < N / 8; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) reinterpret_cast<uint2*>(p)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
    }
  }
}

// The power of two that brings a largest magnitude mx into [2^14, 2^15): fp16
// then holds the hi part of everything that matters beside it, and a lo part
// down to 2^-39 of mx.  1 for zero, infinity and NaN.
__device__ __forceinline__ float normaliser(float mx) {
  const int e = (int)(__float_as_uint(mx) >> 23) & 255;
  if (mx == 0.f || e == 255) return 1.f;
  return __uint_as_float((uint32_t)min(253, 127 + 14 + 127 - e) << 23);
}
// 1 / f for a power of two f that normaliser() returns.
__device__ __forceinline__ float inv_pow2(float f) {
  return __uint_as_float((254u << 23) - __float_as_uint(f));
}

}  // namespace q4
}  // namespace prox
