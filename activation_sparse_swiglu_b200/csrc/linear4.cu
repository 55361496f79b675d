// y = x W for 1..16 tokens, W [K, N] held as INT4 codes with one fp16 scale
// per group of 128 input rows and channel:
//   y[b, n] = sum_g S[g, n] sum_{k in g} q[k, n] x[b, k],   q = code - 8.
//
// The product runs on the tensor cores with the channels as the M dimension
// (A = the codes, 16 channels x 16 input rows) and the tokens as N = 8 columns
// (B = x from shared memory), because at N = 8 the fragment of a code word
// feeds one instruction whatever the batch: the codes, which are all of the
// traffic, are decoded once.  Codes are stored in fragment order, so a lane's 8
// words of a 16 x 128 unit are two 16-byte loads of a stretch that the warp
// reads contiguously, and no shuffle or shared memory stands between HBM and
// the tensor core.
//
// Codes are widened to exact fp16 integers q, 9 instructions for 8 of them
// (decode_words), so that every product is exact and a sum is as good as the
// tensor core's fp32, whatever the inputs' spread.  (For 16-bit inputs a code
// masked out of its word, an fp16 subnormal, would do with 5: but the tensor
// core aligns products by the exponents of their factors, a subnormal's being
// that of the largest one, so an input 10^4 times the others took the others'
// last bits even where its own codes are 0, by percents of a group's sum.  With
// subnormals 28672 x 8192 takes 26.6 us for 5 tokens, 5120 x 131072 76.5 for 16;
// with integers 28.8 and 82.6.)
//
// x is held in fp16, scaled by a power of two per token and group of 128 that
// brings the group's largest magnitude to 2^14: fp16 and bf16 values keep all
// their bits down to 2^-25 of that (below it, an absolute 2^-38), fp32 values
// are split into hi + lo columns (22 significant bits).  A unit's sum over its
// 128 rows is taken by the tensor core in fp32, then scaled and added in fp32,
// so no sum is held in fewer bits and the tensor core's running sum is never
// longer than 8 instructions.
//
// Split: the unit is one group of 128 input rows of a strip of 32 channels
// (2 KB; two tiles, so that a fragment of x read from shared memory serves
// two products).  The units of a cluster's strips are dealt to a CTA's warps as
// equal contiguous ranges; a strip that several warps share is joined through
// shared memory in warp order, and the CTAs of a cluster (which split K when
// there are too few channels to fill the device) join theirs through
// distributed shared memory in rank order, so results do not depend on timing
// and no scratch in global memory is shared between calls.
//
// Bound: HBM at large sizes (0.52 bytes per weight; 5120 x 131072 at one token
// 58 us, 0.91 of the copy bandwidth), issue and the tensor pipe from 9 tokens on
// (two column tiles: 82.6 us at 16), launch and one pass of load latency at small
// ones (4096 x 6144 at one token 5.8 us).
#include "decode4.h"
#include "quant4.cuh"

namespace prox {
namespace {

using namespace q4;

// Warps of a CTA: as many as the registers of NT column tiles allow.
constexpr int warps_of(int nt) { return nt == 1 ? 16 : nt == 2 ? 12 : 8; }
constexpr int kStrip = 32;                // channels of a strip
constexpr int kPartRow = 36;              // floats of a token's results of a strip (bank-conflict-free)
constexpr int kXPad = 64;                 // bytes; makes 16-byte reads of 8 columns conflict-free
constexpr int kCodeBytes = kStrip * 64;   // codes of a unit
constexpr int kScaleBytes = kStrip * 2;   // its scales
constexpr int kSlotBytes = kCodeBytes + 256;  // in a ring: codes, and per lane its four scales
constexpr int kSmemLimit = 227 * 1024 - 128;  // (a table of the warps beside it)

struct LinearArgs {
  const char* codes;
  const char* scales;
  const void* x;
  int64_t x_stride;
  void* out;
  int64_t out_stride;
  int B, N, G;
  int strips;
  int per_clus;    // strips of a cluster
  int per_rank;    // groups of a CTA of the cluster
  int per_phase;   // groups whose x is in shared memory at once
  int cluster;
  int ring_at;     // offset of the warps' rings in shared memory
  int x_vec;       // x allows 16-byte loads
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The value at p (this CTA's shared memory) in the cluster's CTA `rank`.
__device__ __forceinline__ float ld_peer(const float* p, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// 0, known only once v is.
__device__ __forceinline__ uint32_t after(uint32_t v) {
  uint32_t r;
  asm volatile("and.b32 %0, %1, 0;" : "=r"(r) : "r"(v));
  return r;
}

// Start of the w-th of W equal contiguous ranges of U units.
// (A CTA has at most 2^15 strips x 2^9 groups and 16 warps: 32 bits hold it.)
__device__ __forceinline__ int range_at(int U, int w, int W) { return (int)((unsigned)U * (unsigned)w / (unsigned)W); }
// The range that holds unit u.
__device__ __forceinline__ int range_of(int U, int u, int W) {
  return (int)(((unsigned)(u + 1) * (unsigned)W - 1) / (unsigned)U);
}

// A word holds eight codes, two of each of four fields (one per 16-bit half):
// A in bits 6-9, B in 2-5, C in 10-13, and D in 14-15 with its upper two bits
// in bits 0-1 of the other half, so that a rotation by 8 brings D to 6-9 and C
// to 2-5.  r: A fragments in the order a0 (B), a1 (C), a2 (A), a3 (D), as
// integers q: in the mantissas of 256 and of 16 the fields are 256 + n and
// 16 + n.  (Without the fused and_or 28672 x 8192 took 34.6 us at 5 tokens
// instead of 28.8.)
__device__ __forceinline__ void decode_words(uint32_t w, uint32_t (&r)[4]) {
  const uint32_t rot = __funnelshift_r(w, w, 8);
  const __half2 low = bits_h2(0xDC20DC20u), high = bits_h2(0xCE00CE00u);  // -264, -24
  r[2] = h2_bits(__hadd2(bits_h2(and_or(w, 0x03C003C0u, 0x4C004C00u)), high));
  r[3] = h2_bits(__hadd2(bits_h2(and_or(rot, 0x03C003C0u, 0x4C004C00u)), high));
  r[0] = h2_bits(__hadd2(bits_h2(and_or(w, 0x003C003Cu, 0x5C005C00u)), low));
  r[1] = h2_bits(__hadd2(bits_h2(and_or(rot, 0x003C003Cu, 0x5C005C00u)), low));
}

// The largest magnitude of 16 bytes of activations.
template <int DT>
__device__ __forceinline__ float top(const uint4& u) {
  if constexpr (DT == PROX_F16) {
    const __half2 m = __hmax2(__hmax2(__habs2(bits_h2(u.x)), __habs2(bits_h2(u.y))),
                              __hmax2(__habs2(bits_h2(u.z)), __habs2(bits_h2(u.w))));
    return __half2float(__hmax(__low2half(m), __high2half(m)));
  } else if constexpr (DT == PROX_BF16) {
    const float2 a = bf16x2_to_f2(u.x), b = bf16x2_to_f2(u.y), c = bf16x2_to_f2(u.z), d = bf16x2_to_f2(u.w);
    return fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))),
                 fmaxf(fmaxf(fabsf(c.x), fabsf(c.y)), fmaxf(fabsf(d.x), fabsf(d.y))));
  } else {
    return fmaxf(fmaxf(fabsf(__uint_as_float(u.x)), fabsf(__uint_as_float(u.y))),
                 fmaxf(fabsf(__uint_as_float(u.z)), fabsf(__uint_as_float(u.w))));
  }
}
// Two fp16 or bf16 values times a power of two f, as fp16 (exact above 2^-14).
template <int DT>
__device__ __forceinline__ uint32_t scale2(uint32_t w, float f) {
  const float2 v = DT == PROX_F16 ? __half22float2(bits_h2(w)) : bf16x2_to_f2(w);
  return h2_bits(__floats2half2_rn(v.x * f, v.y * f));
}

// NT column tiles of 8 (tokens, or their hi / lo parts), PF units in flight
// per warp.
template <int DT, int NT, int PF>
__global__ void __launch_bounds__(warps_of(NT) * 32, 1) linear4_kernel(const LinearArgs a) {
  using T = typename Act<DT>::T;
  constexpr int kWarps = warps_of(NT), kThreads = kWarps * 32;
  constexpr int PARTS = DT == PROX_F32 ? 2 : 1;
  constexpr int NC = 2 / PARTS;       // tokens of a thread per column tile
  constexpr int TB = 8 * NT / PARTS;  // tokens
  extern __shared__ __align__(16) char smem[];
  __shared__ int2 s_cut[kWarps];  // of warps 0 .. W - 2; the last entry: a bit for each that is cut
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
  const int clus = (int)blockIdx.x / a.cluster;
  const int s0 = min(clus * a.per_clus, a.strips), s1 = min(s0 + a.per_clus, a.strips);
  const int g0 = min(rank * a.per_rank, a.G), g1 = min(g0 + a.per_rank, a.G);
  const int cols = a.B * PARTS;
  const int xs = a.per_phase * 256 + kXPad;  // bytes of a column
  char* s_x = smem;
  float* s_nf = reinterpret_cast<float*>(smem + (size_t)cols * xs);          // [per_phase][TB] 1 / the powers of two
  float* s_res = reinterpret_cast<float*>(s_nf + a.per_phase * TB);          // [per_clus][B][kPartRow]
  // the warp's ring of PF units: this lane's 16 bytes of each row of codes, and
  // its scales
  char* ring_base = smem + a.ring_at;
  const uint32_t ring = smem_u32(ring_base) + warp * (PF * kSlotBytes) + lane * 16;
  const bool use_res = a.cluster > 1 || a.per_phase < a.per_rank;
  T* out = static_cast<T*>(a.out);

  // A warp's results of the strip it is at, and its part of a strip that began
  // in the warp before (few enough to stay in registers).
  float acc[2][NT][2][NC], head_acc[2][NT][2][NC];
  auto each = [&](const float(&v)[2][NT][2][NC], auto&& f) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < NC; ++e) {
            const int b = PARTS == 2 ? 4 * n + t : 8 * n + 2 * t + e;
            if (b < a.B) f(16 * m + 8 * r + g, b, v[m][n][r][e]);
          }
  };
  auto put = [&](int strip, int row, int b, float v) {
    const int n = strip * kStrip + row;
    if (n < a.N) out[b * a.out_stride + n] = Act<DT>::from(v);
  };
  // The parts that a warp leaves of strips it shares: in its ring, idle by then.
  static_assert(PF >= 2 && kLinear4MaxTokens * kPartRow * 4 <= kSlotBytes, "a ring holds two parts");
  auto head = [&](int w) { return reinterpret_cast<float*>(ring_base + (size_t)w * (PF * kSlotBytes)); };
  auto tail = [&](int w) { return reinterpret_cast<float*>(ring_base + (size_t)w * (PF * kSlotBytes) + kSlotBytes); };

  const int phases = max(1, (a.per_rank + a.per_phase - 1) / a.per_phase);
  for (int ph = 0; ph < phases; ++ph) {
    const int pg0 = min(g0 + ph * a.per_phase, g1), pg1 = min(pg0 + a.per_phase, g1);
    const int nG = pg1 - pg0, U = (s1 - s0) * nG;
    const int W = min(U, kWarps);
    const int beg = warp < W ? range_at(U, warp, W) : U, end = warp < W ? range_at(U, warp + 1, W) : U;
    if (ph > 0) __syncthreads();  // x and the parts of the phase before have been read
    if (warp == 0) {
      // the strip that starts in warp w0's range and goes on past it, and the
      // warp that it ends in
      bool cut = false;
      if (lane < W - 1) {
        const int from = range_at(U, lane + 1, W), s = from / nG;
        cut = from != s * nG && range_at(U, lane, W) <= s * nG;
        if (cut) s_cut[lane] = make_int2(s, range_of(U, s * nG + nG - 1, W));
      }
      const unsigned cuts = __ballot_sync(0xffffffffu, cut);
      if (lane == 0) s_cut[kWarps - 1].x = (int)cuts;
    }

    // Every lane copies the very bytes it will read, so its own wait is all the
    // synchronisation there is.  A strip's units are consecutive, and so are
    // the strips where the CTA has all groups.
    int strip = nG ? s0 + beg / nG : 0, gr0 = nG ? beg % nG : 0;
    int lg = gr0;  // the next unit to load
    const char* lp = a.codes + ((size_t)strip * a.G + pg0 + lg) * kCodeBytes + lane * 16;
    const char* lsp = a.scales + ((size_t)strip * a.G + pg0 + lg) * kScaleBytes + g * 8;
    int left = end - beg;
    auto load = [&](uint32_t slot) {
      if (left > 0) {
        --left;
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async16(slot + 512 * i, lp + 512 * i);
        cp_async8(slot - lane * 8 + kCodeBytes, lsp);
        lp += kCodeBytes;
        lsp += kScaleBytes;
        if (++lg == nG) {
          lg = 0;
          lp += (size_t)(a.G - nG) * kCodeBytes;
          lsp += (size_t)(a.G - nG) * kScaleBytes;
        }
      }
      cp_async_commit();
    };
    // The weights do not depend on the kernel before this one in the stream.
#pragma unroll
    for (int j = 0; j < PF; ++j) load(ring + j * kSlotBytes);
    if (ph == 0) {
      pdl_wait();
      pdl_trigger();
    }

    // x of this phase's groups into columns.  A lane takes 64 bytes of a group
    // (four pieces, in an order that spreads the stores over the banks), LPG
    // lanes a group, a warp 32 / LPG groups of a token.
    constexpr int LPG = DT == PROX_F32 ? 8 : 4, GPW = 32 / LPG;
    const int runs = (nG + GPW - 1) / GPW;
    const int turn = DT == PROX_F32 ? (lane >> 2) & 3 : (lane >> 1) & 3;
    struct Item {
      int b, run;
      uint4 raw[4];
    };
    auto settle = [&](Item& it) {
      while (it.run >= runs && it.b < a.B) it.run -= runs, ++it.b;
    };
    auto fetch = [&](Item& it) {
      const int gr = it.run * GPW + lane / LPG;
#pragma unroll
      for (int j = 0; j < 4; ++j) it.raw[j] = make_uint4(0, 0, 0, 0);
      if (it.b >= a.B || gr >= nG) return;
      const T* src = static_cast<const T*>(a.x) + it.b * a.x_stride + (int64_t)(pg0 + gr) * kGroupRows +
                     (lane % LPG) * (64 / (int)sizeof(T));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const T* p = src + ((j + turn) & 3) * (16 / (int)sizeof(T));
        if (a.x_vec) {
          it.raw[j] = *reinterpret_cast<const uint4*>(p);
        } else {
          T v[16 / sizeof(T)];
#pragma unroll
          for (int i = 0; i < (int)(16 / sizeof(T)); ++i) v[i] = p[i];
          memcpy(&it.raw[j], v, 16);
        }
      }
    };
    // the loads of two items are in flight while a third is converted
    Item ahead[2];
    ahead[0].b = runs > 0 ? 0 : a.B;
    ahead[0].run = warp;
    settle(ahead[0]);
    fetch(ahead[0]);
    ahead[1].b = ahead[0].b;
    ahead[1].run = ahead[0].run + kWarps;
    settle(ahead[1]);
    fetch(ahead[1]);
    while (ahead[0].b < a.B) {
      const Item now = ahead[0];
      ahead[0] = ahead[1];
      ahead[1].run += kWarps;
      settle(ahead[1]);
      fetch(ahead[1]);
      const int b = now.b, gr = now.run * GPW + lane / LPG;
      const uint4(&raw)[4] = now.raw;
      float mx = fmaxf(fmaxf(top<DT>(raw[0]), top<DT>(raw[1])), fmaxf(top<DT>(raw[2]), top<DT>(raw[3])));
#pragma unroll
      for (int o = LPG / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      if (gr >= nG) continue;
      const float f = normaliser(mx);
      char* col = s_x + (size_t)(b * PARTS) * xs + gr * 256 + (lane % LPG) * (DT == PROX_F32 ? 32 : 64);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int piece = (j + turn) & 3;
        if constexpr (DT == PROX_F32) {
          const float y[4] = {__uint_as_float(raw[j].x) * f, __uint_as_float(raw[j].y) * f,
                              __uint_as_float(raw[j].z) * f, __uint_as_float(raw[j].w) * f};
          const __half2 h0 = __floats2half2_rn(y[0], y[1]), h1 = __floats2half2_rn(y[2], y[3]);
          const float2 b0 = __half22float2(h0), b1 = __half22float2(h1);
          *reinterpret_cast<uint2*>(col + 8 * piece) = make_uint2(h2_bits(h0), h2_bits(h1));
          const __half2 l0 = __floats2half2_rn(y[0] - b0.x, y[1] - b0.y), l1 = __floats2half2_rn(y[2] - b1.x, y[3] - b1.y);
          *reinterpret_cast<uint2*>(col + xs + 8 * piece) = make_uint2(h2_bits(l0), h2_bits(l1));
        } else {
          *reinterpret_cast<uint4*>(col + 16 * piece) =
              make_uint4(scale2<DT>(raw[j].x, f), scale2<DT>(raw[j].y, f), scale2<DT>(raw[j].z, f),
                         scale2<DT>(raw[j].w, f));
        }
      }
      if (lane % LPG == 0) s_nf[gr * TB + b] = inv_pow2(f);
    }
    __syncthreads();

    // this lane's column of x in each tile (columns past the batch repeat the
    // last one; their results are not used)
    uint32_t xcol[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xcol[n] = smem_u32(s_x) + min(8 * n + g, cols - 1) * xs + 16 * t;
    const uint32_t nf0 = smem_u32(s_nf + NC * t);

    uint32_t slot = ring;
    bool has_head = false, has_tail = false;
    for (int u = beg; u < end;) {
      const int n_units = min(nG - gr0, end - u);  // of this strip
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < NC; ++e) acc[m][n][r][e] = 0.f;
      uint32_t xa[NT], nf = nf0 + gr0 * (TB * 4);
#pragma unroll
      for (int n = 0; n < NT; ++n) xa[n] = xcol[n] + gr0 * 256;
      for (int i_unit = 0; i_unit < n_units; ++i_unit) {
        cp_async_wait<PF - 1>();
        uint4 w[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) w[m][h] = lds128(slot + (2 * m + h) * 512);
        const uint2 scw = lds64(slot - lane * 8 + kCodeBytes);
        float inv[NT][NC];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (PARTS == 2) {
            inv[n][0] = __uint_as_float(lds32(nf + 16 * n));
          } else {
            const uint2 f = lds64(nf + 32 * n);
            inv[n][0] = __uint_as_float(f.x), inv[n][NC - 1] = __uint_as_float(f.y);
          }
        }
        // the copy into the slot just read starts once the reads (which come
        // back in order) are here
        load(slot + after(scw.y));
        slot = slot == ring + (PF - 1) * kSlotBytes ? ring : slot + kSlotBytes;
        float d[2][NT][4];
        uint4 xq[4][NT];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n) xq[i][n] = lds128(xa[n] + i * 64);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4(&xv)[NT] = xq[i];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint4 w4 = w[m][i >> 1];
            uint32_t r[4];
            decode_words((i & 1) ? w4.z : w4.x, r);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (i == 0)
                mma_f16(d[m][n], r[0], r[1], r[2], r[3], xv[n].x, xv[n].y, 0.f, 0.f, 0.f, 0.f);
              else
                mma_f16(d[m][n], r[0], r[1], r[2], r[3], xv[n].x, xv[n].y);
            }
            decode_words((i & 1) ? w4.w : w4.y, r);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(d[m][n], r[0], r[1], r[2], r[3], xv[n].z, xv[n].w);
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float2 s2 = __half22float2(bits_h2(m ? scw.y : scw.x));
          const float s[2] = {s2.x, s2.y};
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int e = 0; e < NC; ++e) {
                const float z = PARTS == 2 ? d[m][n][2 * r] + d[m][n][2 * r + 1] : d[m][n][2 * r + e];
                acc[m][n][r][e] = fmaf(z * s[r], inv[n][e], acc[m][n][r][e]);
              }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) xa[n] += 256;
        nf += TB * 4;
      }
      // the strip's results, or this warp's part of them
      if (n_units == nG) {
        if (!use_res)
          each(acc, [&](int row, int b, float v) { put(strip, row, b, v); });
        else
          each(acc, [&](int row, int b, float v) {
            float* r = s_res + ((strip - s0) * a.B + b) * kPartRow + row;
            *r = ph == 0 ? v : *r + v;
          });
      } else if (gr0 > 0) {
        has_head = true;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int e = 0; e < NC; ++e) head_acc[m][n][r][e] = acc[m][n][r][e];
      } else {
        has_tail = true;  // the range ends here
      }
      u += n_units;
      gr0 = 0;
      ++strip;
    }
    cp_async_wait<0>();
    __syncwarp();
    if (has_head) each(head_acc, [&, p = head(warp)](int row, int b, float v) { p[b * kPartRow + row] = v; });
    if (has_tail) each(acc, [&, p = tail(warp)](int row, int b, float v) { p[b * kPartRow + row] = v; });
    __syncthreads();
    // strips that several warps share, in warp order: the strip at the start of
    // warp w's range, where w is the second to have a part of it; neighbouring
    // threads take neighbouring channels of one token
    for (unsigned cuts = s_cut[kWarps - 1].x; cuts; cuts &= cuts - 1) {
      const int w0 = __ffs(cuts) - 1, s = s_cut[w0].x, wb = s_cut[w0].y;  // w = w0 + 1
      for (int e = threadIdx.x; e < kStrip * a.B; e += kThreads) {
        const int row = e % kStrip, b = e / kStrip;
        float v = tail(w0)[b * kPartRow + row];
        const float* h = head(w0 + 1) + b * kPartRow + row;
#pragma unroll 4
        for (int w = w0 + 1; w <= wb; ++w, h += PF * kSlotBytes / 4) v += *h;
        if (use_res) {
          float* r = s_res + (s * a.B + b) * kPartRow + row;
          *r = ph == 0 ? v : *r + v;
        } else {
          put(s0 + s, row, b, v);
        }
      }
    }
  }
  if (!use_res) return;
  if (a.cluster > 1)
    cluster_sync_all();
  else
    __syncthreads();
  // the cluster's CTAs share out the results; ranks are added in order (a rank
  // without groups holds none)
  const int ranks = min(a.cluster, (a.G + a.per_rank - 1) / a.per_rank);
  for (int e = rank * kThreads + threadIdx.x; e < (s1 - s0) * kStrip * a.B; e += a.cluster * kThreads) {
    const int row = e % kStrip, q = e / kStrip, s = q / a.B, b = q - s * a.B;
    const float* p = s_res + q * kPartRow + row;
    float part[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) part[r] = r >= ranks ? 0.f : a.cluster > 1 ? ld_peer(p, r) : *p;
    float v = part[0];
#pragma unroll
    for (int r = 1; r < 8; ++r) v += part[r];
    put(s0 + s, row, b, v);
  }
  if (a.cluster > 1) cluster_sync_all();  // no CTA leaves while its results are read
}

// codes [strips][G][4][32 lanes][4 words]: row h of tile m (index 2 m + h) holds
// the steps 2h and 2h + 1 of 32 input rows; a word's fields: see decode_words.  scales [strips][G][8][tile][2].  Channels past N hold code 8 and
// scale 0.
__global__ void linear4_pack_kernel(const uint8_t* __restrict__ codes, const __half* __restrict__ scales, int N, int G,
                                    int strips, uint32_t* __restrict__ out, __half* __restrict__ out_scales) {
  const size_t n_word = (size_t)strips * G * (kCodeBytes / 4), n_scale = (size_t)strips * G * kStrip;
  const size_t stride = (size_t)gridDim.x * blockDim.x;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n_word + n_scale; i += stride) {
    if (i < n_word) {
      const int wi = i & 3, l = (i >> 2) & 31, h = (i >> 7) & 1, m = (i >> 8) & 1;
      const size_t unit = i >> 9;
      const int gr = unit % G, strip = unit / G;
      const int k0 = gr * kGroupRows + 32 * (2 * h + (wi >> 1)) + 8 * (l & 3) + 4 * (wi & 1);
      uint32_t w = 0;
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        // fields B, C, A, D of the low half, then of the high: C and D belong to
        // row + 8, A and D to input rows k0 + 2 and k0 + 3
        const int field = f & 3, high = f >> 2;
        const int n = strip * kStrip + 16 * m + (l >> 2) + ((field & 1) ? 8 : 0);
        const int k = k0 + (field >= 2 ? 2 : 0) + high;
        const uint32_t c = n < N ? (codes[(size_t)k * (N / 2) + n / 2] >> (4 * (n & 1))) & 15u : 8u;
        if (field == 3)
          w |= high ? (c & 3) << 30 | c >> 2 : (c & 3) << 14 | (c >> 2) << 16;
        else
          w |= c << ((field == 0 ? 2 : field == 1 ? 10 : 6) + 16 * high);
      }
      out[i] = w;
    } else {
      const size_t u = i - n_word;
      const int r = u & 1, m = (u >> 1) & 1, gq = (u >> 2) & 7;
      const size_t unit = u >> 5;
      const int gr = unit % G, strip = unit / G;
      const int n = strip * kStrip + 16 * m + 8 * r + gq;
      out_scales[u] = n < N ? scales[(size_t)gr * N + n] : __half(0.f);
    }
  }
}

using Kernel = void (*)(const LinearArgs);

// Column tiles for the batch: 8 columns each, one per token (two for fp32).
int col_tiles(int B, int dtype) {
  const int cols = dtype == PROX_F32 ? 2 * B : B;
  return cols <= 8 ? 1 : cols <= 16 ? 2 : 4;
}

// Units in flight per warp: 4 cover a small matrix's whole share at once; 3 or
// 2 where x takes the room.  (With one, 16 tokens x 5120 ran at HBM's latency:
// 83 us for 131072 channels, when two or three took 76.5.)
template <int PF>
Kernel pick_depth(int dtype, int nt) {
  switch (dtype) {
    case PROX_F32:
      return nt == 1 ? linear4_kernel<PROX_F32, 1, PF>
                     : nt == 2 ? linear4_kernel<PROX_F32, 2, PF> : linear4_kernel<PROX_F32, 4, PF>;
    case PROX_F16: return nt == 1 ? linear4_kernel<PROX_F16, 1, PF> : linear4_kernel<PROX_F16, 2, PF>;
    default: return nt == 1 ? linear4_kernel<PROX_BF16, 1, PF> : linear4_kernel<PROX_BF16, 2, PF>;
  }
}
Kernel pick(int dtype, int nt, int depth) {
  return depth == 4 ? pick_depth<4>(dtype, nt) : depth == 3 ? pick_depth<3>(dtype, nt) : pick_depth<2>(dtype, nt);
}

struct Plan {
  int cluster, per_clus, per_rank, per_phase, clusters, depth;
  size_t ring_at, smem;
};

size_t ring_bytes(int nt, int depth) { return (size_t)warps_of(nt) * depth * kSlotBytes; }

// The cluster size whose busiest CTA has the least to do: its units (2 KB of
// codes each, about 90 SM cycles at the copy bandwidth), plus what converting x
// costs (15 cycles per column and group), plus what a launch in clusters and
// the join across them costs, plus 30 per extra phase of x (the rings run dry).
// Measured for bf16 tokens, clusters of 1 / 2 / 4 / 8: at 4096 x 4096 one token
// 4.4 / 5.7 / 6.2 / 8.5 us, 16 tokens 8.3 / 8.5 / 8.7 / 10.6; at 8192 x 1024 5.0 /
// 4.7 / 5.2 / 5.8 and 15.8 / 8.8 / 7.0 / 7.3; at 28672 x 8192 with 16 tokens 87 /
// 62 / 49 / 44 (16 fp32 tokens: 174 / 114 / 79 / 75).
constexpr double kJoin[4] = {0, 35, 45, 75};

bool plan_linear4(const prox_linear4* L, int strips, int B, int dtype, Plan* best) {
  const int nt = col_tiles(B, dtype), parts = dtype == PROX_F32 ? 2 : 1;
  const int cols = B * parts, tb = 8 * nt / parts;
  double least = 1e300;
  for (int ci = 0; ci < 4; ++ci) {
    const int c = 1 << ci;
    if (L->clusters[ci] < 1 || (c > 1 && c > L->G)) continue;
    Plan p;
    p.cluster = c;
    p.clusters = strips < L->clusters[ci] ? strips : L->clusters[ci];
    p.per_clus = (strips + p.clusters - 1) / p.clusters;
    p.clusters = (strips + p.per_clus - 1) / p.per_clus;
    p.per_rank = (L->G + c - 1) / c;
    p.per_phase = p.per_rank;
    auto front = [&] {  // everything before the rings
      const int res = c > 1 || p.per_phase < p.per_rank ? p.per_clus : 0;
      return ((size_t)cols * (p.per_phase * 256 + kXPad) + (size_t)p.per_phase * tb * 4 +
              (size_t)res * kPartRow * B * 4 + 15) & ~(size_t)15;
    };
    while (front() + ring_bytes(nt, 2) > kSmemLimit && p.per_phase > 1) p.per_phase = (p.per_phase + 1) / 2;
    p.ring_at = front();
    if (p.ring_at + ring_bytes(nt, 2) > kSmemLimit) continue;
    for (p.depth = 4; p.ring_at + ring_bytes(nt, p.depth) > kSmemLimit;) --p.depth;
    p.smem = p.ring_at + ring_bytes(nt, p.depth);
    const int phases = (p.per_rank + p.per_phase - 1) / p.per_phase;
    const double cost = (double)p.per_clus * p.per_rank + 0.17 * cols * p.per_rank + kJoin[ci] + 30.0 * (phases - 1);
    if (cost < least) {
      least = cost;
      *best = p;
    }
  }
  return least < 1e300;
}

}  // namespace

cudaError_t launch_linear4_pack(const uint8_t* codes, const uint16_t* scales, const prox_linear4* L, cudaStream_t s) {
  linear4_pack_kernel<<<1184, 256, 0, s>>>(codes, reinterpret_cast<const __half*>(scales), L->N, L->G, L->strips,
                                           reinterpret_cast<uint32_t*>(L->codes),
                                           reinterpret_cast<__half*>(L->scales));
  return cudaGetLastError();
}

cudaError_t setup_linear4(prox_linear4* L) {
  for (int dtype : {PROX_F32, PROX_F16, PROX_BF16})
    for (int nt : {1, 2, 4}) {
      if (nt == 4 && dtype != PROX_F32) continue;
      for (int depth : {2, 3, 4}) {
        cudaError_t e = cudaFuncSetAttribute(pick(dtype, nt, depth), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kSmemLimit);
        if (e != cudaSuccess) return e;
      }
    }
  L->clusters[0] = L->num_sms;
  for (int ci = 1; ci < 4; ++ci) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(L->num_sms >> ci << ci), 1, 1);
    cfg.blockDim = dim3(warps_of(1) * 32, 1, 1);
    cfg.dynamicSmemBytes = kSmemLimit;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << ci;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    cudaError_t e = cudaOccupancyMaxActiveClusters(&n, pick(PROX_BF16, 1, 4), &cfg);
    if (e != cudaSuccess) return e;
    L->clusters[ci] = n;
  }
  return cudaSuccess;
}

cudaError_t launch_linear4(const prox_linear4* L, const void* x, int64_t x_stride, void* out, int64_t out_stride,
                           int B, int dtype, cudaStream_t s) {
  // All strips in one launch, unless x takes several phases (or a cluster) and
  // the results that are then kept in shared memory do not fit: fewer strips a
  // launch.  (16 fp32 tokens over some 10^5 channels or more.)
  Plan p;
  int chunk = L->strips;
  while (!plan_linear4(L, chunk, B, dtype, &p)) {
    if (chunk == 1) return cudaErrorInvalidConfiguration;
    chunk = (chunk + 1) / 2;
  }
  const int nt = col_tiles(B, dtype), size = dtype == PROX_F32 ? 4 : 2;
  LinearArgs a;
  a.x = x;
  a.x_stride = x_stride;
  a.out_stride = out_stride;
  a.B = B;
  a.G = L->G;
  a.x_vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (B == 1 || x_stride % (16 / size) == 0);
  for (int first = 0; first < L->strips; first += chunk) {
    if (L->strips - first < chunk && !plan_linear4(L, L->strips - first, B, dtype, &p))
      return cudaErrorInvalidConfiguration;
    a.codes = reinterpret_cast<const char*>(L->codes) + (size_t)first * L->G * kCodeBytes;
    a.scales = reinterpret_cast<const char*>(L->scales) + (size_t)first * L->G * kScaleBytes;
    a.out = static_cast<char*>(out) + (size_t)first * kStrip * size;
    a.N = L->N - first * kStrip;
    a.strips = L->strips - first < chunk ? L->strips - first : chunk;
    if (a.strips == chunk && first + chunk < L->strips) a.N = chunk * kStrip;
    a.per_clus = p.per_clus;
    a.per_rank = p.per_rank;
    a.per_phase = p.per_phase;
    a.cluster = p.cluster;
    a.ring_at = (int)p.ring_at;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.clusters * p.cluster), 1, 1);
    cfg.blockDim = dim3(warps_of(nt) * 32, 1, 1);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, pick(dtype, nt, p.depth), a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace prox
