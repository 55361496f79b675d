// y = x W for 1..16 tokens, W [K, N] held as INT4 codes with one fp16 scale
// per group of 128 input rows and channel:
//   y[b, n] = sum_g S[g, n] sum_{k in g} q[k, n] x[b, k],   q = code - 8.
//
// The product runs on the tensor cores with the channels as the M dimension
// (A = the codes, widened in registers, 16 channels x 16 input rows) and the
// tokens as N = 8 columns (B = x from shared memory), because at N = 8 the
// fragment of a code word feeds one instruction whatever the batch: the codes,
// which are all of the traffic, are decoded once.  Codes are stored in
// fragment order, so a lane's 8 words of a 16 x 128 unit are two 16-byte loads
// of a stretch that the warp reads contiguously, and no shuffle or shared
// memory stands between HBM and the tensor core.
//
// x is held in fp16: fp16 as it is; bf16 exactly, scaled by a power of two per
// token and group; fp32 as hi + lo columns (22 significant bits) scaled the
// same way.  A unit's sum over its 128 rows is taken by the tensor core in
// fp32, then scaled and added in fp32, so no sum is held in fewer bits and the
// tensor core's running sum is never longer than 8 instructions.
//
// Split: the units (tile of channels, group) of a cluster's tiles are dealt
// to the CTA's warps as equal contiguous ranges; a tile that two warps share
// is joined through shared memory in warp order, and the CTAs of a cluster
// (which split K when there are too few channels to fill the device) join
// theirs through distributed shared memory in rank order, so results do not
// depend on timing and no scratch in global memory is shared between calls.
//
// Bound: HBM at large sizes (0.52 bytes per weight), launch and one pass of
// load latency at small ones.
#include "decode4.h"
#include "quant4.cuh"

namespace prox {
namespace {

using namespace q4;

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kXPad = 64;          // bytes; makes 16-byte reads of 8 columns conflict-free
constexpr int kSmemLimit = 227 * 1024;

struct LinearArgs {
  const uint8_t* codes;
  const __half* scales;
  const void* x;
  int64_t x_stride;
  void* out;
  int64_t out_stride;
  int B, N, G;
  int strips;      // strips of M tiles in all
  int per_clus;    // strips of a cluster
  int per_rank;    // groups of a CTA of the cluster
  int per_phase;   // groups whose x is in shared memory at once
  int cluster;
  int x_vec;       // x rows allow 4-value vector loads
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

// Start of the w-th of W equal contiguous ranges of U units.
__device__ __forceinline__ int range_at(int U, int w, int W) { return (int)((long long)U * w / W); }
// The range that holds unit u.
__device__ __forceinline__ int range_of(int U, int u, int W) { return (int)(((long long)(u + 1) * W - 1) / U); }

// NT column tiles of 8 (tokens, or their hi / lo parts), M tiles of 16
// channels per strip, PF units in flight per warp.
template <int DT, int NT, int M, int PF>
__global__ void __launch_bounds__(kThreads, 1) linear4_kernel(const LinearArgs a) {
  using T = typename Act<DT>::T;
  constexpr int PARTS = DT == PROX_F32 ? 2 : 1;
  constexpr bool NORM = DT != PROX_F16;
  constexpr int TB = 8 * NT / PARTS;  // tokens
  constexpr int ROWS = 16 * M;        // channels of a strip
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
  const int clus = (int)blockIdx.x / a.cluster;
  const int s0 = min(clus * a.per_clus, a.strips), s1 = min(s0 + a.per_clus, a.strips);
  const int g0 = min(rank * a.per_rank, a.G), g1 = min(g0 + a.per_rank, a.G);
  const int cols = a.B * PARTS;
  const int xs = a.per_phase * 256 + kXPad;  // bytes of a column
  char* s_x = smem;
  float* s_nf = reinterpret_cast<float*>(smem + (size_t)cols * xs);          // [per_phase][TB]
  float* s_slot = s_nf + (NORM ? a.per_phase * TB : 0);                      // [kWarps][2][ROWS][B]
  float* s_res = s_slot + kWarps * 2 * ROWS * a.B;                           // [per_clus][ROWS][B]
  const bool use_res = a.cluster > 1 || a.per_phase < g1 - g0 || a.per_phase < a.per_rank;
  T* out = static_cast<T*>(a.out);

  // A warp's results of one strip (token columns in the caller's order).
  float acc[M][NT][4];
  auto each = [&](auto&& f) {
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = 16 * m + 8 * r + g;
          if (PARTS == 2) {
            if (4 * n + t < a.B) f(row, 4 * n + t, acc[m][n][2 * r] + acc[m][n][2 * r + 1]);
          } else {
            if (8 * n + 2 * t < a.B) f(row, 8 * n + 2 * t, acc[m][n][2 * r]);
            if (8 * n + 2 * t + 1 < a.B) f(row, 8 * n + 2 * t + 1, acc[m][n][2 * r + 1]);
          }
        }
  };
  auto put = [&](int strip, int row, int b, float v) {
    const int n = strip * ROWS + row;
    if (n < a.N) out[b * a.out_stride + n] = Act<DT>::from(v);
  };

  const int phases = max(1, (a.per_rank + a.per_phase - 1) / a.per_phase);
  for (int ph = 0; ph < phases; ++ph) {
    const int pg0 = min(g0 + ph * a.per_phase, g1), pg1 = min(pg0 + a.per_phase, g1);
    const int nG = pg1 - pg0, U = (s1 - s0) * nG;
    const int W = min(U, kWarps);
    const int beg = warp < W ? range_at(U, warp, W) : U, end = warp < W ? range_at(U, warp + 1, W) : U;

    uint4 buf[PF][M][2];
    __half2 sc[PF][M];
    int ls = nG ? s0 + beg / nG : 0, lg = nG ? beg % nG : 0;  // the next unit to load
    auto load = [&](int j) {
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const size_t unit = (size_t)(ls * M + m) * a.G + (pg0 + lg);
        const uint4* p = reinterpret_cast<const uint4*>(a.codes) + unit * 64 + lane;
        buf[j][m][0] = ld_stream_v4(p);
        buf[j][m][1] = ld_stream_v4(p + 32);
        sc[j][m] = *(reinterpret_cast<const __half2*>(a.scales) + unit * 8 + g);
      }
      if (++lg == nG) lg = 0, ++ls;
    };
    // The weights do not depend on the kernel before this one in the stream.
#pragma unroll
    for (int j = 0; j < PF; ++j)
      if (beg + j < end) load(j);
    if (ph == 0) {
      pdl_wait();
      pdl_trigger();
    } else {
      __syncthreads();  // the phase before has been read
    }

    // x of this phase's groups into columns: a warp takes a token's group, XB
    // of them at once so that their loads overlap.
    constexpr int XB = 4;
    for (int first = warp; first < a.B * nG; first += XB * kWarps) {
      float v[XB][4];
#pragma unroll
      for (int q = 0; q < XB; ++q) {
        const int item = first + q * kWarps;
        if (item >= a.B * nG) break;
        const T* src = static_cast<const T*>(a.x) + (item / nG) * a.x_stride +
                       (int64_t)(pg0 + item % nG) * kGroupRows + 4 * lane;
        load_vals<DT, 4>(src, a.x_vec, v[q]);
      }
#pragma unroll
      for (int q = 0; q < XB; ++q) {
        const int item = first + q * kWarps;
        if (item >= a.B * nG) break;
        const int b = item / nG, gr = item % nG;
        float f = 1.f;
        if (NORM) {
          float mx = fmaxf(fmaxf(fabsf(v[q][0]), fabsf(v[q][1])), fmaxf(fabsf(v[q][2]), fabsf(v[q][3])));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          f = normaliser(mx);
          if (lane == 0) s_nf[gr * TB + b] = inv_pow2(f);
        }
        float hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = v[q][i] * f;
          hi[i] = __half2float(__float2half_rn(y));
          lo[i] = y - hi[i];
        }
        char* col = s_x + (size_t)(b * PARTS) * xs + gr * 256 + 8 * lane;
        store_vals<PROX_F16, 4>(reinterpret_cast<__half*>(col), true, hi);
        if (PARTS == 2) store_vals<PROX_F16, 4>(reinterpret_cast<__half*>(col + xs), true, lo);
      }
    }
    __syncthreads();

    // this lane's column of x in each tile (columns past the batch repeat the
    // last one; their results are not used)
    const char* xcol[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xcol[n] = s_x + (size_t)min(8 * n + g, cols - 1) * xs + 16 * t;
    const float* nf = s_nf + (PARTS == 2 ? t : 2 * t);

    auto flush = [&](int strip) {
      const int from = (strip - s0) * nG;  // the strip's units: [from, from + nG)
      if (from >= beg && from + nG <= end) {
        if (!use_res)
          each([&](int row, int b, float v) { put(strip, row, b, v); });
        else
          each([&](int row, int b, float v) {
            float* r = s_res + ((size_t)(strip - s0) * ROWS + row) * a.B + b;
            *r = ph == 0 ? v : *r + v;
          });
      } else {
        float* slot = s_slot + (size_t)(warp * 2 + (from < beg ? 0 : 1)) * ROWS * a.B;
        each([&](int row, int b, float v) { slot[row * a.B + b] = v; });
      }
    };
    auto clear = [&]() {
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
    };

    clear();
    int cs = nG ? s0 + beg / nG : 0, cg = nG ? beg % nG : 0;  // the unit to compute
    for (int base = beg; base < end; base += PF) {
#pragma unroll
      for (int j = 0; j < PF; ++j) {
        if (base + j >= end) break;
        // two chains per tile: even and odd 16-row steps
        float part[M][NT][2][4];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[m][n][0][i] = part[m][n][1][i] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 xv[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) xv[n] = lds_v4(xcol[n] + cg * 256 + i * 64);
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const uint4 w4 = buf[j][m][i >> 1];
            const uint32_t w0 = (i & 1) ? w4.z : w4.x, w1 = (i & 1) ? w4.w : w4.y;
            uint32_t r[4];
            widen8(w0, r);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(part[m][n][0], r[0], r[2], r[1], r[3], xv[n].x, xv[n].y);
            widen8(w1, r);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(part[m][n][1], r[0], r[2], r[1], r[3], xv[n].z, xv[n].w);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float f0 = 1.f, f1 = 1.f;
          if (NORM) {
            if (PARTS == 2) {
              f0 = f1 = nf[cg * TB + 4 * n];
            } else {
              const float2 f = *reinterpret_cast<const float2*>(nf + cg * TB + 8 * n);
              f0 = f.x, f1 = f.y;
            }
          }
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const float2 s = __half22float2(sc[j][m]);
            float* p0 = part[m][n][0];
            const float* p1 = part[m][n][1];
            acc[m][n][0] = fmaf((p0[0] + p1[0]) * s.x, f0, acc[m][n][0]);
            acc[m][n][1] = fmaf((p0[1] + p1[1]) * s.x, f1, acc[m][n][1]);
            acc[m][n][2] = fmaf((p0[2] + p1[2]) * s.y, f0, acc[m][n][2]);
            acc[m][n][3] = fmaf((p0[3] + p1[3]) * s.y, f1, acc[m][n][3]);
          }
        }
        if (base + j + PF < end) load(j);
        if (++cg == nG || base + j + 1 == end) {
          flush(cs);
          clear();
          if (cg == nG) cg = 0, ++cs;
        }
      }
    }
    __syncthreads();
    // strips that several warps share, in warp order
    for (int s = s0 + warp; s < s1 && nG > 0; s += kWarps) {
      const int from = (s - s0) * nG;
      const int wa = range_of(U, from, W), wb = range_of(U, from + nG - 1, W);
      if (wa == wb) continue;
      for (int e = lane; e < ROWS * a.B; e += 32) {
        // e runs over the rows of one token first: neighbours in the output
        const int b = e / ROWS, row = e % ROWS;
        float v = s_slot[(size_t)(wa * 2 + 1) * ROWS * a.B + row * a.B + b];
        for (int w = wa + 1; w <= wb; ++w) v += s_slot[(size_t)(w * 2) * ROWS * a.B + row * a.B + b];
        if (use_res) {
          float* r = s_res + ((size_t)(s - s0) * ROWS + row) * a.B + b;
          *r = ph == 0 ? v : *r + v;
        } else {
          put(s, row, b, v);
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
  const int E = (s1 - s0) * ROWS * a.B;
  for (int e = rank * kThreads + threadIdx.x; e < E; e += a.cluster * kThreads) {
    const int s = e / (ROWS * a.B), b = e / ROWS % a.B, row = e % ROWS;
    const float* p = s_res + ((size_t)s * ROWS + row) * a.B + b;
    float v = a.cluster > 1 ? ld_peer(p, 0) : *p;
    for (int r = 1; r < ranks; ++r) v += ld_peer(p, r);
    put(s0 + s, row, b, v);
  }
  if (a.cluster > 1) cluster_sync_all();  // no CTA leaves while its results are read
}

// Word j of lane l of unit (tile, g): see widen8's order; rows past N hold
// zeros with scale 0.
__global__ void linear4_pack_kernel(const uint8_t* __restrict__ codes, const __half* __restrict__ scales, int N, int G,
                                    int S, uint32_t* __restrict__ out, __half* __restrict__ out_scales) {
  const size_t n_word = (size_t)S * G * 256, n_scale = (size_t)S * G * 16;
  const size_t stride = (size_t)gridDim.x * blockDim.x;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n_word + n_scale; i += stride) {
    if (i < n_word) {
      const int wi = i & 3, l = (i >> 2) & 31, j = (i >> 7) & 1;
      const size_t unit = i >> 8;
      const int gr = unit % G, tile = unit / G;
      const int k0 = gr * kGroupRows + 32 * (2 * j + (wi >> 1)) + 8 * (l & 3) + 4 * (wi & 1);
      uint32_t w = 0;
#pragma unroll
      for (int nib = 0; nib < 8; ++nib) {
        // nibbles 0, 4, 1, 5: row l / 4, input rows k0 .. k0 + 3; 2, 6, 3, 7: row + 8
        const int n = tile * 16 + (l >> 2) + ((nib & 2) ? 8 : 0);
        const int k = k0 + 2 * (nib & 1) + (nib >> 2);
        const uint32_t c = n < N ? (codes[(size_t)k * (N / 2) + n / 2] >> (4 * (n & 1))) & 15u : 8u;
        w |= c << (4 * nib);
      }
      out[i] = w;
    } else {
      const size_t u = i - n_word;
      const int r = u & 15;
      const size_t unit = u >> 4;
      const int gr = unit % G, tile = unit / G;
      const int n = tile * 16 + (r >> 1) + 8 * (r & 1);
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
// One tile of channels per strip up to 16 columns.  At 32 columns the x reads
// from shared memory would take longer than the codes from HBM, so two tiles
// share them.
int strip_tiles(int nt) { return nt == 4 ? 2 : 1; }

Kernel pick(int dtype, int nt) {
  switch (dtype) {
    case PROX_F32:
      return nt == 1 ? linear4_kernel<PROX_F32, 1, 1, 4>
                     : nt == 2 ? linear4_kernel<PROX_F32, 2, 1, 4> : linear4_kernel<PROX_F32, 4, 2, 1>;
    case PROX_F16: return nt == 1 ? linear4_kernel<PROX_F16, 1, 1, 4> : linear4_kernel<PROX_F16, 2, 1, 4>;
    default: return nt == 1 ? linear4_kernel<PROX_BF16, 1, 1, 4> : linear4_kernel<PROX_BF16, 2, 1, 4>;
  }
}

struct Plan {
  int cluster, per_clus, per_rank, per_phase, clusters;
  size_t smem;
};

size_t smem_bytes(int cols, int B, int tb, bool norm, int rows, int per_phase, int res_strips) {
  return (size_t)cols * (per_phase * 256 + kXPad) + (norm ? (size_t)per_phase * tb * 4 : 0) +
         (size_t)(kWarps * 2 + res_strips) * rows * B * 4;
}

// The cluster size whose busiest warp has the least to do.  Counted in units
// of one warp (a 16 x 128 block of codes, about 1 KB): a CTA's units over its
// 16 warps, plus what joining across the cluster costs (about 1 us, what 40
// units of the CTA take), plus a penalty per extra phase of x.
bool plan_linear4(const prox_linear4* L, int B, int dtype, Plan* best) {
  const int nt = col_tiles(B, dtype), M = strip_tiles(nt), parts = dtype == PROX_F32 ? 2 : 1;
  const int rows = 16 * M, cols = B * parts, tb = 8 * nt / parts;
  const int strips = (L->S + M - 1) / M;
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
    const bool norm = dtype != PROX_F16;
    while (smem_bytes(cols, B, tb, norm, rows, p.per_phase,
                      c > 1 || p.per_phase < p.per_rank ? p.per_clus : 0) > kSmemLimit) {
      if (p.per_phase == 1) break;
      p.per_phase = (p.per_phase + 1) / 2;
    }
    p.smem = smem_bytes(cols, B, tb, norm, rows, p.per_phase,
                        c > 1 || p.per_phase < p.per_rank ? p.per_clus : 0);
    if (p.smem > kSmemLimit) continue;
    const int phases = (p.per_rank + p.per_phase - 1) / p.per_phase;
    const double cost = (double)p.per_clus * M * p.per_rank + (c > 1 ? 40.0 : 0.0) + 60.0 * (phases - 1);
    if (cost < least) {
      least = cost;
      *best = p;
    }
  }
  return least < 1e300;
}

}  // namespace

cudaError_t launch_linear4_pack(const uint8_t* codes, const uint16_t* scales, const prox_linear4* L, cudaStream_t s) {
  linear4_pack_kernel<<<1184, 256, 0, s>>>(codes, reinterpret_cast<const __half*>(scales), L->N, L->G, L->S,
                                           reinterpret_cast<uint32_t*>(L->codes),
                                           reinterpret_cast<__half*>(L->scales));
  return cudaGetLastError();
}

cudaError_t setup_linear4(prox_linear4* L) {
  for (int dtype : {PROX_F32, PROX_F16, PROX_BF16})
    for (int nt : {1, 2, 4}) {
      if (nt == 4 && dtype != PROX_F32) continue;
      const Kernel k = pick(dtype, nt);
      cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
      if (e != cudaSuccess) return e;
    }
  L->clusters[0] = L->num_sms;
  for (int ci = 1; ci < 4; ++ci) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(L->num_sms >> ci << ci), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemLimit;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << ci;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    cudaError_t e = cudaOccupancyMaxActiveClusters(&n, pick(PROX_BF16, 1), &cfg);
    if (e != cudaSuccess) return e;
    L->clusters[ci] = n;
  }
  return cudaSuccess;
}

cudaError_t launch_linear4(const prox_linear4* L, const void* x, int64_t x_stride, void* out, int64_t out_stride,
                           int B, int dtype, cudaStream_t s) {
  Plan p;
  if (!plan_linear4(L, B, dtype, &p)) return cudaErrorInvalidConfiguration;
  const int nt = col_tiles(B, dtype), M = strip_tiles(nt);
  LinearArgs a;
  a.codes = L->codes;
  a.scales = reinterpret_cast<const __half*>(L->scales);
  a.x = x;
  a.x_stride = x_stride;
  a.out = out;
  a.out_stride = out_stride;
  a.B = B;
  a.N = L->N;
  a.G = L->G;
  a.strips = (L->S + M - 1) / M;
  a.per_clus = p.per_clus;
  a.per_rank = p.per_rank;
  a.per_phase = p.per_phase;
  a.cluster = p.cluster;
  const int bytes4 = dtype == PROX_F32 ? 16 : 8;
  a.x_vec = (reinterpret_cast<uintptr_t>(x) % bytes4) == 0 && x_stride % 4 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.clusters * p.cluster), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
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
  return cudaLaunchKernelEx(&cfg, pick(dtype, nt), a);
}

}  // namespace prox
