// Attention of each request's newest tokens over a paged 4-bit cache.
//
// Mathematics.  With K_j = ks_j q^K_j and V_j = vs_j q^V_j (integers q, one
// fp16 scale per token and head) a query row needs
//   t_j = (scale log2 e) ks_j (Q . q^K_j),   o = sum_j 2^(t_j - m) vs_j q^V_j / sum_j 2^(t_j - m),
// so the scales multiply scores and probabilities, never the codes: both
// products run on integers widened to fp16, exactly.
//
// One warp keeps the running maximum, sum and output of the rows (query heads
// of one group x new tokens) it works on, and takes 32 cache rows a step:
//   S^T = K Q^T   tokens are the M dimension, the rows the N = 8 columns, so a
//                 group of up to 8 heads wastes no tensor work and a code is
//                 widened once for all of them;
//   O^T = V^T P^T the same, with P^T turned into the B operand by movmatrix.
// K words are A fragments as they lie (the order of d inside a product is
// free, so Q takes the codes' order); V needs pairs of tokens in one register,
// one byte permute per word.  Which token stands in which fragment row is free
// too, and chosen so that the shared-memory reads of K and V meet no bank
// conflict at head_dim 128 (see token_of).
// fp16 and bf16 queries are exact in fp16 (bf16 scaled by a power of two);
// fp32 queries and their probabilities are split into hi + lo columns.
// Probabilities times vs are scaled by a power of two per step so that they
// use fp16's range; each step's product starts from zero and joins the fp32
// output with one fused multiply-add, so the tensor core's own sums stay short.
//
// Split.  The unit is 32 rows of one (request, kv head).  All units of the
// call are dealt to the CTAs, one per SM, and in a CTA to its warps, as equal
// contiguous ranges, whatever the requests' lengths: no rows are padded, and
// no length is known to the host.  A warp streams its range through its own
// ring of cp.async copies without any block barrier; at the end contexts that
// several warps share are joined through shared memory, and those that several
// CTAs share by the last of them to arrive, always in the same order.
//
// Bound: HBM, (head_dim + 4) bytes per token and kv head.
#include <type_traits>

#include "decode4.h"
#include "quant4.cuh"

namespace prox {
namespace {

using namespace q4;

constexpr int kStep = 32;    // cache rows of one step
constexpr int kMaxWarps = 12;
constexpr int kStages = 3;   // steps in flight or in use per warp
constexpr int kSmemLimit = 227 * 1024;

struct AttendArgs {
  Attend4Call c;
  const uint8_t* k;
  const uint16_t* ks;
  const uint8_t* v;
  const uint16_t* vs;
  int pages, heads, page_shift;
  int G, R, blocks;  // heads per kv head, rows per kv head, row blocks
  int* err;
  float* part;
  int* arrived;
  bool q_vec;
};

// The token (of 16) that stands in row r of a fragment: rows 2t and 2t + 1 are
// tokens t and 4 + (t ^ 1), the second eight likewise 8 further.  A quarter
// warp then reads K of tokens of both parities (all banks), and V of four
// consecutive tokens.
__device__ __forceinline__ int token_of(int r) { return (r & 8) + ((r & 1) ? 4 + (((r & 7) >> 1) ^ 1) : (r & 7) >> 1); }

// Where 16-byte piece j of row `row` lies in a stage (K, V).
template <int D>
__device__ __forceinline__ int k_piece(int row, int j) {
  if (D == 256) j ^= 4 * (row & 1);
  return row * (D / 2) + 16 * j;
}
template <int D>
__device__ __forceinline__ int v_piece(int row, int j) {
  if (D == 256) j ^= 2 * (row & 3);
  if (D == 128) j ^= 2 * ((row >> 1) & 1);
  return row * (D / 2) + 16 * j;
}

template <int D>
constexpr int stage_bytes() {
  return kStep * D + kStep * 4;
}
// One partial result: [rows][D] output, then maxima and sums.
constexpr int part_floats(int rows, int D) { return rows * D + 2 * rows; }

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// A position in the sequence of units: chunk c of n of (request b, head block hb).
struct Cursor {
  int b, hb, c, n, len;
  long long beg;  // unit of chunk 0
};

template <int DT, int D, int NT>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) attend4_kernel(const AttendArgs a) {
  using T = typename Act<DT>::T;
  constexpr int PARTS = DT == PROX_F32 ? 2 : 1;
  constexpr int RB = 8 * NT / PARTS;   // rows of a block
  constexpr int NC = 2 / PARTS;        // rows a thread has per column tile
  constexpr int KW = D / 32;           // K words per thread and token
  constexpr int VW = D / 64;           // V words per thread and token
  constexpr int PIECES = D / 32;       // 16-byte pieces of a row
  constexpr int SB = stage_bytes<D>();
  constexpr int SLOT = part_floats(RB, D);
  const Attend4Call& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;

  extern __shared__ __align__(16) char smem[];
  char* ring = smem + (size_t)warp * kStages * SB;
  float* heads_part = reinterpret_cast<float*>(smem + (size_t)warps * kStages * SB);  // [warps][SLOT]
  int* pre = reinterpret_cast<int*>(heads_part + (size_t)warps * SLOT);               // [B + 1]
  __shared__ long long s_scan[33];
  __shared__ long long s_head_seg[kMaxWarps], s_tail_seg[kMaxWarps];  // first unit of the context, -1: none
  __shared__ int s_head_done[kMaxWarps];
  __shared__ int s_last;

  pdl_wait();
  pdl_trigger();

  // chunk counts of the requests
  const int max_len = (int)min((long long)c.cols << a.page_shift, 0x7fffffffLL - 64);
  const int per = (c.B + blockDim.x - 1) / blockDim.x;
  const int rlo = min((int)threadIdx.x * per, c.B), rhi = min(rlo + per, c.B);
  long long mine = 0;
  for (int i = rlo; i < rhi; ++i) {
    const int len = c.lens[i];
    if ((len < 0 || len > max_len) && blockIdx.x == 0) atomicOr(a.err, PROX_DEVERR_LEN);
    mine += max(1, (min(max(len, 0), max_len) + kStep - 1) / kStep);
  }
  long long total;
  long long at = block_exclusive_scan(mine, s_scan, &total);
  for (int i = rlo; i < rhi; ++i) {
    pre[i] = (int)at;
    at += max(1, (min(max(c.lens[i], 0), max_len) + kStep - 1) / kStep);
  }
  if (threadIdx.x == 0) pre[c.B] = (int)total;
  if (threadIdx.x < kMaxWarps) s_head_seg[threadIdx.x] = s_tail_seg[threadIdx.x] = -1;
  __syncthreads();

  const int H = a.heads * a.blocks;
  const long long U = total * H;
  const int P = (int)min((long long)gridDim.x, U);  // CTAs with work
  if ((int)blockIdx.x >= P) return;
  const long long cb = U * blockIdx.x / P, ce = U * (blockIdx.x + 1) / P;
  const int W = (int)min((long long)warps, ce - cb);
  const long long wb = warp < W ? cb + (ce - cb) * warp / W : ce;
  const long long we = warp < W ? cb + (ce - cb) * (warp + 1) / W : ce;

  auto enter = [&](Cursor& s) {  // request s.b, whatever head block
    s.n = pre[s.b + 1] - pre[s.b];
    s.len = min(max(c.lens[s.b], 0), max_len);
  };
  auto seek = [&](long long u) {
    Cursor s;
    int lo = 0, hi = c.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)pre[mid] * H <= u)
        lo = mid;
      else
        hi = mid;
    }
    s.b = lo;
    enter(s);
    const long long r = u - (long long)pre[lo] * H;
    s.hb = (int)(r / s.n);
    s.c = (int)(r % s.n);
    s.beg = u - s.c;
    return s;
  };
  auto advance = [&](Cursor& s) {  // not past the last unit
    if (++s.c < s.n) return;
    s.beg += s.n;
    s.c = 0;
    if (++s.hb == H) {
      s.hb = 0;
      if (++s.b < c.B) enter(s);
    }
  };

  // ---- producer: the copies of one step, one page lookup ahead --------------
  int pid[2] = {0, 0};
  auto lookup = [&](const Cursor& s) {
    const int32_t* row = c.table + s.b * c.table_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int tok = s.c * kStep + 16 * h;
      int id = 0;
      if (tok < s.len) {
        id = row[tok >> a.page_shift];
        if (id < 0 || id >= a.pages) {
          atomicOr(a.err, PROX_DEVERR_PAGE);
          id = 0;
        }
      }
      pid[h] = id;
    }
  };
  const int page_mask = (1 << a.page_shift) - 1;
  auto copy = [&](const Cursor& s, int stage) {
    char* dst = ring + stage * SB;
    const int tok0 = s.c * kStep, head = s.hb / a.blocks;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int id = i * 32 + lane, row = id / PIECES, j = id % PIECES;
      if (tok0 + row < s.len) {
        const int64_t r = ((int64_t)((row < 16 ? pid[0] : pid[1])) * a.heads + head << a.page_shift) +
                          ((tok0 + row) & page_mask);
        cp_async16(smem_u32(dst) + k_piece<D>(row, j), a.k + r * (D / 2) + 16 * j);
        cp_async16(smem_u32(dst) + kStep * D / 2 + v_piece<D>(row, j), a.v + r * (D / 2) + 16 * j);
      }
    }
    if (lane < 8) {  // scales: four pieces of 8 tokens each
      const int q = lane & 3;
      if (tok0 + 8 * q < s.len) {
        const int64_t r = ((int64_t)(pid[q >> 1]) * a.heads + head << a.page_shift) + ((tok0 + 8 * q) & page_mask);
        cp_async16(smem_u32(dst) + kStep * D + (lane >> 2) * kStep * 2 + 16 * q, (lane < 4 ? a.ks : a.vs) + r);
      }
    }
  };

  // ---- the rows' state -------------------------------------------------------
  uint32_t qf[KW][2][NT][2];
  float O[VW][4][2][NT][NC];   // [word][tile][row half][column tile][column]
  float mx[NT][NC], sum[NT][NC];
  int lim[NT][NC];             // last visible token
  float cm = 0.f;              // scale log2(e) / the queries' power of two

  auto row_of = [&](int nt, int e) { return PARTS == 2 ? 4 * nt + t : 8 * nt + 2 * t + e; };
  auto out_at = [&](const Cursor& s, int row) {  // element (b, i, h, 0) of row `row` of s's block, -1: none
    const int r = s.hb % a.blocks * RB + row;
    if (r >= a.R) return (int64_t)-1;
    return (((int64_t)s.b * c.Tq + r / a.G) * c.Hq + (s.hb / a.blocks) * a.G + r % a.G) * (int64_t)D;
  };

  auto begin_rows = [&](const Cursor& s) {
    float qv[NT][KW * 8];
    float top = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = s.hb % a.blocks * RB + (PARTS == 2 ? 4 * nt + (g >> 1) : 8 * nt + g);
      const T* q = static_cast<const T*>(c.q) + s.b * c.q_req + (r / a.G) * c.q_tok +
                   ((s.hb / a.blocks) * a.G + r % a.G) * c.q_head;
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        float x[8] = {};
        const int d = D == 64 ? 16 * t + 8 * i : 32 * t + 128 * (i >> 2) + 8 * (i & 3);
        if (r < a.R) load_vals<DT, 8>(q + d, a.q_vec, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          qv[nt][8 * i + j] = x[j];
          top = max_nan(top, fabsf(x[j]));
        }
      }
    }
    float f = 1.f;
    if (DT != PROX_F16) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      f = normaliser(top);
    }
    cm = c.scale * 1.4426950408889634f * inv_pow2(f);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = qv[nt][8 * i + j] * f;
          const __half hi = __float2half_rn(y);
          __half v = hi;
          if (PARTS == 2 && (g & 1)) v = __float2half_rn(y - __half2float(hi));
          w[j] = __half_as_ushort(v);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // pairs (2h, 2h + 4) and (2h + 1, 2h + 5)
          qf[i][h][nt][0] = w[2 * h] | w[2 * h + 4] << 16;
          qf[i][h][nt][1] = w[2 * h + 1] | w[2 * h + 5] << 16;
        }
      }
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        const int r = s.hb % a.blocks * RB + row_of(nt, e);
        lim[nt][e] = r < a.R ? s.len - c.Tq + r / a.G : s.len - 1;
        mx[nt][e] = -INFINITY;
        sum[nt][e] = 0.f;
      }
    }
#pragma unroll
    for (int x = 0; x < VW; ++x)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < NC; ++e) O[x][q][h][nt][e] = 0.f;
  };

  auto step = [&](const Cursor& s, int stage) {
    const char* st = ring + stage * SB;
    const __half* s_ks = reinterpret_cast<const __half*>(st + kStep * D);
    const __half* s_vs = s_ks + kStep;
    const int tok0 = s.c * kStep;
    // scores: token rows token_of(g) (+ 8), two tiles of 16 tokens
    float S[2][NT][4];
    float ksc[2][2], vsc[2][2];
    float vtop = 0.f;
    const int tr = token_of(g);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[m][nt][i] = 0.f;
      uint32_t w[2][KW];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * m + 8 * h + tr;
        if constexpr (D == 64) {
          const uint2 u = *reinterpret_cast<const uint2*>(st + row * 32 + 8 * t);
          w[h][0] = u.x, w[h][1] = u.y;
        } else {
#pragma unroll
          for (int p = 0; p < KW / 4; ++p) {
            const uint4 u = lds_v4(st + k_piece<D>(row, t + 4 * p));
            w[h][4 * p] = u.x, w[h][4 * p + 1] = u.y, w[h][4 * p + 2] = u.z, w[h][4 * p + 3] = u.w;
          }
        }
        const bool there = tok0 + row < s.len;
        ksc[m][h] = there ? __half2float(s_ks[row]) * cm : 0.f;
        vsc[m][h] = there ? __half2float(s_vs[row]) : 0.f;
        vtop = fmaxf(vtop, fabsf(vsc[m][h]) <= 65504.f ? fabsf(vsc[m][h]) : 0.f);
      }
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        uint32_t ra[4], rb[4];
        widen8(w[0][i], ra);
        widen8(w[1][i], rb);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(S[m][nt], ra[0], rb[0], ra[1], rb[1], qf[i][0][nt][0], qf[i][0][nt][1]);
          mma_f16(S[m][nt], ra[2], rb[2], ra[3], rb[3], qf[i][1][nt][0], qf[i][1][nt][1]);
        }
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, o));
    const float vf = normaliser(vtop), vinv = inv_pow2(vf);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) vsc[m][h] *= vf;

    // running softmax, then P^T as B fragments
    const bool masked = tok0 + kStep - 1 > s.len - c.Tq;
    uint32_t pf[2][NT][2];
    float alpha[NT][NC];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float p[2][2][NC];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < NC; ++e) {
            const float z = PARTS == 2 ? S[m][nt][2 * h] + S[m][nt][2 * h + 1] : S[m][nt][2 * h + e];
            p[m][h][e] = z * ksc[m][h];
            if (masked && tok0 + 16 * m + 8 * h + tr > lim[nt][e]) p[m][h][e] = -INFINITY;
          }
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        float top = fmaxf(fmaxf(p[0][0][e], p[0][1][e]), fmaxf(p[1][0][e], p[1][1][e]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, mx[nt][e]);
        const float base = top == -INFINITY ? 0.f : top;
        alpha[nt][e] = exp2_fast(mx[nt][e] - base);
        mx[nt][e] = top;
        float add = 0.f;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float x = p[m][h][e];
            const float y = exp2_fast(x - base);
            add += y;
            p[m][h][e] = masked && tok0 + 16 * m + 8 * h + tr > lim[nt][e] ? 0.f : y * vsc[m][h];
          }
        sum[nt][e] = fmaf(sum[nt][e], alpha[nt][e], add);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          __half2 v;
          if (PARTS == 2) {
            const __half hi = __float2half_rn(p[m][h][0]);
            v = __halves2half2(hi, __float2half_rn(p[m][h][0] - __half2float(hi)));
          } else {
            v = __floats2half2_rn(p[m][h][0], p[m][h][NC - 1]);
          }
          pf[m][nt][h] = transpose8(h2_bits(v));
        }
    }

    // O^T += V^T P^T: thread g has VW words of 8 values of each token
    const char* sv = st + kStep * D / 2;
    uint32_t vw[2][4][VW];  // [16 tokens][tokens of slots 2t, 2t + 1, 2t + 8, 2t + 9]
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = 16 * m + 8 * (q >> 1) + ((q & 1) ? 4 + (t ^ 1) : t);
        if constexpr (D == 64) {
          vw[m][q][0] = *reinterpret_cast<const uint32_t*>(sv + row * 32 + 4 * g);
        } else if constexpr (D == 128) {
          const uint2 u = *reinterpret_cast<const uint2*>(sv + v_piece<D>(row, g >> 1) + 8 * (g & 1));
          vw[m][q][0] = u.x, vw[m][q][1] = u.y;
        } else {
          const uint4 u = lds_v4(sv + v_piece<D>(row, g));
          vw[m][q][0] = u.x, vw[m][q][1] = u.y, vw[m][q][2] = u.z, vw[m][q][3] = u.w;
        }
      }
#pragma unroll
    for (int x = 0; x < VW; ++x)
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // values 8x + 4 half .. + 3 of the thread
        float part[2][NT][4];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[q][nt][i] = 0.f;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t r0[4], r1[4];
          widen8(prmt(vw[m][0][x], vw[m][1][x], half ? 0x7632 : 0x5410), r0);
          widen8(prmt(vw[m][2][x], vw[m][3][x], half ? 0x7632 : 0x5410), r1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16(part[0][nt], r0[0], r0[1], r1[0], r1[1], pf[m][nt][0], pf[m][nt][1]);
            mma_f16(part[1][nt], r0[2], r0[3], r1[2], r1[3], pf[m][nt][0], pf[m][nt][1]);
          }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < NC; ++e) {
                const float z = PARTS == 2 ? part[q][nt][2 * h] + part[q][nt][2 * h + 1] : part[q][nt][2 * h + e];
                float& o = O[x][2 * half + q][h][nt][e];
                o = fmaf(o, alpha[nt][e], z * vinv);
              }
      }
  };

  // The thread's 8 VW contiguous values of a row, times f.
  auto values = [&](int nt, int e, float f, float (&y)[8 * VW]) {
#pragma unroll
    for (int x = 0; x < VW; ++x)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) y[8 * x + 2 * q + h] = O[x][q][h][nt][e] * f;
  };
  auto end_rows = [&](const Cursor& s, float* slot) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        float l = sum[nt][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        const int row = row_of(nt, e);
        float y[8 * VW];
        if (slot) {
          values(nt, e, 1.f, y);
          store_vals<PROX_F32, 8 * VW>(slot + row * D + 8 * VW * g, true, y);
          if (g == 0) slot[RB * D + row] = mx[nt][e], slot[RB * D + RB + row] = l;
          continue;
        }
        const int64_t o = out_at(s, row);
        if (o < 0) continue;
        values(nt, e, l == 0.f ? 0.f : 1.f / l, y);
        store_vals<DT, 8 * VW>(static_cast<T*>(c.out) + o + 8 * VW * g, true, y);
        if (c.lse && g == 0) c.lse[o / D] = l == 0.f ? -INFINITY : 0.6931471805599453f * (mx[nt][e] + log2f(l));
      }
  };

  // ---- the warp's range -------------------------------------------------------
  if (wb < we) {
    Cursor cur = seek(wb), pro = cur;
    long long pu = wb;  // next unit to copy
    lookup(pro);
    auto issue = [&](int stage) {
      if (pu < we) {
        copy(pro, stage);
        if (++pu < we) {
          advance(pro);
          lookup(pro);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);
    int stage = 0;
    begin_rows(cur);
    for (long long u = wb; u < we; ++u) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      issue(stage == 0 ? kStages - 1 : stage - 1);
      step(cur, stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      const bool ends = cur.c + 1 == cur.n;
      if (ends || u + 1 == we) {
        float* slot = nullptr;
        if (cur.beg < wb) {
          slot = heads_part + (size_t)warp * SLOT;
          if (lane == 0) s_head_seg[warp] = cur.beg, s_head_done[warp] = ends;
        } else if (!ends) {
          // the warp's copies are done and read: its ring holds the part
          cp_async_wait<0>();
          __syncwarp();
          slot = reinterpret_cast<float*>(ring);
          if (lane == 0) s_tail_seg[warp] = cur.beg;
        }
        end_rows(cur, slot);
        if (u + 1 < we) {
          advance(cur);
          begin_rows(cur);
        }
      } else {
        advance(cur);
      }
    }
  }
  __syncthreads();

  // ---- contexts that several warps or CTAs share -------------------------------
  // `n` parts of one context, the i-th at part(i) (in shared memory, or written
  // by other CTAs): joined in order into the output, or into one part at `to`.
  auto join = [&](auto shared, int n, auto&& part, const Cursor& s, float* to) {
    constexpr bool kShared = decltype(shared)::value;
    auto ld1 = [](const float* p) { return kShared ? *p : __ldcg(p); };
    auto ld4 = [](const float* p) {
      return kShared ? *reinterpret_cast<const float4*>(p) : __ldcg(reinterpret_cast<const float4*>(p));
    };
    for (int e = threadIdx.x; e < RB * (D / 4); e += blockDim.x) {
      const int row = e / (D / 4), d = e % (D / 4) * 4;
      float top = -INFINITY;
      for (int i = 0; i < n; ++i) top = fmaxf(top, ld1(part(i) + RB * D + row));
      const float base = top == -INFINITY ? 0.f : top;
      float l = 0.f;
      float y[4] = {};
      for (int i = 0; i < n; ++i) {
        const float* p = part(i);
        const float f = exp2_fast(ld1(p + RB * D + row) - base);
        l = fmaf(ld1(p + RB * D + RB + row), f, l);
        const float4 o = ld4(p + row * D + d);
        y[0] = fmaf(o.x, f, y[0]), y[1] = fmaf(o.y, f, y[1]);
        y[2] = fmaf(o.z, f, y[2]), y[3] = fmaf(o.w, f, y[3]);
      }
      if (to) {
        store_vals<PROX_F32, 4>(to + row * D + d, true, y);
        if (d == 0) to[RB * D + row] = top, to[RB * D + RB + row] = l;
        continue;
      }
      const int64_t o = out_at(s, row);
      if (o < 0) continue;
      const float f = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] *= f;
      store_vals<DT, 4>(static_cast<T*>(c.out) + o + d, true, y);
      if (c.lse && d == 0) c.lse[o / D] = l == 0.f ? -INFINITY : 0.6931471805599453f * (top + log2f(l));
    }
  };
  auto close = [&](int first, int last, bool from_head, long long seg, bool done) {
    // parts: the first warp's head or tail, then the heads of the warps after it
    auto part = [&](int i) -> const float* {
      if (i == 0 && !from_head) return reinterpret_cast<const float*>(smem + (size_t)first * kStages * SB);
      return heads_part + (size_t)(first + i) * SLOT;
    };
    const Cursor s = seek(seg);
    const bool left = seg < cb;  // began in an earlier CTA
    if (!left && done) {
      join(std::true_type(), last - first + 1, part, s, nullptr);
      return;
    }
    float* to = a.part + (size_t)(2 * blockIdx.x + (left ? 0 : 1)) * SLOT;
    join(std::true_type(), last - first + 1, part, s, to);
    __threadfence();
    __syncthreads();
    const int c0 = (int)(((seg + 1) * P - 1) / U), c1 = (int)(((seg + s.n) * P - 1) / U);
    if (threadIdx.x == 0) {
      const int n = atomicAdd(a.arrived + c0, 1);
      s_last = n == c1 - c0;
      if (s_last) a.arrived[c0] = 0;  // for the next call
    }
    __syncthreads();
    if (s_last) {
      __threadfence();
      join(std::false_type(), c1 - c0 + 1,
           [&](int i) -> const float* { return a.part + (size_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * SLOT; }, s,
           nullptr);
    }
  };
  int first = -1;
  bool from_head = false;
  long long seg = -1;
  for (int w = 0; w < W; ++w) {
    if (s_head_seg[w] >= 0) {
      if (first < 0) first = w, from_head = true, seg = s_head_seg[w];
      if (s_head_done[w]) {
        close(first, w, from_head, seg, true);
        first = -1;
      }
    }
    if (s_tail_seg[w] >= 0) first = w, from_head = false, seg = s_tail_seg[w];
  }
  if (first >= 0) close(first, W - 1, from_head, seg, false);
}

using Kernel = void (*)(const AttendArgs);

template <int DT>
Kernel pick_d(int D, int nt) {
  if (D == 64) return nt == 1 ? attend4_kernel<DT, 64, 1> : attend4_kernel<DT, 64, 2>;
  if (D == 128) return nt == 1 ? attend4_kernel<DT, 128, 1> : attend4_kernel<DT, 128, 2>;
  return attend4_kernel<DT, 256, 1>;
}
Kernel pick(int dtype, int D, int nt) {
  switch (dtype) {
    case PROX_F32: return pick_d<PROX_F32>(D, nt);
    case PROX_F16: return pick_d<PROX_F16>(D, nt);
    default: return pick_d<PROX_BF16>(D, nt);
  }
}
// Two column tiles where one does not hold a kv head's rows; head_dim 256
// would not fit the registers with two.
int col_tiles(int R, int dtype, int D) {
  const int rb = dtype == PROX_F32 ? 4 : 8;
  return R <= rb || D == 256 ? 1 : 2;
}

size_t smem_bytes(int warps, int D, int rows, int B) {
  const size_t stage = (size_t)kStep * D + kStep * 4;
  return (size_t)warps * (kStages * stage + (size_t)part_floats(rows, D) * 4) + (size_t)(B + 1) * 4;
}

}  // namespace

size_t attend4_part_floats(int D) { return part_floats(16, D); }

cudaError_t setup_attend4() {
  for (int dtype : {PROX_F32, PROX_F16, PROX_BF16})
    for (int D : {64, 128, 256})
      for (int nt : {1, 2}) {
        cudaError_t e =
            cudaFuncSetAttribute(pick(dtype, D, nt), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit - 1024);
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

cudaError_t launch_attend4(const prox_kv4* C, const Attend4Call& c, cudaStream_t s) {
  AttendArgs a;
  a.c = c;
  a.k = C->k, a.ks = C->ks, a.v = C->v, a.vs = C->vs;
  a.pages = C->pages;
  a.heads = C->heads;
  a.page_shift = 0;
  while ((1 << a.page_shift) < C->page) ++a.page_shift;
  a.G = c.Hq / C->heads;
  a.R = a.G * c.Tq;
  const int nt = col_tiles(a.R, c.dtype, C->D);
  const int rb = 8 * nt / (c.dtype == PROX_F32 ? 2 : 1);
  a.blocks = (a.R + rb - 1) / rb;
  a.err = C->err;
  a.part = C->part;
  a.arrived = C->arrived;
  const int per16 = c.dtype == PROX_F32 ? 4 : 8;
  a.q_vec = (reinterpret_cast<uintptr_t>(c.q) & 15) == 0 && c.q_req % per16 == 0 && c.q_tok % per16 == 0 &&
            c.q_head % per16 == 0;
  int warps = kMaxWarps;
  while (smem_bytes(warps, C->D, rb, c.B) > (size_t)kSmemLimit - 1024) --warps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C->num_sms, 1, 1);
  cfg.blockDim = dim3(warps * 32, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes(warps, C->D, rb, c.B);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pick(c.dtype, C->D, nt), a);
}

}  // namespace prox
