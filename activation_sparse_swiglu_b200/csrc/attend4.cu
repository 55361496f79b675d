// Attention of each request's newest tokens over a paged 4-bit cache.
//
// Mathematics.  With K_j = ks_j q^K_j and V_j = vs_j q^V_j (integers q, one
// fp16 scale per token and head) a query row needs
//   t_j = (scale log2 e) ks_j (Q . q^K_j),   o = sum_j 2^(t_j - m) vs_j q^V_j / sum_j 2^(t_j - m),
// so the scales multiply scores and probabilities, never the codes.
//
// One warp keeps the running maximum, sum and output of the rows (query heads
// of one group x new tokens) it works on, and takes up to 64 cache rows a step:
//   S^T = K Q^T   tokens are the M dimension, the rows the N = 8 columns, so a
//                 group of up to 8 heads wastes no tensor work and a code is
//                 decoded once for all of them;
//   O^T = V^T P^T the same, with P^T turned into the B operand by movmatrix.
// K words are A fragments as they lie (the order of d inside a product is
// free, so Q takes the codes' order); V needs pairs of tokens in one register,
// one byte permute per word.  Which token stands in which fragment row is free
// too, and chosen so that the shared-memory reads of K and V meet no bank
// conflict at head_dim 128 and 256 (see token_of).
//
// The kernel is bound by issue before it is by HBM unless decoding is cheap.
// Codes are widened to exact fp16 integers (widen8, 9/8 of an instruction per
// code), so products are exact and sums are fp32.  (A nibble masked out of a
// word is an fp16 subnormal, 5/8 of an instruction; but the tensor core aligns
// products by their factors' exponents, so a large query element or a heavy row
// took the others' bits even where its own codes are 0.  64 ragged requests of the
// 8B-shaped model: 540 instructions per 32 cache rows and 70.6 us with
// subnormals, 662 and 78 with integers.)  Each bf16 or fp32
// query row is scaled by a power of two of its own, so that no head takes bits
// from another; fp32 queries and their probabilities are split into hi + lo
// columns.
// Probabilities times vs are scaled by a power of two per step so that they
// use fp16's range: 11 bits for fp16 and bf16 queries (an fp16 result has no
// more, and the roundings of many rows average out; hi + lo would double the
// columns), 22 for fp32 ones.  Each step's product starts afresh and joins the
// fp32 output with one fused multiply-add, so the tensor core's own sums stay
// short.
//
// Split.  The unit is 32 rows of one (request, kv head).  All units of the
// call are dealt to the CTAs, one per SM, and in a CTA to its warps, as equal
// contiguous ranges, whatever the requests' lengths: no rows are padded, and
// no length is known to the host.  A warp streams its range through its own
// ring of cp.async copies without any block barrier; at the end contexts that
// several warps share are joined through shared memory, and those that several
// CTAs share by the last of them to arrive, always in the same order.
//
// Bound: HBM, (head_dim + 4) bytes per token and kv head, for a few rows per kv
// head (301 MB in 78 us for the 64 requests above, 0.59 of the copy bandwidth);
// issue for more (drafted tokens, prompt chunks: each block of rows decodes the
// cache again).  Where head_dim 128 has two column tiles, 8 to 16 registers a
// thread are spilled.
#include <type_traits>

#include "decode4.h"
#include "quant4.cuh"

namespace prox {
namespace {

using namespace q4;

constexpr int kUnit = 32;    // cache rows that are dealt out together
// What starting a context costs beside its rows, in units (its queries, page
// entries and lengths are fetched, its result is written): contexts are dealt
// out as that many units longer.  (Without it a run of empty or short contexts
// kept one warp busy for twice as long as the others.)
constexpr int kStartUnits = 2;
// Units of a CTA at least: a step for every warp.  Spreading a short context
// over more CTAs saves less than joining them costs.
constexpr int kCtaUnits = 24;
constexpr int kMaxWarps = 12;
constexpr int kSmemLimit = 227 * 1024 - 2048;  // dynamic, beside the joins' tables

// Cache rows of a step, and steps in flight or in use per warp.
constexpr int step_rows(int D) { return D == 256 ? 32 : 64; }
// Warps: as many as the registers of the column tiles allow.
constexpr int warps_of(int D, int nt, int parts) { return D == 256 || (nt == 2 && parts == 1) ? 8 : kMaxWarps; }
constexpr int stages_of(int D, int nt, int parts) { return warps_of(D, nt, parts) == 8 ? 3 : 2; }
constexpr int parts_of(int dtype) { return dtype == PROX_F32 ? 2 : 1; }

struct AttendArgs {
  Attend4Call c;
  const uint8_t* k;
  const uint16_t* ks;
  const uint8_t* v;
  const uint16_t* vs;
  int pages, heads, page_shift;
  int G, R, blocks;  // heads per kv head, rows per kv head, row blocks
  int* err;
  float* part;       // [2 * CTAs] parts that go on in another CTA
  float* warp_part;  // [CTAs * warps] parts that end amid a warp's range
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

// A stage: K rows, V rows, their scales (those as the step uses them lie behind
// the rings).
template <int D>
constexpr int stage_bytes() {
  return step_rows(D) * (D + 4);
}
// One partial result: [rows][D] output, then maxima and sums.
constexpr int part_floats(int rows, int D) { return rows * D + 2 * rows; }

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// A position in the sequence of units: unit c of n of a context (request b, kv
// head, row block).
struct Cursor {
  int b, head, block, c, n, len;
  long long beg;  // number of unit 0
};

// A run of parts of one context that warps [first, last] of a CTA hold.
struct Chain {
  Cursor s;
  int first, last;
  bool from_head;  // the first part is the warp's head
  bool right;      // goes on in the next CTA
};

template <int DT, int D, int NT>
__global__ void __launch_bounds__(warps_of(D, NT, parts_of(DT)) * 32, 1) attend4_kernel(const AttendArgs a) {
  using T = typename Act<DT>::T;
  constexpr int PARTS = parts_of(DT);
  constexpr int RB = 8 * NT / PARTS;   // rows of a block
  constexpr int NC = 2 / PARTS;        // rows a thread has per column tile
  constexpr int KW = D / 32;           // K words per thread and token
  constexpr int VW = D / 64;           // V words per thread and token
  constexpr int PIECES = D / 32;       // 16-byte pieces of a row
  constexpr int ROWS = step_rows(D);
  constexpr int MT = ROWS / 16;        // tiles of 16 tokens
  constexpr int STAGES = stages_of(D, NT, PARTS);
  constexpr int SB = stage_bytes<D>();
  constexpr int SLOT = part_floats(RB, D);
  static_assert(SLOT * 4 <= STAGES * SB, "a part fits a ring");
  const Attend4Call& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;

  extern __shared__ __align__(16) char smem[];
  const uint32_t ring = smem_u32(smem) + warp * (STAGES * SB);
  // the step's scales, ready for use: (ks scale log2 e, vs times its power of two)
  const uint32_t sc_at = smem_u32(smem) + warps * (STAGES * SB) + warp * (ROWS * 8);
  int* pre = reinterpret_cast<int*>(smem + (size_t)warps * (STAGES * SB + ROWS * 8));  // [B + 1]
  __shared__ long long s_scan[33];
  __shared__ Cursor s_head[kMaxWarps], s_tail[kMaxWarps];  // the contexts a warp has parts of
  __shared__ int s_head_at[kMaxWarps], s_tail_at[kMaxWarps];  // 0: none; else kOpen, kDone, kEarly
  __shared__ Chain s_chain[kMaxWarps + 1];
  __shared__ int s_chains, s_last[2];
  __shared__ int2 s_ctas[2];  // the CTAs that share those contexts
  constexpr int kOpen = 1, kDone = 2, kEarly = 3;  // goes on; ends with the range; ends before it

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
    mine += kStartUnits + max(1, (min(max(len, 0), max_len) + kUnit - 1) / kUnit);
  }
  long long total;
  long long at = block_exclusive_scan(mine, s_scan, &total);
  for (int i = rlo; i < rhi; ++i) {
    pre[i] = (int)at;
    at += kStartUnits + max(1, (min(max(c.lens[i], 0), max_len) + kUnit - 1) / kUnit);
  }
  if (threadIdx.x == 0) pre[c.B] = (int)total;  // (the host has seen that B full tables stay below 2^31)
  if (threadIdx.x < kMaxWarps) s_head_at[threadIdx.x] = s_tail_at[threadIdx.x] = 0;
  if (threadIdx.x == 0) s_chains = 0;
  __syncthreads();

  const int H = a.heads * a.blocks;
  // Places count every context's units with its start's.
  const long long places = total * H;
  const int P = (int)min((long long)gridDim.x, (places + kCtaUnits - 1) / kCtaUnits);  // CTAs with work
  if ((int)blockIdx.x >= P) return;

  auto enter = [&](Cursor& s) {  // request s.b, whatever head and block
    s.n = pre[s.b + 1] - pre[s.b] - kStartUnits;
    s.len = min(max(c.lens[s.b], 0), max_len);
  };
  // The unit at a place: the first of its context at the places of the start
  // and the one behind them (no part is left without a unit).
  auto seek = [&](long long place) {
    Cursor s;
    int lo = 0, hi = c.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)pre[mid] * H <= place)
        lo = mid;
      else
        hi = mid;
    }
    s.b = lo;
    enter(s);
    const unsigned r = (unsigned)(place - (long long)pre[lo] * H), m = s.n + kStartUnits;
    const unsigned hb = r / m;
    s.head = hb / a.blocks;
    s.block = hb % a.blocks;
    s.c = max(0, (int)(r - hb * m) - kStartUnits);
    s.beg = (long long)H * (pre[lo] - kStartUnits * lo) + (long long)hb * s.n;
    return s;
  };
  // Three places sought at once, in three lanes: the CTA's first, the warp's
  // first and the one behind its last.
  const long long cta0 = places * blockIdx.x / P, cta1 = places * (blockIdx.x + 1) / P;
  Cursor start;
  long long cb, wb, we;
  {
    const long long all = (long long)H * (total - (long long)kStartUnits * c.B);  // units
    const long long span = cta1 - cta0;  // (places are below 2^31 units times 2^20 row blocks)
    const long long place = lane == 0 ? cta0 : cta0 + span * (warp + (lane == 2)) / warps;
    Cursor s = seek(place < places ? place : places - 1);
    const long long u = place < places ? s.beg + s.c : all;
    cb = __shfl_sync(0xffffffffu, u, 0);
    wb = __shfl_sync(0xffffffffu, u, 1);
    we = __shfl_sync(0xffffffffu, u, 2);
    start.b = __shfl_sync(0xffffffffu, s.b, 1);
    start.head = __shfl_sync(0xffffffffu, s.head, 1);
    start.block = __shfl_sync(0xffffffffu, s.block, 1);
    start.c = __shfl_sync(0xffffffffu, s.c, 1);
    start.n = __shfl_sync(0xffffffffu, s.n, 1);
    start.len = __shfl_sync(0xffffffffu, s.len, 1);
    start.beg = __shfl_sync(0xffffffffu, s.beg, 1);
  }

  // n units on, to the next context at its end (not past the last unit)
  auto advance = [&](Cursor& s, int n) {
    if ((s.c += n) < s.n) return;
    s.beg += s.n;
    s.c = 0;
    if (++s.block < a.blocks) return;
    s.block = 0;
    if (++s.head < a.heads) return;
    s.head = 0;
    if (++s.b < c.B) enter(s);
  };
  // units of the step at s, with `left` to the range's end
  auto units = [&](const Cursor& s, long long left) {
    return (int)min((long long)min(s.n - s.c, ROWS / kUnit), left);
  };

  // ---- producer: the copies of one step, the page lookups one step ahead ------
  constexpr int RPI = 32 / PIECES;  // rows of one copy instruction of the warp
  int pid[MT];
  // whether the step's rows all lie in one page
  auto one_page = [&](const Cursor& s, int n) {
    return (((s.c * kUnit) ^ ((s.c + n) * kUnit - 1)) >> a.page_shift) == 0;
  };
  auto lookup = [&](const Cursor& s, int n) {
    const int32_t* row = c.table + s.b * c.table_stride;
    const int end = min(s.len, (s.c + n) * kUnit), tok0 = s.c * kUnit;
    pid[0] = tok0 < end ? row[tok0 >> a.page_shift] : -1;
    if (one_page(s, n)) return;
#pragma unroll
    for (int h = 1; h < MT; ++h) {
      const int tok = tok0 + 16 * h;
      pid[h] = tok < end ? row[tok >> a.page_shift] : -1;
    }
  };
  const int page_mask = (1 << a.page_shift) - 1;
  const int src_at = lane / PIECES * (D / 2) + lane % PIECES * 16;
  const int k_at = k_piece<D>(lane / PIECES, lane % PIECES), v_at = v_piece<D>(lane / PIECES, lane % PIECES);
  const uint16_t* const sc_src = (lane < 2 ? a.ks : a.vs) + 8 * (lane & 1);  // lanes 0-3: pieces of eight scales
  const int sc_dst = ROWS * D + ((lane >> 1) & 1) * (ROWS * 2) + 16 * (lane & 1);
  auto page_of = [&](int id) {
    if ((unsigned)id < (unsigned)a.pages) return id;
    atomicOr(a.err, PROX_DEVERR_PAGE);
    return 0;
  };
  // 16 rows, h 16 rows into the stage, from row r of the cache
  auto copy16 = [&](const uint8_t* kp, const uint8_t* vp, const uint16_t* sp, int h, uint32_t dst) {
#pragma unroll
    for (int i = 0; i < 16 / RPI; ++i) {
      cp_async16(dst + k_at + (16 * h + RPI * i) * (D / 2), kp + RPI * i * (D / 2));
      cp_async16(dst + v_at + (ROWS + 16 * h + RPI * i) * (D / 2), vp + RPI * i * (D / 2));
    }
    if (lane < 4) cp_async16(dst + sc_dst + 32 * h, sp);
  };
  auto copy = [&](const Cursor& s, int n, uint32_t dst) {
    const int tok0 = s.c * kUnit, end = min(s.len, (s.c + n) * kUnit);
    if (tok0 >= end) return;
    if (one_page(s, n)) {
      const int64_t r = (((int64_t)page_of(pid[0]) * a.heads + s.head) << a.page_shift) + (tok0 & page_mask);
      const uint8_t* kp = a.k + r * (D / 2) + src_at;
      const uint8_t* vp = a.v + r * (D / 2) + src_at;
      const uint16_t* sp = sc_src + r;
#pragma unroll
      for (int h = 0; h < MT; ++h)
        if (h < 2 * n) copy16(kp + h * 8 * D, vp + h * 8 * D, sp + 16 * h, h, dst);
      return;
    }
#pragma unroll
    for (int h = 0; h < MT; ++h) {  // 16 rows lie in one page
      const int tok = tok0 + 16 * h;
      if (tok >= end) break;
      const int64_t r = (((int64_t)page_of(pid[h]) * a.heads + s.head) << a.page_shift) + (tok & page_mask);
      copy16(a.k + r * (D / 2) + src_at, a.v + r * (D / 2) + src_at, sc_src + r, h, dst);
    }
  };

  // ---- the rows' state -------------------------------------------------------
  uint32_t qf[KW][2][NT][2];
  float O[VW][4][2][NT][NC];   // [word][tile][row half][column tile][column]
  float mx[NT][NC], sum[NT][NC];
  float cm = 0.f;              // scale log2(e) / the smallest of the rows' powers of two
  float rf[NT][NC];            // that one / the row's own (fp16 queries enter as they are: 1)
  float vscale = 1.f;          // O's power of two

  auto row_of = [&](int nt, int e) { return PARTS == 2 ? 4 * nt + t : 8 * nt + 2 * t + e; };
  // New token of row r of a kv head (r < 2^20: the product with 1 / G is off by
  // less than the half that keeps it from the next integer).
  const float inv_g = 1.f / (float)a.G;
  auto token_of_row = [&](int r) { return (int)(((float)r + 0.5f) * inv_g); };
  auto out_at = [&](const Cursor& s, int row) {  // element (b, i, h, 0) of row `row` of s's block, -1: none
    const int r = s.block * RB + row, i = token_of_row(r);
    if (r >= a.R) return (int64_t)-1;
    return (((int64_t)s.b * c.Tq + i) * c.Hq + s.head * a.G + (r - i * a.G)) * (int64_t)D;
  };

  auto begin_rows = [&](const Cursor& s) {
    float qv[NT][KW * 8];
    float f[NT];                // of the lane's rows
    float least = 0x1p126f;     // of all rows that are neither zero nor non-finite
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top = 0.f;
      const int r = s.block * RB + (PARTS == 2 ? 4 * nt + (g >> 1) : 8 * nt + g), i0 = token_of_row(r);
      const T* q = static_cast<const T*>(c.q) + s.b * c.q_req + i0 * c.q_tok +
                   (s.head * a.G + (r - i0 * a.G)) * c.q_head;
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        float x[8] = {};
        const int d = D == 64 ? 16 * t + 8 * i : 32 * t + 128 * (i >> 2) + 8 * (i & 3);
        if (r < a.R && s.len > 0) load_vals<DT, 8>(q + d, a.q_vec, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          qv[nt][8 * i + j] = x[j];
          top = max_nan(top, fabsf(x[j]));
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      f[nt] = DT == PROX_F16 ? 1.f : normaliser(top);
      if (top > 0.f && top < INFINITY) least = fminf(least, f[nt]);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
    // The scores of the row with the smallest power (the largest queries) are
    // cm ks z; the other rows' come out larger by their rf's inverse, which the
    // softmax takes off.  (At least 2^-126: a masked score, -inf, stays that.)
    cm = c.scale * 1.4426950408889634f * inv_pow2(DT == PROX_F16 ? 1.f : least);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float own = fmaxf(inv_pow2(f[nt]) * least, 0x1p-126f);
#pragma unroll
      for (int e = 0; e < NC; ++e) rf[nt][e] = DT == PROX_F16 ? 1.f : __shfl_sync(0xffffffffu, own, 8 * t + 4 * e);
    }
    vscale = 1.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = qv[nt][8 * i + j] * f[nt];
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

  // Last token that a row sees (worked out where a step needs it: registers are scarcer).
  auto last_of = [&](const Cursor& s, int nt, int e) {
    const int r = s.block * RB + row_of(nt, e);
    return r < a.R ? s.len - c.Tq + token_of_row(r) : s.len - 1;
  };
  auto step = [&](const Cursor& s, int n, uint32_t st) {
    const int tok0 = s.c * kUnit, end = min(s.len, tok0 + n * kUnit);
    // the step's scales; rows behind the end may hold anything and count as 0
    float ksv[ROWS / 32], vsv[ROWS / 32];
    uint32_t vbits = 0;
#pragma unroll
    for (int i = 0; i < ROWS / 32; ++i) {
      const int row = 32 * i + lane;
      const uint32_t kb = lds16(st + ROWS * D + 2 * row), vb = lds16(st + ROWS * (D + 2) + 2 * row);
      const bool there = tok0 + row < end;
      ksv[i] = there ? __half2float(__ushort_as_half((unsigned short)kb)) * cm : 0.f;
      vsv[i] = there ? __half2float(__ushort_as_half((unsigned short)vb)) : 0.f;
      const uint32_t m = vb & 0x7FFFu;  // magnitudes order like their bits; infinity and NaN do not count
      if (there && m < 0x7C00u) vbits = max(vbits, m);
    }
    vbits = __reduce_max_sync(0xffffffffu, vbits);
    const float vf = normaliser(__half2float(__ushort_as_half((unsigned short)vbits)));
#pragma unroll
    for (int i = 0; i < ROWS / 32; ++i)
      sts64(sc_at + (32 * i + lane) * 8, __float_as_uint(ksv[i]), __float_as_uint(vsv[i] * vf));

    // scores: token rows token_of(g) (+ 8) of MT tiles of 16 tokens
    float S[MT][NT][4];
    const int tr = token_of(g);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t w[2][KW];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * m + 8 * h;  // + tr
        if constexpr (D == 64) {
          const uint2 u = lds64(st + (row + tr) * 32 + 8 * t);
          w[h][0] = u.x, w[h][1] = u.y;
        } else {
#pragma unroll
          for (int p = 0; p < KW / 4; ++p) {
            // (adding 16 m + 8 h rows leaves the pieces' order as it is)
            const uint4 u = lds128(st + k_piece<D>(tr, t + 4 * p) + row * (D / 2));
            w[h][4 * p] = u.x, w[h][4 * p + 1] = u.y, w[h][4 * p + 2] = u.z, w[h][4 * p + 3] = u.w;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        uint32_t ra[4], rb[4];
        widen8(w[0][i], ra);
        widen8(w[1][i], rb);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (i == 0)
            mma_f16(S[m][nt], ra[0], rb[0], ra[1], rb[1], qf[i][0][nt][0], qf[i][0][nt][1], 0.f, 0.f, 0.f, 0.f);
          else
            mma_f16(S[m][nt], ra[0], rb[0], ra[1], rb[1], qf[i][0][nt][0], qf[i][0][nt][1]);
          mma_f16(S[m][nt], ra[2], rb[2], ra[3], rb[3], qf[i][1][nt][0], qf[i][1][nt][1]);
        }
      }
    }
    __syncwarp();  // the scales are there
    float ksc[MT][2], vsc[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 u = lds64(sc_at + (16 * m + 8 * h + tr) * 8);
        ksc[m][h] = __uint_as_float(u.x), vsc[m][h] = __uint_as_float(u.y);
      }

    // running softmax, then P^T as B fragments
    const bool masked = tok0 + ROWS > min(s.len - c.Tq + 1, end);
    uint32_t pf[MT][NT][2];
    float alpha[NT][NC];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float p[MT][2][NC];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < NC; ++e) {
            const float z = PARTS == 2 ? S[m][nt][2 * h] + S[m][nt][2 * h + 1] : S[m][nt][2 * h + e];
            p[m][h][e] = z * ksc[m][h];
          }
      if (masked) {
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          const int last = min(last_of(s, nt, e), end - 1) - tok0 - tr;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (16 * m + 8 * h > last) p[m][h][e] = -INFINITY;
        }
      }
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        float top = -INFINITY;
#pragma unroll
        for (int m = 0; m < MT; ++m) top = fmaxf(top, fmaxf(p[m][0][e], p[m][1][e]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(mx[nt][e], top * rf[nt][e]);
        const float base = top == -INFINITY ? 0.f : top;
        const float al = exp2_fast(mx[nt][e] - base);
        mx[nt][e] = top;
        float add = 0.f;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float y = exp2_fast(fmaf(p[m][h][e], rf[nt][e], -base));
            add += y;
            p[m][h][e] = y * vsc[m][h];
          }
        sum[nt][e] = fmaf(sum[nt][e], al, add);
        alpha[nt][e] = al * (vf * inv_pow2(vscale));
      }
      if (masked) {  // an infinite or NaN scale of a masked row times 0 is NaN
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          const int last = min(last_of(s, nt, e), end - 1) - tok0 - tr;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (16 * m + 8 * h > last) p[m][h][e] = 0.f;
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
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
    vscale = vf;

    // O^T += V^T P^T: thread g has VW words of 8 values of each token
    const uint32_t sv = st + ROWS * (D / 2);
#pragma unroll
    for (int x0 = 0; x0 < VW; x0 += 2) {  // two words at a time (head_dim 64 has one)
      constexpr int XN = VW < 2 ? 1 : 2;
      float part[XN][4][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t vw[4][XN];  // tokens of slots 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int in8 = (q & 1) ? 4 + (t ^ 1) : t, row = 16 * m + 8 * (q >> 1);  // row + in8
          if constexpr (D == 64) {
            vw[q][0] = lds32(sv + (row + in8) * 32 + 4 * g);
          } else if constexpr (D == 128) {
            const uint2 u = lds64(sv + v_piece<D>(in8, g >> 1) + row * (D / 2) + 8 * (g & 1));
            vw[q][0] = u.x, vw[q][1] = u.y;
          } else {
            const uint2 u = lds64(sv + v_piece<D>(in8, g) + row * (D / 2) + 4 * x0);
            vw[q][0] = u.x, vw[q][1] = u.y;
          }
        }
#pragma unroll
        for (int x = 0; x < XN; ++x)
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // values 8x + 4 half .. + 3 of the thread
            uint32_t r0[4], r1[4];
            widen8(prmt(vw[0][x], vw[1][x], half ? 0x7632 : 0x5410), r0);
            widen8(prmt(vw[2][x], vw[3][x], half ? 0x7632 : 0x5410), r1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float(&d0)[4] = part[x][2 * half][nt];
              float(&d1)[4] = part[x][2 * half + 1][nt];
              const uint32_t b0 = pf[m][nt][0], b1 = pf[m][nt][1];
              if (m == 0) {
                mma_f16(d0, r0[0], r0[1], r1[0], r1[1], b0, b1, 0.f, 0.f, 0.f, 0.f);
                mma_f16(d1, r0[2], r0[3], r1[2], r1[3], b0, b1, 0.f, 0.f, 0.f, 0.f);
              } else {
                mma_f16(d0, r0[0], r0[1], r1[0], r1[1], b0, b1);
                mma_f16(d1, r0[2], r0[3], r1[2], r1[3], b0, b1);
              }
            }
          }
      }
#pragma unroll
      for (int x = 0; x < XN; ++x)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < NC; ++e) {
                const float(&d)[4] = part[x][q][nt];
                float& o = O[x0 + x][q][h][nt][e];
                o = fmaf(o, alpha[nt][e], PARTS == 2 ? d[2 * h] + d[2 * h + 1] : d[2 * h + e]);
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
    const float unscale = inv_pow2(vscale);
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
          values(nt, e, unscale, y);
          store_vals<PROX_F32, 8 * VW>(slot + row * D + 8 * VW * g, true, y);
          if (g == 0) slot[RB * D + row] = mx[nt][e], slot[RB * D + RB + row] = l;
          continue;
        }
        const int64_t o = out_at(s, row);
        if (o < 0) continue;
        values(nt, e, l == 0.f ? 0.f : unscale / l, y);
        store_vals<DT, 8 * VW>(static_cast<T*>(c.out) + o + 8 * VW * g, true, y);
        if (c.lse && g == 0) c.lse[o / D] = l == 0.f ? -INFINITY : 0.6931471805599453f * (mx[nt][e] + log2f(l));
      }
  };

  // ---- the warp's range -------------------------------------------------------
  float* warp_parts = a.warp_part + (size_t)blockIdx.x * warps * SLOT;  // of parts that end early
  auto ring_part = [&](int w) { return reinterpret_cast<float*>(smem + (size_t)w * (STAGES * SB)); };
  if (wb < we) {
    Cursor cur = start, pro = cur;
    long long left = we - wb, pleft = left;  // units to compute, to copy
    int pn = units(pro, pleft);
    lookup(pro, pn);
    auto issue = [&](uint32_t dst) {
      if (pleft > 0) {
        copy(pro, pn, dst);
        if ((pleft -= pn) > 0) {
          advance(pro, pn);
          pn = units(pro, pleft);
          lookup(pro, pn);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue(ring + i * SB);
    uint32_t st = ring, next = ring + (STAGES - 1) * SB;  // the stage to read, to fill
    begin_rows(cur);
    while (left > 0) {
      const int n = units(cur, left);
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      issue(next);
      next = st;
      if (cur.len > 0) step(cur, n, st);
      st = st == ring + (STAGES - 1) * SB ? ring : st + SB;
      left -= n;
      const bool ends = cur.c + n == cur.n;
      if (ends || left == 0) {
        float* slot = nullptr;
        if (cur.beg < wb || !ends) {  // a part; at the range's end the ring is free for it
          slot = left > 0 ? warp_parts + (size_t)warp * SLOT : ring_part(warp);
          if (left == 0) {
            cp_async_wait<0>();
            __syncwarp();
          }
          if (lane == 0) {
            if (cur.beg < wb)
              s_head[warp] = cur, s_head_at[warp] = !ends ? kOpen : left > 0 ? kEarly : kDone;
            else
              s_tail[warp] = cur, s_tail_at[warp] = kOpen;
          }
        }
        end_rows(cur, slot);
        if (left > 0) {
          advance(cur, n);
          begin_rows(cur);
        }
      } else {
        advance(cur, n);
      }
    }
  }
  __syncthreads();

  // ---- contexts that several warps or CTAs share -------------------------------
  // A chain ends where a head is done, or with the CTA's last warp that has a
  // part; it begins at the tail before it, or with the CTA's first part.
  if (lane == 0) {
    auto add = [&](const Cursor& s, int last, bool tail_only, bool right) {
      int f = last;
      bool from_head = !tail_only;
      while (from_head && f > 0) {
        int p = f - 1;  // the warp before it with a part
        while (p >= 0 && !s_head_at[p] && !s_tail_at[p]) --p;
        if (p < 0) break;
        from_head = !s_tail_at[p];
        if (from_head && s_head_at[p] != kOpen) {  // that head is of another context
          from_head = true;
          break;
        }
        f = p;
      }
      Chain& ch = s_chain[atomicAdd(&s_chains, 1)];
      ch.s = s;
      ch.first = f;
      ch.last = last;
      ch.from_head = from_head;
      ch.right = right;
    };
    bool more = false;  // a later warp has a head
    for (int w = warp + 1; w < warps; ++w) more |= s_head_at[w] != 0;
    if (s_head_at[warp] >= kDone) add(s_head[warp], warp, false, false);
    if (s_head_at[warp] == kOpen && !more) add(s_head[warp], warp, false, true);
    if (s_tail_at[warp] && !more) add(s_tail[warp], warp, true, true);
  }
  __syncthreads();
  const int chains = s_chains;
  if (chains == 0) return;
  // A thread joins NV runs of four values of one row, D / 16 NV threads a row
  // (neighbours take neighbouring runs).
  auto result = [&](const Cursor& s, int row, int d0, int apart, float top, float l, auto& y, float* to) {
    constexpr int NV = sizeof(y) / sizeof(y[0]);
    if (to) {
#pragma unroll
      for (int j = 0; j < NV; ++j) store_vals<PROX_F32, 4>(to + row * D + d0 + j * apart, true, y[j]);
      if (d0 == 0) to[RB * D + row] = top, to[RB * D + RB + row] = l;
      return;
    }
    const int64_t o = out_at(s, row);
    if (o < 0) return;
    const float f = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[j][i] *= f;
      store_vals<DT, 4>(static_cast<T*>(c.out) + o + d0 + j * apart, true, y[j]);
    }
    if (c.lse && d0 == 0) c.lse[o / D] = l == 0.f ? -INFINITY : 0.6931471805599453f * (top + log2f(l));
  };
  // adds parts with maxima m (-inf: none), sums q and values o to top, l and y
  auto add_parts = [](const auto& m, const auto& q, const auto& o, float* top, float* l, auto& y) {
    constexpr int n = sizeof(m) / sizeof(m[0]), NV = sizeof(y) / sizeof(y[0]);
    float up = *top;
#pragma unroll
    for (int i = 0; i < n; ++i) up = fmaxf(up, m[i]);
    const float base = up == -INFINITY ? 0.f : up;
    float f = exp2_fast(*top - base);
    *top = up;
    *l *= f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) y[j][i] *= f;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      f = exp2_fast(m[i] - base);  // 0 without a visible row (a NaN in the part stays)
      *l = fmaf(q[i], f, *l);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        y[j][0] = fmaf(o[i][j].x, f, y[j][0]), y[j][1] = fmaf(o[i][j].y, f, y[j][1]);
        y[j][2] = fmaf(o[i][j].z, f, y[j][2]), y[j][3] = fmaf(o[i][j].w, f, y[j][3]);
      }
    }
  };
  const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kRuns = D / 16;  // threads of a row, four runs each
  for (int e = threadIdx.x; e < chains * RB * kRuns; e += blockDim.x) {
    const Chain& ch = s_chain[e / (RB * kRuns)];
    const int row = e / kRuns % RB, d0 = e % kRuns * 4;
    auto part = [&](int w) -> const float* {  // the chain's part in warp w, NULL: none
      if (w == ch.first && !ch.from_head) return ring_part(w);
      if (!s_head_at[w]) return nullptr;
      return s_head_at[w] == kEarly ? warp_parts + (size_t)w * SLOT : ring_part(w);
    };
    // (four parts' loads at once: some lie in global memory)
    float top = -INFINITY, l = 0.f, y[4][4] = {};
    for (int w0 = ch.first; w0 <= ch.last; w0 += 4) {
      float m[4], q[4];
      float4 o[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* p = w0 + i <= ch.last ? part(w0 + i) : nullptr;
        m[i] = p ? p[RB * D + row] : -INFINITY;
        q[i] = p ? p[RB * D + RB + row] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[i][j] = p ? *reinterpret_cast<const float4*>(p + row * D + d0 + j * (D / 4)) : zero4;
      }
      add_parts(m, q, o, &top, &l, y);
    }
    const bool left = ch.s.beg < cb;  // began in an earlier CTA
    result(ch.s, row, d0, D / 4, top, l, y,
           left || ch.right ? a.part + (size_t)(2 * blockIdx.x + (left ? 0 : 1)) * SLOT : nullptr);
  }
  bool shared = false;
  for (int i = 0; i < chains; ++i) shared |= s_chain[i].right || s_chain[i].s.beg < cb;
  if (!shared) return;
  // the last CTA to leave its part of a context joins them all
  __threadfence();
  __syncthreads();
  if (threadIdx.x < 2) {  // the context from the left, the one that goes on to the right
    int found = -1;
    for (int i = 0; i < chains; ++i) {
      const bool left = s_chain[i].s.beg < cb;
      if (threadIdx.x == 0 ? left : !left && s_chain[i].right) found = i;
    }
    if (found >= 0) {
      const Cursor& s = s_chain[found].s;
      const long long first = (long long)H * pre[s.b] +
                              (long long)(s.head * a.blocks + s.block) * (s.n + kStartUnits) +
                              kStartUnits;  // the place behind the context's start
      const int c0 = (int)(((first + 1) * P - 1) / places), c1 = (int)(((first + s.n) * P - 1) / places);
      s_ctas[threadIdx.x] = make_int2(c0, c1);
      if (atomicAdd(a.arrived + c0, 1) == c1 - c0)
        a.arrived[c0] = 0;  // for the next call
      else
        found = -1;
    }
    s_last[threadIdx.x] = found;
  }
  __syncthreads();
  if (s_last[0] < 0 && s_last[1] < 0) return;
  __threadfence();
  constexpr int kSlices = RB * (D / 4);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (s_last[k] < 0) continue;
    const int c0 = s_ctas[k].x, c1 = s_ctas[k].y;
    for (int e = threadIdx.x; e < kSlices; e += blockDim.x) {
      const int row = e / (D / 4), d = e % (D / 4) * 4;
      float top = -INFINITY, l = 0.f, y[1][4] = {};
      for (int i0 = c0; i0 <= c1; i0 += 8) {
        float m[8], q[8];
        float4 o[8][1];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool there = i0 + i <= c1;
          const float* p = a.part + (size_t)(2 * (i0 + i) + (i0 + i == c0 ? 1 : 0)) * SLOT;
          m[i] = there ? __ldcg(p + RB * D + row) : -INFINITY;
          q[i] = there ? __ldcg(p + RB * D + RB + row) : 0.f;
          o[i][0] = there ? __ldcg(reinterpret_cast<const float4*>(p + row * D + d)) : zero4;
        }
        add_parts(m, q, o, &top, &l, y);
      }
      result(s_chain[s_last[k]].s, row, d, 4, top, l, y, nullptr);
    }
  }
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
  const int rb = 8 / parts_of(dtype);
  return R <= rb || D == 256 ? 1 : 2;
}

size_t smem_bytes(int warps, int D, int nt, int dtype, int B) {
  const size_t rows = step_rows(D);
  return (size_t)warps * (stages_of(D, nt, parts_of(dtype)) * rows * (D + 4) + rows * 8) + (size_t)(B + 1) * 4;
}

}  // namespace

size_t attend4_part_floats(int D) { return part_floats(D == 256 ? 8 : 16, D); }
int attend4_warps() { return kMaxWarps; }

cudaError_t setup_attend4() {
  for (int dtype : {PROX_F32, PROX_F16, PROX_BF16})
    for (int D : {64, 128, 256})
      for (int nt : {1, 2}) {
        cudaError_t e =
            cudaFuncSetAttribute(pick(dtype, D, nt), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
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
  const int rb = 8 * nt / parts_of(c.dtype);
  a.blocks = (a.R + rb - 1) / rb;
  a.err = C->err;
  a.part = C->part;
  a.warp_part = C->warp_part;
  a.arrived = C->arrived;
  const int per16 = c.dtype == PROX_F32 ? 4 : 8;
  a.q_vec = (reinterpret_cast<uintptr_t>(c.q) & 15) == 0 && c.q_req % per16 == 0 && c.q_tok % per16 == 0 &&
            c.q_head % per16 == 0;
  int warps = warps_of(C->D, nt, parts_of(c.dtype));
  while (smem_bytes(warps, C->D, nt, c.dtype, c.B) > (size_t)kSmemLimit) --warps;  // (large batches)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C->num_sms, 1, 1);
  cfg.blockDim = dim3(warps * 32, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes(warps, C->D, nt, c.dtype, c.B);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pick(c.dtype, C->D, nt), a);
}

}  // namespace prox
