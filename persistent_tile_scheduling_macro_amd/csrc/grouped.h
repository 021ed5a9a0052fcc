// Products of rows that are sorted by expert. offsets[e] .. offsets[e+1]-1
// are the rows of expert e, known only on the device:
//   rows form:      c[r][n] = sum_k a[r][k] * b[e(r)][k][n]     (the forward product, and the
//                   gradient of its rows with the other layout of b)
//   gradient form:  c[e][i][j] = sum over e's rows r of a[r][i] * b[r][j]
// Sums are fp32, in the order of k, rounded once; each output tile is one
// workgroup's, so a result does not depend on which workgroup runs when.
//
// An operand is "k-contiguous" (kc: its rows run along the sum) or
// "outer-contiguous" (oc: its rows run along an output axis). LDS tiles and
// fragment reads are those of the fast GEMM body (gemm_fast.h): kc as rows of
// 128 bytes read 16 bytes a lane, oc as k-rows read by the transposing LDS
// reads, both with that body's swizzles.
#pragma once

#include "gemm_fast.h"
#include "moe_rows.h"

namespace pgemm {
namespace grouped {

using fast::b_swz;
using fast::read_a;
using fast::read_b;
using moe::u32x4;

struct Args {
  const uint16_t *a, *b;
  int64_t lda, ldb; // distance of two rows
  int64_t b_expert; // rows form: elements of one expert's matrix
  const int* offsets;
  uint16_t* c;
  int R, E; // rows, experts
  int M;    // gradient form: rows of c[e] (the rows form has an expert's number of rows)
  int N;    // columns of c
  int K;    // rows form: length of the sum (the gradient form has an expert's number of rows)
  int n_n;  // tiles along N
};

// Rows of expert e, bounds kept inside [0, R] whatever offsets hold; e == E
// stands for the rows of no expert (before the first and behind the last).
__device__ inline void expert_rows(const Args& a, int e, int* first, int* rows) {
  const int lo = min(max(a.offsets[e == a.E ? 0 : e], 0), a.R);
  const int hi = min(max(a.offsets[e == a.E ? e : e + 1], lo), a.R);
  *first = lo;
  *rows = e == a.E ? a.R - (hi - lo) : hi - lo;
}

struct Place {
  int e, first, rows; // expert (E: the rows of none), its first row (or the length of the gap they leave out) and rows
  int m, n;           // tile of it
};

// Tile `block` of the rows form. Experts follow each other, each with
// ceil(rows / BM) x n_n tiles in the grouped order; each XCD (block mod 8)
// takes one stretch of that sequence, so that the tiles that share an
// expert's rows and matrix share an L2. The grid is larger than the sequence
// (only the device knows its length); false: no tile.
template <int BM>
__device__ inline bool place_tile(const Args& a, int block, Place* p) {
  const int lane = threadIdx.x & 63;
  auto tiles_of = [&](int e) {
    int first, rows;
    if (e > a.E) return 0;
    expert_rows(a, e, &first, &rows);
    return (rows + BM - 1) / BM * a.n_n;
  };
  int total = 0;
  for (int e0 = 0; e0 <= a.E; e0 += 64) total += tiles_of(e0 + lane);
#pragma unroll
  for (int d = 32; d; d >>= 1) total += __shfl_xor(total, d);
  const int per = (total + 7) / 8, u = (block & 7) * per + (block >> 3);
  if ((block >> 3) >= per || u >= total) return false;
  int before = 0;
  for (int e0 = 0; e0 <= a.E; e0 += 64) {
    const int t = tiles_of(e0 + lane);
    int s = t;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(s, d);
      if (lane >= d) s += v;
    }
    const uint64_t hit = __ballot(before + s > u);
    if (hit) {
      const int l = (int)__builtin_ctzll(hit);
      const int e = __builtin_amdgcn_readfirstlane(e0 + l);
      const int at = u - before - __builtin_amdgcn_readfirstlane(__shfl(s - t, l));
      expert_rows(a, e, &p->first, &p->rows);
      p->e = e;
      p->first = __builtin_amdgcn_readfirstlane(p->first);
      p->rows = __builtin_amdgcn_readfirstlane(p->rows);
      grouped_tile(__builtin_amdgcn_readfirstlane(at), (p->rows + BM - 1) / BM, a.n_n, 8, &p->m, &p->n);
      return true;
    }
    before += __shfl(s, 63);
  }
  return false;
}

// n (up to 8) elements at any even address, the rest zeros.
__device__ inline u32x4 load_upto(const uint16_t* p, int n) {
  if (n >= 8) return moe::load8<false>(p);
  if (n > 0) return moe::load_part(p, n);
  return u32x4{0, 0, 0, 0};
}

template <int DT>
__device__ inline u32x4 pack8(floatx4_t a, floatx4_t b) {
  const float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return moe::pack<DT>(f);
}

// The body for operands of any alignment: 128 x 128 tile, four waves of
// 64 x 64, steps of 64 k. Chunks of eight elements go through registers (the
// direct load to LDS wants 16-byte addresses): step s+1 is loaded while step
// s is multiplied, then written to the other LDS stage.
template <int DT, bool GRAD, bool NK>
__global__ void __launch_bounds__(256, 2) grouped_kernel(Args a) {
  constexpr int BM = 128, BN = 128, BK = 64;
  constexpr bool A_KC = !GRAD, B_KC = !GRAD && NK;
  constexpr int B_ROW = 256; // bytes of an oc row in LDS
  typedef typename fast::Frag<DT>::t frag_t;
  __shared__ __attribute__((aligned(1024))) uint8_t sA[2][BM * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t sB[2][BN * 128];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave >> 1, wn = wave & 1;
  const int g = lane >> 4, s16 = lane & 15;

  int M, K, m0, n0;
  const uint16_t *A, *B;
  uint16_t* C;
  int gap_at = 0, gap = 0; // rows of no expert: from row gap_at on they lie `gap` rows further
  if constexpr (GRAD) {
    const int n_m = (a.M + BM - 1) / BM, per_expert = n_m * a.n_n;
    const int e = blockIdx.x / per_expert;
    int pm, pn, first;
    grouped_tile(blockIdx.x - e * per_expert, n_m, a.n_n, 8, &pm, &pn);
    expert_rows(a, e, &first, &K);
    M = a.M;
    m0 = pm * BM;
    n0 = pn * BN;
    A = a.a + first * a.lda;
    B = a.b + first * a.ldb;
    C = a.c + (int64_t)e * a.M * a.N;
  } else {
    Place p;
    if (!place_tile<BM>(a, blockIdx.x, &p)) return;
    M = p.rows;
    K = p.e == a.E ? 0 : a.K;
    m0 = p.m * BM;
    n0 = p.n * BN;
    A = a.a + p.first * a.lda;
    B = a.b + (p.e == a.E ? 0 : p.e) * a.b_expert;
    C = a.c;
    if (p.e == a.E) {
      gap_at = p.first;
      gap = a.R - p.rows;
    } else {
      C += (int64_t)p.first * a.N;
    }
  }
  const int nk = (K + BK - 1) / BK;

  u32x4 ra[4], rb[4];
  // operand rows along k: 128 rows x 8 chunks; else 64 k-rows x 16 chunks
  auto load_operand = [&](u32x4 (&r)[4], const uint16_t* p, int64_t ld, int o0, int O, int k0, auto kc)
                          __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (decltype(kc)::value) {
        const int o = o0 + (tid >> 3) + 32 * j, k = k0 + 8 * (tid & 7);
        r[j] = load_upto(p + o * ld + k, o < O ? K - k : 0);
      } else {
        const int k = k0 + (tid >> 4) + 16 * j, o = o0 + 8 * (tid & 15);
        r[j] = load_upto(p + k * ld + o, k < K ? O - o : 0);
      }
    }
  };
  auto write_operand = [&](const u32x4 (&r)[4], uint8_t* s, auto kc) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      int at;
      if constexpr (decltype(kc)::value) {
        const int o = (tid >> 3) + 32 * j;
        at = o * 128 + 16 * ((tid & 7) ^ (o & 7));
      } else {
        const int k = (tid >> 4) + 16 * j;
        at = k * B_ROW + 16 * ((tid & 15) ^ b_swz<2, B_ROW>(k));
      }
      *reinterpret_cast<u32x4*>(s + at) = r[j];
    }
  };
  typedef std::integral_constant<bool, A_KC> AKC;
  typedef std::integral_constant<bool, B_KC> BKC;
  auto load = [&](int step) __attribute__((always_inline)) {
    load_operand(ra, A, a.lda, m0, M, step * BK, AKC{});
    load_operand(rb, B, a.ldb, n0, a.N, step * BK, BKC{});
  };
  auto write = [&](int stage) __attribute__((always_inline)) {
    write_operand(ra, sA[stage], AKC{});
    write_operand(rb, sB[stage], BKC{});
  };

  // Fragment offsets. The n-position s16 of block nb is wave column
  // 32*(nb/2) + 8q + 4*((nb+q)&1) + r with s16 = 4q + r, so that a lane ends
  // up with eight consecutive columns of blocks 2P and 2P+1. oc rows of A use
  // the same order for output rows.
  int a_off[4], b_off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = s16 >> 2, qt = s16 & 3, k = 8 * g + q;
    const int kc_col = 32 * (i >> 1) + 8 * q + 4 * ((i + q) & 1) + qt;
    const int oc_at = 16 * ((4 * (i >> 1) + qt) ^ b_swz<2, B_ROW>(k)) + 8 * ((i + qt) & 1);
    a_off[i] = A_KC ? (wm * 64 + 16 * i + s16) * 128 + 16 * (g ^ (s16 & 7))
                    : k * B_ROW + (oc_at ^ (wm * 128));
    const int r = wn * 64 + kc_col;
    b_off[i] = B_KC ? r * 128 + 16 * (g ^ (r & 7)) : k * B_ROW + (oc_at ^ (wn * 128));
  }
  auto frag = [&](const uint8_t* s, int off, int kk, auto kc) __attribute__((always_inline)) -> frag_t {
    if constexpr (decltype(kc)::value) return read_a<DT>(s + (off ^ (64 * kk)), nullptr);
    else return read_b<DT, B_ROW>(s + off + kk * 32 * B_ROW);
  };

  floatx4_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

  if (nk > 0) {
    load(0);
    write(0);
    __syncthreads();
    for (int s = 0; s < nk; ++s) {
      const bool more = s + 1 < nk;
      if (more) load(s + 1);
      const uint8_t *pa = sA[s & 1], *pb = sB[s & 1];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        frag_t af[4], bf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) af[i] = frag(pa, a_off[i], kk, AKC{});
#pragma unroll
        for (int i = 0; i < 4; ++i) bf[i] = frag(pb, b_off[i], kk, BKC{});
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = mfma(bf[j], af[i], acc[i][j]);
      }
      if (more) write((s + 1) & 1);
      __syncthreads();
    }
  }

  const int n = n0 + wn * 64 + 8 * g;
  const bool odd = (g & 1) != 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = s16 >> 2;
    const int m = m0 + wm * 64 + (A_KC ? 16 * i + s16 : 32 * (i >> 1) + 8 * q + 4 * ((i + q) & 1) + (s16 & 3));
    if (m >= M) continue;
    uint16_t* row = C + (int64_t)(m < gap_at ? m : m + gap) * a.N;
#pragma unroll
    for (int P = 0; P < 2; ++P) {
      const floatx4_t x = acc[i][2 * P], y = acc[i][2 * P + 1];
      if (n + 32 * P < a.N) moe::store_row<false>(row, n + 32 * P, a.N, odd ? pack8<DT>(y, x) : pack8<DT>(x, y));
    }
  }
}

// Bodies: this file's, grouped_pp.h's, and grouped_few.h's (rows form) for
// 16 or 32 rows at once, with one or two column blocks of N x K weights.
enum Body : int { kAnyAlignment, kPingPong, kFew16, kFew16Wide, kFew32Wide };
typedef void (*kernel_fn)(Args);
kernel_fn pick_f16(int body, bool grad, bool nk);
kernel_fn pick_bf16(int body, bool grad, bool nk);

} // namespace grouped
} // namespace pgemm
