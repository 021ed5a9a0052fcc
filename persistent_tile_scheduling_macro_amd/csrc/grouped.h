// Products of rows that are sorted by expert. offsets[e] .. offsets[e+1]-1
// are the rows of expert e, known only on the device:
//   rows form:      c[r][n] = sum_k a[r][k] * b[e(r)][k][n]     (the forward product, and the
//                   gradient of its rows with the other layout of b)
//   gradient form:  c[e][i][j] = sum over e's rows r of a[r][i] * b[r][j]
// Sums are fp32, in an order that the sizes fix, rounded once: along k, in the few-row bodies eight waves' shares of it
// and in a split gradient the pieces, joined in order. Each output tile (or piece) is one workgroup's, so a result does
// not depend on which workgroup runs when.
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
  int most_tiles; // no ascending bounds give more tiles
  int split;   // gradient form: pieces an expert's rows are cut into
  float* part; // split > 1: their sums, [E][split][M][N rounded up to 8]
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

// The last n < 8 elements of a row of `len`, or any 8, the rest zeros. A row of eight is read as its
// last eight, moved: loads of single elements would wait for each other.
__device__ inline u32x4 load_upto(const uint16_t* p, int n, int len) {
  if (n >= 8) return moe::load8<moe::kAnyAddress>(p);
  if (n <= 0) return u32x4{0, 0, 0, 0};
  return len >= 8 ? moe::shift_down(moe::load8<moe::kAnyAddress>(p + n - 8), 8 - n) : moe::load_part(p, n);
}

template <int DT>
__device__ inline u32x4 pack8(floatx4_t a, floatx4_t b) {
  const float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return moe::pack<DT>(f);
}

// Piece `piece` of an expert's `rows` rows, whole steps of 64: its first row and its rows.
__device__ inline void piece_rows(const Args& a, int rows, int piece, int* from, int* count) {
  const int steps = (rows + 63) / 64;
  const int lo = (int)((int64_t)steps * piece / a.split) * 64, hi = (int)((int64_t)steps * (piece + 1) / a.split) * 64;
  *from = min(lo, rows);
  *count = min(hi, rows) - *from;
}
__device__ inline int64_t part_row(const Args& a, int e, int piece, int m) {
  return (((int64_t)e * a.split + piece) * a.M + m) * ((a.N + 7) & ~7);
}

// The body for operands of any alignment: 128 x 128 tile, four waves of
// 64 x 64, steps of 64 k. Chunks of eight elements go through registers (the
// direct load to LDS wants 16-byte addresses): step s+1 is loaded while step
// s is multiplied, then written to the other LDS stage. A load never waits
// for another or branches: its address is kept inside the matrix (a chunk over
// a row's end is read as the row's last eight elements), and what it then has
// wrong is put right on the way to LDS, in the steps and tiles at an edge
// only: positions moved, zeros past the sum's end. (Reading the edge element
// by element took ten times an inner tile's time, and with it the call's.)
// One step takes 1.0 us alone on a CU, 1.25 us for two workgroups together:
// the chain of loads, LDS and MFMAs of a wave, with one or two waves a SIMD.
// Odd sizes cost a second pass through the address unit (16-byte loads at odd
// addresses run at 25 bytes a clock and CU against 60 at multiples of four):
// 30000 rows, eight experts, 1023 x 1023 120 us, 1024 x 1024 in the ping-pong
// body 64 us. Eight waves of 64 x 32 (5 to 10% faster for N x K weights, 12%
// slower for K x N) and loads two steps ahead (level or slower) were not kept.
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
  float* part = nullptr;
  int gap_at = 0, gap = 0; // rows of no expert: from row gap_at on they lie `gap` rows further
  if constexpr (GRAD) {
    const int n_m = (a.M + BM - 1) / BM, per = n_m * a.n_n;
    const int e = blockIdx.x / (per * a.split), u = blockIdx.x - e * per * a.split, piece = u / per;
    int pm, pn, first, rows, from;
    grouped_tile(u - piece * per, n_m, a.n_n, 8, &pm, &pn);
    expert_rows(a, e, &first, &rows);
    piece_rows(a, rows, piece, &from, &K);
    M = a.M;
    m0 = pm * BM;
    n0 = pn * BN;
    A = a.a + (first + from) * a.lda;
    B = a.b + (first + from) * a.ldb;
    C = a.c + (int64_t)e * a.M * a.N;
    if (a.split > 1) part = a.part + part_row(a, e, piece, 0);
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
  const int nk = (K + BK - 1) / BK, N = a.N;

  // A thread's chunks of an operand. Rows along k: 128 rows x 8 chunks; else 64 k-rows x 16 chunks.
  u32x4 ra[4], rb[4];
  auto load_operand = [&](u32x4 (&r)[4], const uint16_t* p, int64_t ld, int o0, int O, int k0, auto kc, auto first)
                          __attribute__((always_inline)) {
    if constexpr (decltype(kc)::value) {
      const int k = min(k0 + 8 * (tid & 7), K - 8);
      if (K < 8) { // fewer than eight in a row
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = load_upto(p + min(o0 + (tid >> 3) + 32 * j, O - 1) * ld, tid & 7 ? 0 : K, K);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = moe::load8<moe::kAnyAddress>(p + min(o0 + (tid >> 3) + 32 * j, O - 1) * ld + k);
      }
    } else {
      const int o = min(o0 + 8 * (tid & 15), O - 8);
      if (O < 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = load_upto(p + min(k0 + (tid >> 4) + 16 * j, K - 1) * ld, tid & 15 ? 0 : O, O);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) // a sum of few rows (the first step is all) leaves out what lies past them
          if (!decltype(first)::value || 16 * j < K) r[j] = moe::load8<moe::kAnyAddress>(p + min(k0 + (tid >> 4) + 16 * j, K - 1) * ld + o);
      }
    }
  };
  auto write_operand = [&](u32x4 (&r)[4], uint8_t* s, int o0, int O, int k0, auto kc) __attribute__((always_inline)) {
    const bool last = k0 + BK > K;
    if constexpr (decltype(kc)::value) {
      if (last) {
        const int left = K - k0 - 8 * (tid & 7);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (left <= 0) r[j] = u32x4{0, 0, 0, 0};
          else if (left < 8 && K >= 8) r[j] = moe::shift_down(r[j], 8 - left);
        }
      }
    } else {
      if (o0 + 128 > O && O >= 8) { // what lies past O is used for outputs past O only
        const int left = O - o0 - 8 * (tid & 15);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (left > 0 && left < 8) r[j] = moe::shift_down(r[j], 8 - left);
      }
      if (last) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k0 + (tid >> 4) + 16 * j >= K) r[j] = u32x4{0, 0, 0, 0};
      }
    }
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
  auto load = [&](int step, auto first) __attribute__((always_inline)) {
    load_operand(ra, A, a.lda, m0, M, step * BK, AKC{}, first);
    load_operand(rb, B, a.ldb, n0, N, step * BK, BKC{}, first);
  };
  auto write = [&](int step) __attribute__((always_inline)) {
    write_operand(ra, sA[step & 1], m0, M, step * BK, AKC{});
    write_operand(rb, sB[step & 1], n0, N, step * BK, BKC{});
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
    load(0, std::true_type{});
    write(0);
    __syncthreads();
    for (int s = 0; s < nk; ++s) {
      const bool more = s + 1 < nk;
      if (more) load(s + 1, std::false_type{});
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
      if (more) write(s + 1);
      __syncthreads();
    }
  }

  // Output: fp32 sums of a piece go out from the registers; rounded rows are put together in LDS first,
  // so that 16 lanes store 256 bytes of a row (four lanes and 64 bytes otherwise, which at odd
  // addresses costs most of the time of a product of few rows).
  const bool odd = (g & 1) != 0;
  uint8_t* sC = sA[0];
  static_assert(sizeof(sA) == BM * BN * 2, "the tile's rounded output fits A's stages");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = s16 >> 2;
    const int m = wm * 64 + (A_KC ? 16 * i + s16 : 32 * (i >> 1) + 8 * q + 4 * ((i + q) & 1) + (s16 & 3));
#pragma unroll
    for (int P = 0; P < 2; ++P) {
      const floatx4_t x = odd ? acc[i][2 * P + 1] : acc[i][2 * P], y = odd ? acc[i][2 * P] : acc[i][2 * P + 1];
      const int chunk = wn * 8 + 4 * P + g;
      if (GRAD && part) {
        float* to = part + (int64_t)(m0 + m) * ((N + 7) & ~7) + n0 + 8 * chunk;
        if (m0 + m < M && n0 + 8 * chunk < N) {
          *reinterpret_cast<floatx4_t*>(to) = x;
          *reinterpret_cast<floatx4_t*>(to + 4) = y;
        }
      } else {
        *reinterpret_cast<u32x4*>(sC + m * 256 + 16 * (chunk ^ (m & 15))) = pack8<DT>(x, y);
      }
    }
  }
  if (GRAD && part) return;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = (tid >> 4) + 16 * j, m = m0 + r, n = n0 + 8 * (tid & 15);
    if (m < M && n < N)
      moe::store_row<moe::kAnyAddress>(C + (int64_t)(m < gap_at ? m : m + gap) * N, n, N,
                            *reinterpret_cast<const u32x4*>(sC + r * 256 + 16 * ((tid & 15) ^ (r & 15))));
  }
}

// c[e] = the sum of its pieces' sums, rounded. Eight columns a thread; G threads share their pieces (every
// G-th), and the first adds the shares in order.
template <int DT, int G>
__global__ void __launch_bounds__(256) join_pieces_kernel(Args a) {
  __shared__ floatx4_t share[G > 1 ? 2 * 256 : 1];
  const int tid = threadIdx.x, w = tid % (256 / G), group = tid / (256 / G);
  const int chunks = (a.N + 7) / 8;
  const int64_t i = (int64_t)blockIdx.x * (256 / G) + w, at = i / chunks;
  const bool live = at < (int64_t)a.E * a.M;
  const int n = (int)(i % chunks) * 8, e = (int)(at / a.M), m = (int)(at % a.M);
  floatx4_t x = {0.f, 0.f, 0.f, 0.f}, y = x;
  if (live) {
#pragma unroll 4
    for (int s = group; s < a.split; s += G) {
      const float* p = a.part + part_row(a, e, s, m) + n;
      x += *reinterpret_cast<const floatx4_t*>(p);
      y += *reinterpret_cast<const floatx4_t*>(p + 4);
    }
  }
  if constexpr (G > 1) {
    share[tid] = x;
    share[256 + tid] = y;
    __syncthreads();
    if (group) return;
#pragma unroll
    for (int o = 1; o < G; ++o) {
      x += share[o * (256 / G) + w];
      y += share[256 + o * (256 / G) + w];
    }
  }
  if (live) moe::store_row<moe::kAnyAddress>(a.c + at * a.N, n, a.N, pack8<DT>(x, y));
}

// Bodies: this file's, grouped_pp.h's, and grouped_few.h's (rows form) for
// 16 or 32 rows at once, with one or two column blocks of N x K weights, and for
// the weight gradient of few rows.
enum Body : int { kAnyAlignment, kPingPong, kFew16, kFew16Wide, kFew32Wide, kFewGrad };
typedef void (*kernel_fn)(Args);
kernel_fn pick_f16(int body, bool grad, bool nk);
kernel_fn pick_bf16(int body, bool grad, bool nk);
kernel_fn join_f16(bool shared); // eight threads to a sum, or one
kernel_fn join_bf16(bool shared);

} // namespace grouped
} // namespace pgemm
