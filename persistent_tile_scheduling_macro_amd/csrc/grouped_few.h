// The grouped products' body for experts of few rows: every byte of the
// experts' matrices is read once for up to 32 rows, and that reading bounds
// it. A workgroup takes one expert's 16 * MB rows and 16 * BLK columns; its
// eight waves take the steps of the sum in turn (so together they read
// stretches of a matrix row) and join their fp32 sums in LDS, in a fixed
// order. Loads go to registers, D steps ahead.
//
// The MFMA wants row or column s in lane (g, s), but loads in that layout
// make every lane its own request (consecutive lanes lie a row apart), a
// quarter of the address unit's rate or less; measured, they took 64-76 us for
// 32 x 2048 x 1536 weights. So loads run along the rows, eight lanes to a
// 128-byte line, and each wave turns its step's operands in its own LDS:
//   x, N x K weights: 16-byte chunks of rows, read back as MFMA operands;
//     steps of 64 k (x of K x N weights: 32 k).
//   K x N weights need no turn: lane (g, s) reads four columns, 4s.., of rows
//     8g .. 8g+7 (128 bytes of a row over 16 lanes), and half-word permutes
//     pair the rows into the operands of four column blocks: block t's column
//     s is 4s + t.
// 256 rows over 32 experts, 2048 x 1536 bf16 N x K: 32 us, 6.3 TB/s, the rate of
// plain reads. Any even address is taken. The weights are the MFMA's first operand, so
// that a lane's four outputs are columns of one row.
#pragma once

#include "grouped.h"

namespace pgemm {
namespace grouped {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

constexpr int kFewWaves = 8;

// A wave's LDS copy of 16 rows of a step, ROW bytes (128 or 64) each: the
// swizzle keeps both the row-wise writes and the operand reads free of bank
// conflicts.
template <int ROW>
__device__ inline int turn_at(int row, int chunk) {
  return row * ROW + 16 * (chunk ^ (ROW == 128 ? row & 7 : 2 * ((row >> 2) & 1)));
}

template <int DT, bool NK, int MB, int BLK>
__global__ void __launch_bounds__(kFewWaves * 64, 4) grouped_few_kernel(Args a) {
  static_assert(NK || BLK == 4, "K x N: four columns a lane");
  constexpr int STEP = NK ? 64 : 32, H = STEP / 32;
  constexpr int ROW = STEP * 2, LPR = ROW / 16, RPL = 64 / LPR; // bytes of a step's row, lanes to a row, rows of a load
  constexpr int L = 16 / RPL;                                   // loads of 16 rows
  constexpr int D = 2; // steps in flight; three or four (fewer waves a SIMD) were 5 to 15% slower
  typedef typename fast::Frag<DT>::t frag_t;
  typedef typename Traits<DT>::out_t out_t;
  constexpr int TURN = 16 * ROW * (MB + (NK ? BLK : 0)), JOIN = BLK * MB * 64 * 16; // LDS bytes of a wave
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kFewWaves * (TURN > JOIN ? TURN : JOIN)];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, s = lane & 15;
  Place p;
  if (!place_tile<16 * MB>(a, blockIdx.x, &p)) return;
  const int m0 = p.m * 16 * MB, n0 = p.n * 16 * BLK, N = a.N, K = a.K;
  if (p.e == a.E) { // rows of no expert are zeros
    for (int i = tid; i < 16 * MB * 16 * BLK; i += kFewWaves * 64) {
      const int m = m0 + i / (16 * BLK), n = n0 + i % (16 * BLK);
      if (m < p.rows && n < N) a.c[(int64_t)(m < p.first ? m : m + a.R - p.rows) * N + n] = 0;
    }
    return;
  }

  // Rows past the last and columns past N repeat the last one; K x N lanes at
  // the edge start at N - 4. What is read twice is stored once.
  const int row = lane / LPR, chunk = lane % LPR;
  const uint16_t* x[MB * L];
#pragma unroll
  for (int i = 0; i < MB * L; ++i) x[i] = a.a + (p.first + min(m0 + RPL * i + row, p.rows - 1)) * a.lda + 8 * chunk;
  constexpr int WP = NK ? BLK * L : 1;
  const uint16_t* w[WP];
#pragma unroll
  for (int i = 0; i < WP; ++i)
    w[i] = a.b + p.e * a.b_expert +
           (NK ? min(n0 + RPL * i + row, N - 1) * a.ldb + 8 * chunk : 8 * g * a.ldb + min(n0 + 4 * s, N - 4));

  struct Slot { // what a step reads
    u32x4 x[MB * L];
    u32x4 w[NK ? BLK * L : 4]; // K x N: rows 2i and 2i + 1, four columns each
  };
  auto load = [&](Slot& t, int step) __attribute__((always_inline)) {
    const int64_t k0 = (int64_t)step * STEP;
    if constexpr (NK) {
#pragma unroll
      for (int i = 0; i < BLK * L; ++i) t.w[i] = moe::load8<moe::kAnyAddress>(w[i] + k0);
    } else {
      const uint16_t* r = w[0] + k0 * a.ldb;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x2 lo = *reinterpret_cast<const u32x2_any*>(r + 2 * i * a.ldb);
        const u32x2 hi = *reinterpret_cast<const u32x2_any*>(r + (2 * i + 1) * a.ldb);
        t.w[i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
      }
    }
#pragma unroll
    for (int i = 0; i < MB * L; ++i) t.x[i] = moe::load8<moe::kAnyAddress>(x[i] + k0);
  };
  floatx4_t acc[MB][BLK];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int c = 0; c < BLK; ++c) acc[b][c] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  uint8_t *turn_x = lds + wave * TURN, *turn_w = turn_x + 16 * ROW * MB;
  auto wave_fence = [&]() __attribute__((always_inline)) { // LDS serves a wave in order: only the compiler has to be held
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  auto multiply = [&](const Slot& t) __attribute__((always_inline)) {
    wave_fence(); // the last step's reads come first
#pragma unroll
    for (int i = 0; i < MB * L; ++i) *reinterpret_cast<u32x4*>(turn_x + turn_at<ROW>(RPL * i + row, chunk)) = t.x[i];
    if constexpr (NK) {
#pragma unroll
      for (int i = 0; i < BLK * L; ++i) *reinterpret_cast<u32x4*>(turn_w + turn_at<ROW>(RPL * i + row, chunk)) = t.w[i];
    }
    wave_fence();
#pragma unroll
    for (int h = 0; h < H; ++h) {
      frag_t xf[MB];
#pragma unroll
      for (int b = 0; b < MB; ++b) xf[b] = *reinterpret_cast<const frag_t*>(turn_x + turn_at<ROW>(16 * b + s, 4 * h + g));
#pragma unroll
      for (int c = 0; c < BLK; ++c) {
        frag_t f;
        if constexpr (NK) {
          f = *reinterpret_cast<const frag_t*>(turn_w + turn_at<ROW>(16 * c + s, 4 * h + g));
        } else {
          u32x4 v;
#pragma unroll
          for (int i = 0; i < 4; ++i) // column c of rows 2i and 2i + 1
            v[i] = __builtin_amdgcn_perm(t.w[i][2 + c / 2], t.w[i][c / 2], c % 2 ? 0x07060302u : 0x05040100u);
          f = __builtin_bit_cast(frag_t, v);
        }
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[b][c] = mfma(f, xf[b], acc[b][c]);
      }
    }
  };

  const int whole = K / STEP;
  const int mine = (whole - wave + kFewWaves - 1) / kFewWaves; // steps wave, wave + 8, ... (none if not positive)
  if (mine > 0) {
    auto at = [&](int i) __attribute__((always_inline)) { return wave + kFewWaves * min(i, mine - 1); };
    Slot t[D];
#pragma unroll
    for (int j = 0; j < D; ++j) load(t[j], at(j));
    for (int i = 0; i < mine; i += D) {
#pragma unroll
      for (int j = 0; j < D; ++j) {
        if (i + j < mine) multiply(t[j]);
        load(t[j], at(i + j + D)); // past the range the last one again, not used
      }
    }
  }
  if (whole * STEP < K && wave == whole % kFewWaves) { // the partial step, zeros past K
    const int k0 = whole * STEP;
    Slot t;
    if constexpr (NK) {
#pragma unroll
      for (int i = 0; i < BLK * L; ++i) t.w[i] = load_upto(w[i] + k0, K - k0 - 8 * chunk, K);
    } else {
      const int left = K - k0 - 8 * g;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint16_t* r = w[0] + (k0 + 2 * i) * a.ldb;
        u32x2 lo = {0, 0}, hi = {0, 0};
        if (2 * i < left) lo = *reinterpret_cast<const u32x2_any*>(r);
        if (2 * i + 1 < left) hi = *reinterpret_cast<const u32x2_any*>(r + a.ldb);
        t.w[i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
      }
    }
#pragma unroll
    for (int i = 0; i < MB * L; ++i) t.x[i] = load_upto(x[i] + k0, K - k0 - 8 * chunk, K);
    multiply(t);
  }

  __syncthreads(); // every wave is through with its part of the LDS
  floatx4_t* join = reinterpret_cast<floatx4_t*>(lds);
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int c = 0; c < BLK; ++c) join[(wave * BLK * MB + c * MB + b) * 64 + lane] = acc[b][c];
  __syncthreads();
  for (int i = tid; i < BLK * MB * 64; i += kFewWaves * 64) {
    floatx4_t v = join[i];
#pragma unroll
    for (int o = 1; o < kFewWaves; ++o) v += join[o * BLK * MB * 64 + i];
    const int l = i & 63, b = (i >> 6) % MB, c = (i >> 6) / MB;
    const int m = m0 + 16 * b + (l & 15);
    if (m >= p.rows) continue;
    uint16_t* row = a.c + (int64_t)(p.first + m) * N;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int at = 4 * (l >> 4) + r; // position in the block
      int n, from;                     // its column, and the first one that this position stores
      if constexpr (NK) {
        n = from = n0 + 16 * c + at;
      } else {
        from = n0 + 4 * at;
        n = min(from, N - 4) + c;
      }
      if (from < N && n >= from) row[n] = __builtin_bit_cast(uint16_t, to_out(v[r], (out_t*)nullptr));
    }
  }
}

// The gradient form for experts of few rows: writing c bounds it, and what
// keeps the writes going is many tiles in flight. So steps are 32 rows (one
// MFMA's depth), LDS holds one step or the rounded tile (32 KiB) and a wave
// 64 x 32 of the 128 x 128 tile: three workgroups of eight waves to a CU, where
// the any-alignment body has two of four. 27 experts of some five rows,
// 3224 x 2968 bf16 (516 MB of c): 147 us there,
// 106 us here. The rule that chooses it knows the mean only, and a step's loads are waited for: an expert with far more
// rows than the mean holds the call up (64 experts, 1024 x 1024, 96 rows each 41 us; 5514 of the 6144 rows in one 121 us).
template <int DT>
__global__ void __launch_bounds__(512, 6) grad_few_kernel(Args a) {
  constexpr int BM = 128, BN = 128, BK = 32, ROW = 256;
  typedef typename fast::Frag<DT>::t frag_t;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[BM * BN * 2];
  uint8_t *sA = lds, *sB = lds + BK * ROW;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave >> 2, wn = wave & 3;
  const int g = lane >> 4, q = (lane & 15) >> 2, qt = lane & 3;
  const int M = a.M, N = a.N, n_m = (M + BM - 1) / BM, per = n_m * a.n_n;
  const int e = blockIdx.x / per;
  int pm, pn, first, K;
  grouped_tile(blockIdx.x - e * per, n_m, a.n_n, 8, &pm, &pn);
  expert_rows(a, e, &first, &K);
  const int m0 = pm * BM, n0 = pn * BN;

  // a thread's chunk of a step: row tid / 16, eight elements of each operand
  const int kr = tid >> 4, m_at = m0 + 8 * (tid & 15), n_at = n0 + 8 * (tid & 15);
  const int at = kr * ROW + 16 * ((tid & 15) ^ b_swz<2, ROW>(kr));
  const int k = 8 * g + q; // fragment row; oc order of grouped.h
  const int frag_at = k * ROW + 16 * (qt ^ b_swz<2, ROW>(k)) + 8 * (qt & 1);
  auto block = [](int i) __attribute__((always_inline)) { return 64 * (i >> 1) + 8 * (i & 1); };

  floatx4_t acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < K; k0 += BK) {
    u32x4 x = {0, 0, 0, 0}, y = x;
    if (k0 + kr < K) {
      x = load_upto(a.a + (first + k0 + kr) * a.lda + m_at, M - m_at, M);
      y = load_upto(a.b + (first + k0 + kr) * a.ldb + n_at, N - n_at, N);
    }
    if (k0) __syncthreads();
    *reinterpret_cast<u32x4*>(sA + at) = x;
    *reinterpret_cast<u32x4*>(sB + at) = y;
    __syncthreads();
    frag_t bf[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) bf[j] = read_b<DT, ROW>(sB + ((frag_at ^ block(j)) ^ (wn * 64)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const frag_t af = read_b<DT, ROW>(sA + ((frag_at ^ block(i)) ^ (wm * 128)));
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma(bf[j], af, acc[i][j]);
    }
  }
  __syncthreads();
  const bool odd = (g & 1) != 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = wm * 64 + 32 * (i >> 1) + 8 * q + 4 * ((i + q) & 1) + qt, chunk = wn * 4 + g;
    *reinterpret_cast<u32x4*>(lds + m * 256 + 16 * (chunk ^ (m & 15))) =
        odd ? pack8<DT>(acc[i][1], acc[i][0]) : pack8<DT>(acc[i][0], acc[i][1]);
  }
  __syncthreads();
  uint16_t* C = a.c + (int64_t)e * M * N;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = kr + 32 * j, m = m0 + r;
    if (m < M && n_at < N)
      moe::store_row<moe::kAnyAddress>(C + (int64_t)m * N, n_at, N,
                                       *reinterpret_cast<const u32x4*>(lds + r * 256 + 16 * ((tid & 15) ^ (r & 15))));
  }
}

} // namespace grouped
} // namespace pgemm
