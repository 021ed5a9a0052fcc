// Tiles of BM x 128 with eight waves in a ring of LDS stages.
//
// Waves: two along the rows, two along the columns, and two that share each
// 64-k step (each takes one MFMA's depth, 32). Sharing the step halves what a
// wave reads from LDS for the same MFMAs: a 128 x 128 step then costs 64 KiB
// of LDS reads, 512 clocks, as long as its MFMAs, where eight waves with
// tiles of 64 x 32 would read 96 KiB. The two halves' sums meet once, in LDS,
// after the loop, each wave finishing half of the rows.
//
// The ring: S - 1 steps are in flight. A step waits for its own wave's copies
// of that stage, passes one barrier (which publishes everyone's copies and
// tells that the stage read a step ago is free), issues the copies into that
// stage, reads its fragments and multiplies. Copies past the end of the sum
// are issued masked, so that every wait counts the same number of loads.
#pragma once

#include "dense.h"
#include "gemm_pingpong.h"

namespace pgemm {
namespace dense {

using fast::b_swz;
using fast::read_a;
using fast::read_b;
using fast::static_for;
using fast::wait_vmcnt;

template <int DT, int FORM, bool GATED, int BM, int S>
__global__ void __launch_bounds__(512, S == 2 ? 4 : 2) tile_kernel(Args a) {
  constexpr int BN = 128, BK = 64;
  constexpr bool A_KC = FORM != kGrad, B_KC = FORM == kRowsNK;
  static_assert(A_KC || BM == 128, "the transposed rows of A are 256 bytes in LDS");
  constexpr int MB = BM / 32;           // 16-row blocks of a wave
  constexpr int AL = BM / 64, L = AL + 2; // copies of a wave: of A, and in all
  constexpr int ROW_OC = 256;
  typedef typename fast::Frag<DT>::t frag_t;
  __shared__ __attribute__((aligned(1024))) uint8_t sA0[BM * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t sA1[BM * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t sA2[S > 2 ? BM * 128 : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t sA3[S > 3 ? BM * 128 : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t sB0[BN * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t sB1[BN * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t sB2[S > 2 ? BN * 128 : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t sB3[S > 3 ? BN * 128 : 16];
  auto stage_a = [&](auto c) __attribute__((always_inline)) -> uint8_t* {
    constexpr int C = decltype(c)::value;
    return C == 0 ? sA0 : C == 1 ? sA1 : C == 2 ? sA2 : sA3;
  };
  auto stage_b = [&](auto c) __attribute__((always_inline)) -> uint8_t* {
    constexpr int C = decltype(c)::value;
    return C == 0 ? sB0 : C == 1 ? sB1 : C == 2 ? sB2 : sB3;
  };

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kw = wave >> 2, wm = (wave >> 1) & 1, wn = wave & 1;
  const int g = lane >> 4, s16 = lane & 15, q = s16 >> 2, qt = s16 & 3;

  // tiles of one piece follow each other; each XCD takes one stretch of the sequence
  const int per = a.n_m * a.n_n, total = per * a.split, share = (total + 7) / 8;
  const int u = (int)(blockIdx.x & 7) * share + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= share || u >= total) return;
  const int piece = u / per;
  int pm, pn, first, nk;
  grouped_tile(u - piece * per, a.n_m, a.n_n, 8, &pm, &pn);
  piece_steps(a.K, a.split, piece, &first, &nk);
  const int m0 = pm * BM, n0 = pn * (GATED ? BN / 2 : BN);
  const int mrem = a.M - m0, nrem = a.N - n0, K = a.K;

  // ---- copies: block wave + 8j of 1 KiB. kc: eight rows of 128 bytes, chunk c of row r at c ^ (r & 7);
  // oc: four k-rows of 256 bytes, chunk c of row k at c ^ b_swz(k) (k + 32 has the same swizzle).
  const int a_row = A_KC ? 8 * wave + (lane >> 3) : 4 * wave + (lane >> 4);
  const int a_chunk = A_KC ? (lane & 7) ^ (lane >> 3) : (lane & 15) ^ b_swz<2, ROW_OC>(a_row);
  const int b_row = B_KC ? 8 * wave + (lane >> 3) : 4 * wave + (lane >> 4);
  const int b_chunk = B_KC ? (lane & 7) ^ (lane >> 3) : (lane & 15) ^ b_swz<2, ROW_OC>(b_row);
  // Gated: of each 64 columns of the tile the first 32 are gate columns, the others their up columns.
  // N x K: a block of eight rows lies in one of them; K x N: a lane's chunk does.
  const int b_up = GATED ? (B_KC ? (wave >> 2) & 1 : (b_chunk >> 2) & 1) : 0;
  auto b_col = [&](int j) __attribute__((always_inline)) { // tile column of the lane's row (kc) or chunk (oc)
    const int r = B_KC ? b_row + 64 * j : 8 * b_chunk;
    return GATED ? (r >> 6) * 32 + (r & 31) : r;
  };
  const uint16_t* const A = A_KC ? a.a + m0 * a.lda : a.a + m0;
  const uint16_t* const B = (B_KC ? a.b + n0 * a.ldb : a.b + n0) + (GATED && B_KC ? b_up * a.half : 0);
  auto copy = [&](int step, auto stage) __attribute__((always_inline)) {
    const int k0 = (first + step) * BK;
    const int krem = step < nk ? K - k0 : 0;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(A + (A_KC ? (int64_t)k0 : k0 * a.lda));
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(B + (B_KC ? (int64_t)k0 : k0 * a.ldb));
    uint8_t *pa = stage_a(stage) + 1024 * wave, *pb = stage_b(stage) + 1024 * wave;
    static_for<AL>([&](auto jc) __attribute__((always_inline)) {
      constexpr int J = decltype(jc)::value;
      const int r = a_row + (A_KC ? 64 : 32) * J;
      const bool ok = A_KC ? (r < mrem) & (8 * a_chunk < krem) : (r < krem) & (8 * a_chunk < mrem);
      const uint32_t at = (uint32_t)r * (uint32_t)(a.lda * 2) + 16u * (uint32_t)a_chunk;
      load16_to_lds(ra, pa + 8192 * J, ok ? at : kOOB);
    });
    static_for<2>([&](auto jc) __attribute__((always_inline)) {
      constexpr int J = decltype(jc)::value;
      uint32_t at;
      bool ok;
      if constexpr (B_KC) {
        const int r = b_col(J);
        ok = (r < nrem) & (8 * b_chunk < krem);
        at = (uint32_t)r * (uint32_t)(a.ldb * 2) + 16u * (uint32_t)b_chunk;
      } else {
        const int r = b_row + 32 * J, n = b_col(0);
        ok = (r < krem) & (n < nrem);
        at = (uint32_t)r * (uint32_t)(a.ldb * 2) + 2u * (uint32_t)n + (GATED ? 2u * (uint32_t)a.half * (uint32_t)b_up : 0u);
      }
      load16_to_lds(rb, pb + 8192 * J, ok ? at : kOOB);
    });
  };

  // ---- fragments: the column order of grouped.h, which leaves a lane eight consecutive columns
  int a_off[MB], b_off[4];
  {
    const int k = 8 * g + q;
    auto oc_at = [&](int i) __attribute__((always_inline)) {
      return 16 * ((4 * (i >> 1) + qt) ^ b_swz<2, ROW_OC>(k)) + 8 * ((i + qt) & 1);
    };
#pragma unroll
    for (int i = 0; i < MB; ++i)
      a_off[i] = A_KC ? ((wm * (BM / 2) + 16 * i + s16) * 128 + 16 * (g ^ (s16 & 7))) ^ (64 * kw)
                      : (k + 32 * kw) * ROW_OC + (oc_at(i) ^ (wm * 128));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = wn * 64 + 32 * (i >> 1) + 8 * q + 4 * ((i + q) & 1) + qt;
      b_off[i] = B_KC ? (r * 128 + 16 * (g ^ (r & 7))) ^ (64 * kw) : (k + 32 * kw) * ROW_OC + (oc_at(i) ^ (wn * 128));
    }
  }

  floatx4_t acc[MB][4];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

  static_for<S - 1>([&](auto c) __attribute__((always_inline)) { copy(decltype(c)::value, c); });
  for (int s = 0; s < nk; s += S) {
    static_for<S>([&](auto c) __attribute__((always_inline)) {
      constexpr int C = decltype(c)::value;
      if (s + C < nk) {
        wait_vmcnt<(S - 2) * L>();
        pp::barrier_raw();
        copy(s + C + S - 1, std::integral_constant<int, (C + S - 1) % S>{});
        const uint8_t *pa = stage_a(c), *pb = stage_b(c);
        frag_t af[MB], bf[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (B_KC) bf[j] = read_a<DT>(pb + b_off[j], nullptr);
          else bf[j] = read_b<DT, ROW_OC>(pb + b_off[j]);
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          if constexpr (A_KC) af[i] = read_a<DT>(pa + a_off[i], nullptr);
          else af[i] = read_b<DT, ROW_OC>(pa + a_off[i]);
        }
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = mfma(bf[j], af[i], acc[i][j]);
      }
    });
  }

  // ---- the two halves of the steps: each wave gives the rows it does not finish
  wait_vmcnt<0>(); // the masked copies write LDS too
  __syncthreads();
  constexpr int HB = MB / 2;
  {
    uint8_t* part = (wave & 2 ? (wave & 1 ? sB1 : sB0) : (wave & 1 ? sA1 : sA0)) + (BM * 64) * kw; // HB * 4 KiB a wave
    floatx4_t* to = reinterpret_cast<floatx4_t*>(part);
#pragma unroll
    for (int i = 0; i < HB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) to[(i * 4 + j) * 64 + lane] = kw ? acc[i][j] : acc[HB + i][j];
  }
  __syncthreads();
  {
    const uint8_t* part = (wave & 2 ? (wave & 1 ? sB1 : sB0) : (wave & 1 ? sA1 : sA0)) + (BM * 64) * (kw ^ 1);
    const floatx4_t* from = reinterpret_cast<const floatx4_t*>(part);
#pragma unroll
    for (int i = 0; i < HB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const floatx4_t o = from[(i * 4 + j) * 64 + lane], mine = kw ? acc[HB + i][j] : acc[i][j];
        acc[i][j] = kw ? o + mine : mine + o; // the first half's sum first
      }
  }

  // ---- output
  const bool odd = (g & 1) != 0;
  const Epilogue<DT, GATED> epilogue(a);
  auto row_of = [&](int i) __attribute__((always_inline)) {
    const int b = kw * HB + i;
    return m0 + wm * (BM / 2) + (A_KC ? 16 * b + s16 : 32 * (b >> 1) + 8 * q + 4 * ((b + q) & 1) + qt);
  };
  auto eight = [&](int i, int P, float* v) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      v[r] = odd ? acc[i][2 * P + 1][r] : acc[i][2 * P][r];
      v[4 + r] = odd ? acc[i][2 * P][r] : acc[i][2 * P + 1][r];
    }
  };
  if (a.split > 1) {
    const int64_t ld = part_ld(a, GATED);
#pragma unroll
    for (int P = 0; P < 2; ++P) {
      const int n = n0 + (GATED ? wn * 32 : wn * 64 + 32 * P) + 8 * g;
      if (n >= a.N) continue;
      float* col = a.part + (int64_t)piece * a.M * ld + n + (GATED && P ? ld / 2 : 0);
#pragma unroll
      for (int i = 0; i < HB; ++i) {
        const int m = row_of(i);
        float v[8];
        eight(i, P, v);
        if (m < a.M) {
          float* to = col + m * ld;
          *reinterpret_cast<floatx4_t*>(to) = floatx4_t{v[0], v[1], v[2], v[3]};
          *reinterpret_cast<floatx4_t*>(to + 4) = floatx4_t{v[4], v[5], v[6], v[7]};
        }
      }
    }
    return;
  }
#pragma unroll
  for (int P = 0; P < (GATED ? 1 : 2); ++P) {
    const int n = n0 + (GATED ? wn * 32 : wn * 64 + 32 * P) + 8 * g;
    float bv[8], bu[8];
    epilogue.bias_of(n, bv, bu);
#pragma unroll
    for (int i = 0; i < HB; ++i) {
      const int m = row_of(i);
      float v[8], w[8];
      eight(i, P, v);
      if constexpr (GATED) eight(i, 1, w);
      if (m < a.M && n < a.N) epilogue.finish(m, n, v, w, bv, bu);
    }
  }
}

} // namespace dense
} // namespace pgemm
