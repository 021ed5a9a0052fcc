// Tiles of BM x 128 with eight waves in a ring of LDS stages.
//
// Waves: two along the rows, two along the columns, and two that share each
// 64-k step (each takes one MFMA's depth, 32). Sharing the step halves what a
// wave reads from LDS for the same MFMAs: a 128 x 128 step then costs 64 KiB
// of LDS reads, 512 clocks, as long as its MFMAs, where eight waves with
// tiles of 64 x 32 would read 96 KiB. The two halves' sums meet once, in LDS,
// after the loop.
//
// The ring: S - 1 steps are in flight. A step waits for its own wave's copies
// of the next stage, passes one barrier (which publishes everyone's copies and
// tells that the stage multiplied a step ago is free), issues the copies into
// that stage, and multiplies while it reads the next step's fragments into a
// second set of registers. With two stages (two workgroups to a CU, whose
// phases overlap instead) there is one set. Copies past the end of the sum are
// issued masked, so that every wait counts the same number of loads.
//
// LDS reads and MFMAs bound a step together: 0.53 us on every CU, 1.02 PFLOP/s
// at 2.4 GHz's 2.5; a tile's first copies and its output add some 3 us. 512 x
// 4096 x 8192 in two pieces: 36 us (MFMA busy 0.37), 6 more to join them.
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

constexpr int ring_bytes(int rows, int stages) { return stages * (rows + 128) * 128; }

// The tile of workgroup `block` of a's grid, with `ring` its LDS.
template <int DT, int FORM, bool GATED, int BM, int S>
__device__ __attribute__((always_inline)) inline void run_tile(const Args& a, int block, uint8_t* ring) {
  constexpr int BN = 128, BK = 64;
  constexpr bool A_KC = FORM != kGrad, B_KC = FORM == kRowsNK;
  static_assert(A_KC || BM == 128, "the transposed rows of A are 256 bytes in LDS");
  constexpr int MB = BM / 32;           // 16-row blocks of a wave
  constexpr int AL = BM / 64, L = AL + 2; // copies of a wave: of A, and in all
  constexpr int ROW_OC = 256;
  typedef typename fast::Frag<DT>::t frag_t;
  constexpr int A_BYTES = BM * 128, STAGE = A_BYTES + BN * 128; // A's tile, then B's
  static_assert(S * STAGE == ring_bytes(BM, S), "the ring is its stages");
  auto stage_a = [&](auto c) __attribute__((always_inline)) -> uint8_t* { return ring + decltype(c)::value * STAGE; };
  auto stage_b = [&](auto c) __attribute__((always_inline)) -> uint8_t* { return stage_a(c) + A_BYTES; };

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kw = wave >> 2, wm = (wave >> 1) & 1, wn = wave & 1;
  const int g = lane >> 4, s16 = lane & 15, q = s16 >> 2, qt = s16 & 3;

  // tiles of one piece follow each other; each XCD takes one stretch of the sequence
  const int per = a.n_m * a.n_n, total = per * a.split, share = (total + 7) / 8;
  const int u = (block & 7) * share + (block >> 3);
  if ((block >> 3) >= share || u >= total) return;
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
  auto copy_one = [&](int step, auto stage, auto which) __attribute__((always_inline)) { // the wave's copy `which` of a step
    constexpr int J = decltype(which)::value;
    const int k0 = (first + step) * BK, krem = step < nk ? K - k0 : 0;
    const uint32_t to = (uint32_t)(uintptr_t)PGEMM_LDS(uint8_t, stage_a(stage)) + 1024 * wave;
    uint32_t at;
    bool ok;
    if constexpr (J < AL) {
      const int r = a_row + (A_KC ? 64 : 32) * J;
      ok = A_KC ? (r < mrem) & (8 * a_chunk < krem) : (r < krem) & (8 * a_chunk < mrem);
      at = (uint32_t)r * (uint32_t)(a.lda * 2) + 16u * (uint32_t)a_chunk;
      copy16(rsrc_words(A + (A_KC ? (int64_t)k0 : k0 * a.lda)), to + 8192 * J, ok ? at : kOOB);
    } else {
      constexpr int JB = J - AL;
      if constexpr (B_KC) {
        const int r = b_col(JB);
        ok = (r < nrem) & (8 * b_chunk < krem);
        at = (uint32_t)r * (uint32_t)(a.ldb * 2) + 16u * (uint32_t)b_chunk;
      } else {
        const int r = b_row + 32 * JB, n = b_col(0);
        ok = (r < krem) & (n < nrem);
        at = (uint32_t)r * (uint32_t)(a.ldb * 2) + 2u * (uint32_t)n + (GATED ? 2u * (uint32_t)a.half * (uint32_t)b_up : 0u);
      }
      copy16(rsrc_words(B + (B_KC ? (int64_t)k0 : k0 * a.ldb)), to + A_BYTES + 8192 * JB, ok ? at : kOOB);
    }
  };
  auto copy = [&](int step, auto stage) __attribute__((always_inline)) {
    static_for<L>([&](auto j) __attribute__((always_inline)) { copy_one(step, stage, j); });
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

  struct Frags { frag_t a[MB], b[4]; };
  auto read_one_a = [&](Frags& f, auto stage, auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value;
    if constexpr (A_KC) f.a[i] = read_a<DT>(stage_a(stage) + a_off[i], nullptr);
    else f.a[i] = read_b<DT, ROW_OC>(stage_a(stage) + a_off[i]);
  };
  auto read_all_b = [&](Frags& f, auto stage) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (B_KC) f.b[j] = read_a<DT>(stage_b(stage) + b_off[j], nullptr);
      else f.b[j] = read_b<DT, ROW_OC>(stage_b(stage) + b_off[j]);
    }
  };
  auto read = [&](Frags& f, auto stage) __attribute__((always_inline)) {
    read_all_b(f, stage);
    static_for<MB>([&](auto i) __attribute__((always_inline)) { read_one_a(f, stage, i); });
  };
  auto multiply_row = [&](const Frags& f, auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value;
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = mfma(f.b[j], f.a[i], acc[i][j]);
  };
  static_for<S - 1>([&](auto c) __attribute__((always_inline)) { copy(decltype(c)::value, c); });
  if constexpr (S == 2) {
    for (int s = 0; s < nk; s += 2) {
      static_for<2>([&](auto c) __attribute__((always_inline)) {
        constexpr int C = decltype(c)::value;
        if (s + C < nk) {
          wait_vmcnt<0>();
          pp::barrier_raw();
          copy(s + C + 1, std::integral_constant<int, C ^ 1>{});
          Frags f;
          read(f, c);
          static_for<MB>([&](auto i) __attribute__((always_inline)) { multiply_row(f, i); });
        }
      });
    }
  } else {
    constexpr int U = S % 2 ? 2 * S : S; // steps after which stages and register sets repeat
    Frags f[2];
    wait_vmcnt<(S - 2) * L>();
    pp::barrier_raw();
    read(f[0], std::integral_constant<int, 0>{});
    for (int s = 0; s < nk; s += U) {
      static_for<U>([&](auto c) __attribute__((always_inline)) {
        constexpr int C = decltype(c)::value;
        if (s + C < nk) {
          wait_vmcnt<(S - 3) * L>(); // the next step's copies
          pp::barrier_raw();
          // between the rows' MFMAs: the copies into the freed stage, the next step's fragments
          std::integral_constant<int, (C + S - 1) % S> freed;
          std::integral_constant<int, (C + 1) % S> next;
          static_for<MB>([&](auto i) __attribute__((always_inline)) {
            constexpr int I = decltype(i)::value;
            multiply_row(f[C % 2], i);
            __builtin_amdgcn_sched_barrier(0);
            static_for<L * (I + 1) / MB - L * I / MB>([&](auto j) __attribute__((always_inline)) {
              copy_one(s + C + S - 1, freed, std::integral_constant<int, L * I / MB + decltype(j)::value>{});
            });
            if constexpr (I == 0) read_all_b(f[(C + 1) % 2], next);
            read_one_a(f[(C + 1) % 2], next, i);
            __builtin_amdgcn_sched_barrier(0);
          });
        }
      });
    }
  }

  // ---- output. Both halves of the steps go to LDS as fp32 rows (in two turns where LDS holds half of them) and come
  // back added, eight columns a thread and 16 threads (gated: 8) to a row, so that a row's stores are 256 bytes side by
  // side: from the MFMA's layout they would be 64 (4099 x 2057 x 1021, whose rows lie at odd addresses: 52 us, now 45).
  // The 16-byte chunk c of row r lies at c ^ (r & 15).
  wait_vmcnt<0>(); // the masked copies write LDS too
  constexpr int TURNS = 2 * BM * 512 > S * STAGE ? 2 : 1, ROWS = BM / TURNS, HB = MB / TURNS; // rows of a turn
  static_assert(2 * ROWS * 512 <= S * STAGE && MB % TURNS == 0, "both halves of a turn's rows fit the stages");
  const Epilogue<DT, GATED> epilogue(a);
  constexpr int LANES = GATED ? 8 : 16; // to a row
  const int c8 = tid % LANES, n = n0 + 8 * c8;
  const int col = GATED ? (c8 >> 2) * 64 + 8 * (c8 & 3) : 8 * c8; // tile column of the thread's first; up: 32 further
  float bv[8], bu[8];
  if (a.split <= 1) epilogue.bias_of(n, bv, bu);
  auto at = [&](int half, int r, int chunk) __attribute__((always_inline)) -> floatx4_t* { // stages follow each other in `ring`
    return reinterpret_cast<floatx4_t*>(ring + half * (ROWS * 512) + r * 512 + 16 * (chunk ^ (r & 15)));
  };
  // A turn's rows: of each wave row wm its blocks turn * HB .. + HB - 1
#pragma unroll
  for (int turn = 0; turn < TURNS; ++turn) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < HB; ++i) {
      const int r = wm * (16 * HB) + (A_KC ? 16 * i + s16 : 32 * (i >> 1) + 8 * q + 4 * ((i + q) & 1) + qt);
#pragma unroll
      for (int j = 0; j < 4; ++j) // columns 64 wn + 32 (j / 2) + 8 g + 4 ((j + g) & 1) ..
        *at(kw, r, 16 * wn + 8 * (j >> 1) + 2 * g + ((j + g) & 1)) = acc[turn * HB + i][j];
    }
    __syncthreads();
#pragma unroll
    for (int pass = 0; pass < ROWS * LANES / 512; ++pass) {
      const int r = tid / LANES + pass * (512 / LANES);
      const int m = m0 + (r / (16 * HB)) * (BM / 2) + turn * (16 * HB) + r % (16 * HB);
      float v[8], w[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const floatx4_t x = *at(0, r, col / 4 + h) + *at(1, r, col / 4 + h);
        floatx4_t y = x;
        if constexpr (GATED) y = *at(0, r, col / 4 + 8 + h) + *at(1, r, col / 4 + 8 + h);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[4 * h + k] = x[k];
          w[4 * h + k] = y[k];
        }
      }
      if (m >= a.M || n >= a.N) continue;
      if (a.split > 1) {
        const int64_t ld = part_ld(a, GATED);
        float* to = a.part + ((int64_t)piece * a.M + m) * ld + n;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          *reinterpret_cast<floatx4_t*>(to + 4 * h) = floatx4_t{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
          if constexpr (GATED)
            *reinterpret_cast<floatx4_t*>(to + ld / 2 + 4 * h) = floatx4_t{w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]};
        }
      } else {
        act::with_path(epilogue.k, [&](auto path) __attribute__((always_inline)) {
          epilogue.template finish<decltype(path)::value>(m, n, v, w, bv, bu);
        });
      }
    }
  }
}

template <int DT, int FORM, bool GATED, int BM, int S>
__global__ void __launch_bounds__(512, S == 2 ? 4 : 2) tile_kernel(Args a) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[ring_bytes(BM, S)];
  run_tile<DT, FORM, GATED, BM, S>(a, blockIdx.x, ring);
}

// Both products of a backward pass in one launch, dx in form FORM: their tiles fill the card together, which the tiles
// of one alone often do not (forward and backward of 4477 x 1552 x 1988: 156 us, in two launches 179; 802 x 1400 x 96: 27 and
// 35 us; 4099 x 2057 x 1021: 145 and 153). The first `head` workgroups (a multiple of 8) have the longer sums. Four stages
// rather than five: the unrolled steps of both products then fit the scalar registers.
template <int DT, int FORM, int S>
__global__ void __launch_bounds__(512, S == 2 ? 4 : 2) both_kernel(Args dx, Args dw, int head, int dw_first) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[ring_bytes(128, S)];
  const bool first = (int)blockIdx.x < head;
  const int block = first ? blockIdx.x : blockIdx.x - head;
  if (first == (dw_first != 0)) run_tile<DT, kGrad, false, 128, S>(dw, block, ring);
  else run_tile<DT, FORM, false, 128, S>(dx, block, ring);
}

} // namespace dense
} // namespace pgemm
