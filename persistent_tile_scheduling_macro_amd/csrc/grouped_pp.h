// The grouped products' body for operands at 16-byte addresses and experts of
// many rows: the ping-pong 256 x 256 tile of gemm_pingpong.h (eight waves of
// 128 x 64 in two groups of opposite phases, copies that write LDS directly),
// persistent over tiles that only the device can count.
//
// What differs from that body:
// * A workgroup lays out the tile sequence itself: a table in LDS of the
//   tiles before each expert, from which it looks up its tiles.
// * The gradient form sums over an expert's rows, so its tiles have different
//   lengths, and its A is outer-contiguous: k-rows of 128 elements per half,
//   read by the transposing LDS reads like a K x N B.
// * A tile without a sum (an expert or a gap without rows to sum over) runs
//   two steps whose copies are all masked and read zeros.
//
// 32768 rows over 32 experts, 4096 x 2048 bf16, product and both gradients in turn: with N x K matrices 490 us (1120
// TFLOP/s), with K x N 520 us (1060), weight gradient 583 us (940), either operand as its rows; its tiles sum 16 steps
// only and store 128 KiB each, 537 MB in all. (Under the profiler's trace 535, 571 and 643 us, MFMAs busy 0.59, 0.55 and
// 0.46 at the clock that power allows; torch's product of 8192^3 runs at 1222 TFLOP/s on the same card.)
// With fewer tiles than workgroups, in a launch's last part round, and with a grid of no multiple of 8, tiles are
// taken in plain order: neighbours, which share rows and a matrix, go to eight L2s. 8200 rows over seven experts, rows of
// 2056 fp16 to 1000: 144 tiles read 202 MB of 58 and take 57 us, where the choosing rule's estimate is 42.
// Measured and not kept: tile heights that divide an expert's rows evenly with the MFMAs of empty row blocks left out
// (the jumps between the MFMAs cost 7% of full tiles, and partial tiles, whose copies and reads bound them, gained
// nothing); nontemporal stores of c (6% slower: a store covers half lines); a tile's stores after the next tile's
// copies (spills).
#pragma once

#include "gemm_pingpong.h"
#include "grouped.h"

namespace pgemm {
namespace grouped {

using fast::static_for;
using fast::wait_vmcnt;

template <int DT, bool GRAD, bool NK>
__global__ void __launch_bounds__(512, 2) grouped_pp_kernel(Args a) {
  constexpr int BM = 256, BN = 256, BK = 64, MB = 8, WN = 64, NB = 4;
  constexpr bool A_KC = !GRAD, B_KC = !GRAD && NK;
  constexpr int HALF = 16384, B_BYTES = 32768;
  constexpr int A_ROW = A_KC ? 128 : 256, B_ROW = B_KC ? 128 : 512; // bytes of an LDS row
  constexpr int B_RPI = 1024 / B_ROW, A_RPI = 1024 / A_ROW;         // rows of a 1 KiB copy
  typedef typename fast::Frag<DT>::t frag_t;
  typedef typename Traits<DT>::out_t out_t;
  typedef std::integral_constant<int, 0> I0;
  typedef std::integral_constant<int, 1> I1;

  __shared__ __attribute__((aligned(1024))) uint8_t sAt0[HALF];
  __shared__ __attribute__((aligned(1024))) uint8_t sAt1[HALF];
  __shared__ __attribute__((aligned(1024))) uint8_t sAb0[HALF];
  __shared__ __attribute__((aligned(1024))) uint8_t sAb1[HALF];
  __shared__ __attribute__((aligned(1024))) uint8_t sB0[B_BYTES];
  __shared__ __attribute__((aligned(1024))) uint8_t sB1[B_BYTES];
  __shared__ int s_tiles[moe::kMaxExperts + 2]; // rows form: tiles up to and with each expert

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave >> 2; // 0 = X (tile rows 0-127), 1 = Y (128-255)
  const int wl = wave & 3;   // wave column (64 columns each)
  const int G = gridDim.x;

  // ---- the tile sequence ------------------------------------------------------
  int T; // tiles in all
  const int g_nm = (a.M + BM - 1) / BM; // gradient form: tile rows of every expert
  if constexpr (GRAD) {
    T = a.E * a.split * g_nm * a.n_n;
  } else {
    if (wave == 0) {
      int before = 0;
      for (int e0 = 0; e0 <= a.E; e0 += 64) {
        const int e = e0 + lane;
        int first, rows, s = 0;
        if (e <= a.E) {
          expert_rows(a, e, &first, &rows);
          s = (rows + BM - 1) / BM * a.n_n;
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int v = __shfl_up(s, d);
          if (lane >= d) s += v;
        }
        if (e <= a.E) s_tiles[e] = before + s;
        before += __shfl(s, 63);
      }
    }
    __syncthreads();
    T = min(__builtin_amdgcn_readfirstlane(s_tiles[a.E]), a.most_tiles); // bounds that run backwards stay finite
  }
  if ((int)blockIdx.x >= T) return;

  struct Tile {
    const uint16_t *A, *B; // row 0 of the tile's rows and columns, k = 0
    int m0, n0, M, K;      // tile origin; rows of c; length of the sum
    int e, first, gap_at, gap; // e: expert; gradient form: expert * split + piece
    int nk;                // steps, an even number
  };
  auto tile_at = [&](int t) __attribute__((always_inline)) -> Tile {
    const int u = xcd_remap(t, T, G);
    Tile r;
    int pm, pn;
    r.gap_at = r.gap = 0;
    if constexpr (GRAD) {
      const int per = g_nm * a.n_n, ep = u / per;
      const int e = ep / a.split;
      r.e = ep;
      grouped_tile(u - ep * per, g_nm, a.n_n, 4, &pm, &pn);
      int first, rows, from, count;
      expert_rows(a, e, &first, &rows);
      piece_rows(a, rows, ep - e * a.split, &from, &count);
      r.first = __builtin_amdgcn_readfirstlane(first + from);
      r.K = __builtin_amdgcn_readfirstlane(count);
      r.M = a.M;
      r.m0 = pm * BM;
      r.n0 = pn * BN;
      r.A = a.a + r.first * a.lda + r.m0;
      r.B = a.b + r.first * a.ldb + r.n0;
    } else {
      int e0 = 0;
      uint64_t hit;
      for (;; e0 += 64) { // the first expert whose tiles reach past u
        const int at = s_tiles[min(e0 + lane, a.E)];
        hit = __ballot(at > u);
        if (hit || e0 + 64 > a.E) break;
      }
      r.e = min(e0 + (hit ? (int)__builtin_ctzll(hit) : 63), a.E);
      const int before = r.e ? __builtin_amdgcn_readfirstlane(s_tiles[r.e - 1]) : 0;
      int first, rows;
      expert_rows(a, r.e, &first, &rows);
      r.first = __builtin_amdgcn_readfirstlane(first);
      r.M = __builtin_amdgcn_readfirstlane(rows);
      grouped_tile(u - before, (r.M + BM - 1) / BM, a.n_n, 4, &pm, &pn);
      const bool none = r.e == a.E;
      r.K = none ? 0 : a.K;
      r.m0 = pm * BM;
      r.n0 = pn * BN;
      r.A = a.a + (r.first + r.m0) * a.lda;
      r.B = a.b + (none ? 0 : r.e) * a.b_expert + (B_KC ? r.n0 * a.ldb : r.n0);
      if (none) {
        r.gap_at = r.first;
        r.gap = a.R - r.M;
        r.first = 0;
      }
    }
    r.nk = max(((r.K + BK - 1) / BK + 1) & ~1, 2);
    return r;
  };

  // ---- copy lanes ----------------------------------------------------------------
  // A half, block wl + 4j (j < 4); B, block wl + 4j (j < 8), X waves only. kc: eight
  // rows of 128 B a block, chunk c of row r at c ^ (r & 7). oc: k-rows, chunk c of
  // row k at c ^ b_swz(k); of the bits that b_swz uses, block j's 8j can set only
  // the one of 8, so B's swizzle changes with j's parity, A's (16j) not at all.
  const int b_row = B_RPI * wl + lane / (B_ROW / 16);
  const int a_row_kept = A_RPI * wl + lane / (A_ROW / 16);
  const int b_chunk = (lane % (B_ROW / 16)) ^ (B_KC ? b_row & 7 : b_swz<2, B_ROW>(b_row));

  // ---- fragment lanes --------------------------------------------------------------
  const int g = lane >> 4, s16 = lane & 15;
  // Block i's offset in an oc tile is one lane constant XOR oc_block(i) (see the
  // column order in grouped.h), which saves a register for each block.
  auto oc_block = [](int i) __attribute__((always_inline)) { return 64 * (i >> 1) + 8 * (i & 1); };
  int a_off, b_off[B_KC ? NB : 1];
  {
    const int q = s16 >> 2, qt = s16 & 3, k = 8 * g + q;
    a_off = A_KC ? s16 * 128 + 16 * (g ^ (s16 & 7)) : k * A_ROW + 16 * (qt ^ b_swz<2, A_ROW>(k)) + 8 * (qt & 1);
    if constexpr (B_KC) {
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int r = wl * WN + 32 * (i >> 1) + 8 * q + 4 * ((i + q) & 1) + qt;
        b_off[i] = r * 128 + 16 * (g ^ (r & 7));
      }
    } else {
      b_off[0] = k * B_ROW + 16 * ((wl * (WN / 8) + qt) ^ b_swz<2, B_ROW>(k)) + 8 * (qt & 1);
    }
  }

  // ---- producer: this wave's copies of the next step ---------------------------------
  int u_t = blockIdx.x, u_kt = 0;
  bool u_done = false;
  Tile u = tile_at(u_t);
  auto copy_step = [&](auto grp_c, auto stage) __attribute__((always_inline)) {
    constexpr int GR = decltype(grp_c)::value, C = decltype(stage)::value;
    uint8_t* sAh = GR == 0 ? (C == 0 ? sAt0 : sAt1) : (C == 0 ? sAb0 : sAb1);
    uint8_t* sB = C == 0 ? sB0 : sB1;
    if (u_done) return;
    if (u_kt == u.nk) {
      u_t += G;
      if (u_t >= T) {
        u_done = true;
        return;
      }
      u = tile_at(u_t);
      u_kt = 0;
    }
    const int k0 = u_kt * BK, krem = u.K - k0;
    const int mrem = u.M - u.m0 - 128 * GR, nrem = a.N - u.n0;
    // row strides in bytes and the wave's 1 KiB column of LDS blocks, made opaque so that row
    // offsets (soffset) and LDS addresses are recomputed by one scalar operation each
    int lda_s = (int)a.lda * 2, ldb_s = (int)a.ldb * 2, wl_s = wl * 1024;
    asm volatile("" : "+s"(lda_s), "+s"(ldb_s), "+s"(wl_s));
    const bool full = (mrem >= 128) & (krem >= BK) & (nrem >= BN);
    if constexpr (GR == 0) {
      const __amdgpu_buffer_rsrc_t rb = make_rsrc(u.B + (B_KC ? (int64_t)k0 : k0 * a.ldb));
      static_for<8>([&](auto jc) __attribute__((always_inline)) {
        constexpr int ROW = 4 * B_RPI * decltype(jc)::value;
        int c = b_chunk;
        bool ok;
        if constexpr (B_KC) {
          ok = (b_row + ROW < nrem) & (8 * c < krem);
        } else {
          c ^= b_swz<2, B_ROW>(ROW);
          ok = (b_row + ROW < krem) & (8 * c < nrem);
        }
        const uint32_t base = (uint32_t)b_row * (uint32_t)ldb_s + 16u * (uint32_t)c;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, PGEMM_LDS(void, sB + 4096 * decltype(jc)::value + wl_s), 16,
                                                 full || ok ? base : kOOB, ROW * ldb_s, 0, 0);
      });
    }
    int a_row = a_row_kept, l = lane;
    if constexpr (GRAD) { // read again each step: kept live, these two take the loop past its registers
      asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
      a_row = A_RPI * wl + l / (A_ROW / 16);
    }
    const int a_chunk = (l % (A_ROW / 16)) ^ (A_KC ? a_row & 7 : b_swz<2, A_ROW>(a_row));
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(u.A + (A_KC ? 128 * GR * a.lda + k0 : k0 * a.lda + 128 * GR));
    static_for<4>([&](auto jc) __attribute__((always_inline)) {
      constexpr int ROW = 4 * A_RPI * decltype(jc)::value;
      bool ok;
      if constexpr (A_KC) ok = (a_row + ROW < mrem) & (8 * a_chunk < krem);
      else ok = (a_row + ROW < krem) & (8 * a_chunk < mrem);
      const uint32_t base = (uint32_t)a_row * (uint32_t)lda_s + 16u * (uint32_t)a_chunk;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, PGEMM_LDS(void, sAh + 4096 * decltype(jc)::value + wl_s), 16,
                                               full || ok ? base : kOOB, ROW * lda_s, 0, 0);
    });
    ++u_kt;
  };

  // ---- accumulators, fragments ----------------------------------------------------------
  floatx4_t acc[MB][NB];
  frag_t af[2][MB], bf[2][NB];
  auto read_frags = [&](auto grp_c, auto stage) __attribute__((always_inline)) {
    constexpr int GR = decltype(grp_c)::value, C = decltype(stage)::value;
    const uint8_t* sAh = GR == 0 ? (C == 0 ? sAt0 : sAt1) : (C == 0 ? sAb0 : sAb1);
    const uint8_t* sB = C == 0 ? sB0 : sB1;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        if constexpr (B_KC) bf[kk][i] = read_a<DT>(sB + (b_off[i] ^ (64 * kk)), nullptr);
        else bf[kk][i] = read_b<DT, B_ROW>(sB + (b_off[0] ^ oc_block(i)) + kk * 32 * B_ROW);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        if constexpr (A_KC) af[kk][i] = read_a<DT>(sAh + (a_off ^ (64 * kk)) + i * 16 * 128, nullptr);
        else af[kk][i] = read_b<DT, A_ROW>(sAh + (a_off ^ oc_block(i)) + kk * 32 * A_ROW);
      }
    }
  };
  auto compute = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) mfma_acc(acc[i][j], bf[kk][j], af[kk][i]);
  };
  auto zero_acc = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    acc_drain();
  };

  // ---- epilogue: this wave's 128 x 64 block, rounded and stored ----------------------------
  auto epilogue = [&](auto grp_c, const Tile& c) __attribute__((always_inline)) {
    constexpr int GR = decltype(grp_c)::value;
    acc_drain();
    int lane_e; // recomputed here rather than kept live through the k-loop
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(lane_e));
    const int s16 = lane_e & 15, g = lane_e >> 4, q = s16 >> 2;
    const int n = c.n0 + wl * WN + 8 * g;
    const bool odd = (g & 1) != 0;
    if constexpr (GRAD) {
      if (a.split > 1) { // N is a multiple of 8
        float* part = a.part + (int64_t)c.e * a.M * a.N + n;
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          const int m = c.m0 + 128 * GR + 32 * (i >> 1) + 8 * q + 4 * ((i + q) & 1) + (s16 & 3);
#pragma unroll
          for (int j = 0; j < NB; ++j) { // block j's columns: the first or the second four of eight
            const int at = 32 * (j >> 1) + 4 * ((j ^ g) & 1);
            if (m < c.M && n + 32 * (j >> 1) < a.N) *reinterpret_cast<floatx4_t*>(part + (int64_t)m * a.N + at) = acc_read(acc[i][j]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        return;
      }
    }
    out_t* C = reinterpret_cast<out_t*>(a.c) + (GRAD ? (int64_t)c.e * a.M : c.first) * a.N + n;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int m = c.m0 + 128 * GR + (A_KC ? 16 * i + s16 : 32 * (i >> 1) + 8 * q + 4 * ((i + q) & 1) + (s16 & 3));
      if (m < c.M) {
        out_t* dst = C + (int64_t)(m < c.gap_at ? m : m + c.gap) * a.N;
#pragma unroll
        for (int P = 0; P < NB / 2; ++P)
          if (n + 32 * P < a.N) store8(dst + 32 * P, acc_read(acc[i][2 * P]), acc_read(acc[i][2 * P + 1]), odd);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // ---- the ping-pong, one instance per group -----------------------------------------------
  auto run = [&](auto grp_c) __attribute__((always_inline)) {
    constexpr int GR = decltype(grp_c)::value;
    copy_step(grp_c, I0{});
    wait_vmcnt<0>();
    pp::barrier_raw();
    if constexpr (GR == 1) pp::barrier_raw(); // Y runs one phase behind X
    auto step = [&](auto stage) __attribute__((always_inline)) {
      typedef std::integral_constant<int, decltype(stage)::value ^ 1> NEXT;
      copy_step(grp_c, NEXT{});
      read_frags(grp_c, stage);
      pp::wait_lgkm0();
      pp::barrier_raw();
      compute();
      __builtin_amdgcn_sched_barrier(0);
      wait_vmcnt<0>(); // this wave's copies of the next step (and its stores) have landed
      pp::barrier_raw();
    };
    Tile c = u; // the tile being summed; u runs one step ahead
    zero_acc();
    for (;;) {
      for (int kt = 0; kt < c.nk; kt += 2) {
        step(I0{});
        step(I1{});
      }
      if (u_done) break;
      epilogue(grp_c, c);
      c = u;
      zero_acc();
    }
    if constexpr (GR == 0) pp::barrier_raw(); // X matches Y's extra barrier
    epilogue(grp_c, c);
  };
  if (grp == 0)
    run(I0{});
  else
    run(I1{});
}

} // namespace grouped
} // namespace pgemm
