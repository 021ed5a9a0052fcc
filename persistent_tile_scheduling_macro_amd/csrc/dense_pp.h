// The linear layer's body for large products: the ping-pong 256 x 256 tile of
// gemm_pingpong.h (eight waves of 128 x 64 in two groups of opposite phases,
// copies that write LDS directly), persistent over the tiles and their pieces.
//
// What differs from that body: the epilogue of dense.h; the gated form, in
// which each 64 columns of a wave are 32 gate columns and the 32 up columns
// that belong to them (only the copies of W know: its rows or chunks are
// fetched from both halves); sums cut into pieces; and the last round of
// tiles, which is dealt in eight stretches, one to an XCD, like a whole round
// (neighbouring tiles share rows of x and columns of W in one L2). And at a
// tile's end the groups meet, so that both are in the epilogue at once: with one
// wave a SIMD in it and the other group waiting, the training step of 8192 x 8192
// x 4096 took 1498 us and that of 4096 x 4096 x 2048 gated 428, now 1425 and 410.
//
// 8192 x 8192 x 4096 bf16: the product with gelu and z 479 to 503 us, dx 459 to 484
// and dW 495 to 513 (at best 1150, 1200 and 1110 TFLOP/s; a plain library product
// in the same call 1130), MFMA busy 0.55 to 0.61 at the clock that power leaves. A
// body of four waves with 128 x 128 each, which reads a third less from LDS, took
// 543 us for 8192 x 4096 x 8192, where this took 497.
#pragma once

#include "dense.h"
#include "gemm_pingpong.h"

namespace pgemm {
namespace dense {

using fast::static_for;
using fast::wait_vmcnt;

template <int DT, int FORM, bool GATED>
__global__ void __launch_bounds__(512, 2) ping_kernel(Args a) {
  constexpr int BM = 256, BN = 256, BK = 64, MB = 8, WN = 64, NB = 4;
  constexpr bool GRAD = FORM == kGrad, A_KC = !GRAD, B_KC = FORM == kRowsNK;
  constexpr int HALF = 16384, B_BYTES = 32768;
  constexpr int A_ROW = A_KC ? 128 : 256, B_ROW = B_KC ? 128 : 512; // bytes of an LDS row
  constexpr int B_RPI = 1024 / B_ROW, A_RPI = 1024 / A_ROW;         // rows of a 1 KiB copy
  constexpr int OUT_N = GATED ? BN / 2 : BN;                        // columns of c in a tile
  typedef typename fast::Frag<DT>::t frag_t;
  typedef std::integral_constant<int, 0> I0;
  typedef std::integral_constant<int, 1> I1;

  __shared__ __attribute__((aligned(1024))) uint8_t sAt0[HALF];
  __shared__ __attribute__((aligned(1024))) uint8_t sAt1[HALF];
  __shared__ __attribute__((aligned(1024))) uint8_t sAb0[HALF];
  __shared__ __attribute__((aligned(1024))) uint8_t sAb1[HALF];
  __shared__ __attribute__((aligned(1024))) uint8_t sB0[B_BYTES];
  __shared__ __attribute__((aligned(1024))) uint8_t sB1[B_BYTES];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave >> 2; // 0 = X (tile rows 0-127), 1 = Y (128-255)
  const int wl = wave & 3;   // wave column (64 columns each)
  const int G = gridDim.x;   // a multiple of 8, or as many as there are tiles
  const int per = a.n_m * a.n_n, T = per * a.split;

  struct Tile {
    const uint16_t *A, *B; // row 0 of the tile's rows and columns, k = the piece's first
    int m0, n0, K;         // tile origin; length of the sum from there
    int piece, nk;         // steps, an even number
  };
  // The tile of the workgroup's round `round`; false past its last one.
  auto tile_at = [&](int round, Tile* r) __attribute__((always_inline)) -> bool {
    const int base = round * G, left = min(T - base, G), b = blockIdx.x;
    if (left <= 0) return false;
    int u = b;
    if ((G & 7) == 0) {
      const int share = (left + 7) >> 3;
      u = (b & 7) * share + (b >> 3);
      if ((b >> 3) >= share) return false;
    }
    if (u >= left) return false;
    u += base;
    int pm, pn, first;
    r->piece = u / per;
    grouped_tile(u - r->piece * per, a.n_m, a.n_n, 4, &pm, &pn);
    const int steps = (a.K + BK - 1) / BK;
    first = (int)((int64_t)steps * r->piece / a.split);
    const int last = (int)((int64_t)steps * (r->piece + 1) / a.split);
    r->K = min(a.K, last * BK) - first * BK;
    r->m0 = pm * BM;
    r->n0 = pn * OUT_N;
    const int64_t k0 = (int64_t)first * BK;
    r->A = A_KC ? a.a + r->m0 * a.lda + k0 : a.a + k0 * a.lda + r->m0;
    r->B = B_KC ? a.b + r->n0 * a.ldb + k0 : a.b + k0 * a.ldb + r->n0;
    r->nk = max((last - first + 1) & ~1, 2);
    return true;
  };

  // ---- copy lanes (grouped_pp.h)
  const int b_row = B_RPI * wl + lane / (B_ROW / 16);
  const int a_row_kept = A_RPI * wl + lane / (A_ROW / 16);
  const int b_chunk = (lane % (B_ROW / 16)) ^ (B_KC ? b_row & 7 : fast::b_swz<2, B_ROW>(b_row));

  // ---- fragment lanes
  const int g = lane >> 4, s16 = lane & 15;
  auto oc_block = [](int i) __attribute__((always_inline)) { return 64 * (i >> 1) + 8 * (i & 1); };
  int a_off, b_off[B_KC ? NB : 1];
  {
    const int q = s16 >> 2, qt = s16 & 3, k = 8 * g + q;
    a_off = A_KC ? s16 * 128 + 16 * (g ^ (s16 & 7)) : k * A_ROW + 16 * (qt ^ fast::b_swz<2, A_ROW>(k)) + 8 * (qt & 1);
    if constexpr (B_KC) {
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int r = wl * WN + 32 * (i >> 1) + 8 * q + 4 * ((i + q) & 1) + qt;
        b_off[i] = r * 128 + 16 * (g ^ (r & 7));
      }
    } else {
      b_off[0] = k * B_ROW + 16 * ((wl * (WN / 8) + qt) ^ fast::b_swz<2, B_ROW>(k)) + 8 * (qt & 1);
    }
  }

  // ---- producer: this wave's copies of the next step
  int u_round = 0, u_kt = 0;
  Tile u;
  if (!tile_at(0, &u)) return;
  bool u_done = false;
  auto copy_step = [&](auto grp_c, auto stage) __attribute__((always_inline)) {
    constexpr int GR = decltype(grp_c)::value, C = decltype(stage)::value;
    uint8_t* sAh = GR == 0 ? (C == 0 ? sAt0 : sAt1) : (C == 0 ? sAb0 : sAb1);
    uint8_t* sB = C == 0 ? sB0 : sB1;
    if (u_done) return;
    if (u_kt == u.nk) {
      if (!tile_at(++u_round, &u)) {
        u_done = true;
        return;
      }
      u_kt = 0;
    }
    const int k0 = u_kt * BK, krem = u.K - k0;
    const int mrem = a.M - u.m0 - 128 * GR, nrem = a.N - u.n0;
    // row strides in bytes and the wave's 1 KiB column of LDS blocks, made opaque so that row
    // offsets (soffset) and LDS addresses are recomputed by one scalar operation each
    int lda_s = (int)a.lda * 2, ldb_s = (int)a.ldb * 2, wl_s = wl * 1024;
    asm volatile("" : "+s"(lda_s), "+s"(ldb_s), "+s"(wl_s));
    const bool full = (mrem >= 128) & (krem >= BK) & (nrem >= OUT_N);
    if constexpr (GR == 0) {
      const uint16_t* from = u.B + (B_KC ? (int64_t)k0 : k0 * a.ldb);
      const __amdgpu_buffer_rsrc_t rb = make_rsrc(from), rb_up = make_rsrc(GATED && B_KC ? from + a.half : from);
      static_for<8>([&](auto jc) __attribute__((always_inline)) {
        constexpr int J = decltype(jc)::value, ROW = 4 * B_RPI * J;
        int c = b_chunk;
        bool ok;
        uint32_t base;
        int at = ROW * ldb_s;
        if constexpr (B_KC) {
          // gated: LDS rows 64 i + 32 h + c hold columns 32 i + c, gate for h = 0, up for h = 1
          constexpr int COL = GATED ? (J >> 1) * 32 : ROW;
          ok = (b_row + COL < nrem) & (8 * c < krem);
          base = (uint32_t)b_row * (uint32_t)ldb_s + 16u * (uint32_t)c;
          at = COL * ldb_s;
        } else {
          c ^= fast::b_swz<2, B_ROW>(ROW);
          const int n = GATED ? (c >> 3) * 32 + 8 * (c & 3) : 8 * c;
          ok = (b_row + ROW < krem) & (n < nrem);
          base = (uint32_t)b_row * (uint32_t)ldb_s + 2u * (uint32_t)n;
          if constexpr (GATED) base += 2u * (uint32_t)a.half * (uint32_t)((c >> 2) & 1);
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(GATED && B_KC && (J & 1) ? rb_up : rb,
                                                 PGEMM_LDS(void, sB + 4096 * J + wl_s), 16, full || ok ? base : kOOB, at, 0, 0);
      });
    }
    int a_row = a_row_kept, l = lane;
    if constexpr (!B_KC) { // read again each step: kept live, these two take the loop past its registers
      asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
      a_row = A_RPI * wl + l / (A_ROW / 16);
    }
    const int a_chunk = (l % (A_ROW / 16)) ^ (A_KC ? a_row & 7 : fast::b_swz<2, A_ROW>(a_row));
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

  // ---- accumulators, fragments
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
        if constexpr (B_KC) bf[kk][i] = fast::read_a<DT>(sB + (b_off[i] ^ (64 * kk)), nullptr);
        else bf[kk][i] = fast::read_b<DT, B_ROW>(sB + (b_off[0] ^ oc_block(i)) + kk * 32 * B_ROW);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        if constexpr (A_KC) af[kk][i] = fast::read_a<DT>(sAh + (a_off ^ (64 * kk)) + i * 16 * 128, nullptr);
        else af[kk][i] = fast::read_b<DT, A_ROW>(sAh + (a_off ^ oc_block(i)) + kk * 32 * A_ROW);
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

  // ---- epilogue of this wave's 128 x 64 block
  auto finish_tile = [&](auto grp_c, const Tile& c) __attribute__((always_inline)) {
    constexpr int GR = decltype(grp_c)::value;
    acc_drain();
    int lane_e; // recomputed here rather than kept live through the k-loop
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(lane_e));
    const int s16 = lane_e & 15, g = lane_e >> 4, q = s16 >> 2;
    const bool odd = (g & 1) != 0;
    auto row_of = [&](int i) __attribute__((always_inline)) {
      return c.m0 + 128 * GR + (A_KC ? 16 * i + s16 : 32 * (i >> 1) + 8 * q + 4 * ((i + q) & 1) + (s16 & 3));
    };
    auto eight = [&](int i, int P, float* v) __attribute__((always_inline)) {
      const floatx4_t x = acc_read(acc[i][2 * P]), y = acc_read(acc[i][2 * P + 1]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[r] = odd ? y[r] : x[r];
        v[4 + r] = odd ? x[r] : y[r];
      }
    };
    const int n = c.n0 + wl * (GATED ? 32 : WN) + 8 * g; // columns of P: 32 P further (gated: the up columns of the same)
    if (a.split > 1) {
      const int64_t ld = part_ld(a, GATED);
      float* part = a.part + (int64_t)c.piece * a.M * ld + n;
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int m = row_of(i);
#pragma unroll
        for (int P = 0; P < 2; ++P) {
          float v[8];
          eight(i, P, v);
          if (m < a.M && n + (GATED ? 0 : 32 * P) < a.N) {
            float* to = part + m * ld + (GATED ? P * (ld / 2) : 32 * P);
            *reinterpret_cast<floatx4_t*>(to) = floatx4_t{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<floatx4_t*>(to + 4) = floatx4_t{v[4], v[5], v[6], v[7]};
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      return;
    }
    const Epilogue<DT, GATED, true> epilogue(a); // N is a multiple of 8 here
#pragma unroll
    for (int P = 0; P < (GATED ? 1 : 2); ++P) {
      float bv[8], bu[8];
      epilogue.bias_of(n + 32 * P, bv, bu);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int m = row_of(i);
        float v[8], w[8];
        eight(i, P, v);
        if constexpr (GATED) eight(i, 1, w);
        if (m < a.M && n + 32 * P < a.N)
          act::with_path(epilogue.k, [&](auto path) __attribute__((always_inline)) {
            epilogue.template finish<decltype(path)::value>(m, n + 32 * P, v, w, bv, bu);
          });
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // ---- the ping-pong, one instance per group
  auto run = [&](auto grp_c) __attribute__((always_inline)) {
    constexpr int GR = decltype(grp_c)::value;
    copy_step(grp_c, I0{});
    wait_vmcnt<0>();
    pp::barrier_raw();
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
    for (;;) {
      const Tile c = u; // the tile being summed; u runs one step ahead
      zero_acc();
      if constexpr (GR == 1) pp::barrier_raw(); // Y runs one phase behind X
      for (int kt = 0; kt < c.nk; kt += 2) {
        step(I0{});
        step(I1{});
      }
      if constexpr (GR == 0) pp::barrier_raw(); // X matches Y's extra barrier
      finish_tile(grp_c, c); // both groups at once
      if (u_done) break;
    }
  };
  if (grp == 0)
    run(I0{});
  else
    run(I1{});
}

} // namespace dense
} // namespace pgemm
