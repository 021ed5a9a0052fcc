// The linear layer's body for few rows, ROWS (8, 16 or 32) at once: every byte of
// W is read once for them, and that reading bounds it.
//
// The scheme is that of grouped_few.h: a workgroup takes 16 * BLK columns of W
// (gated: half of them gate columns, half their up columns), its waves take
// the steps of the sum in turn and join their fp32 sums in LDS in a fixed
// order. Loads run along rows, D steps ahead, into registers; each wave turns
// its step's operands in its own LDS (N x K weights and x), or pairs rows by
// half-word permutes (K x N weights). W is the MFMA's first operand, so a
// lane's four outputs are columns of one row of y. Bias and residual are read
// before the loop.
//
// 1 x 4096 x 4096 bf16: 8.0 us a call among others, 4.2 TB/s, of which a bare
// launch is 3.9 (8.7 between the kernel's own timestamps); 16 x 4096 x 2 * 8192
// gated fp16: 24.2 us for the kernel, 5.6 TB/s, 26.7 a call.
#pragma once

#include "dense.h"
#include "grouped_few.h"

namespace pgemm {
namespace dense {

using grouped::load_upto;
using grouped::turn_at;
using grouped::u32x2;
using grouped::u32x2_any;

template <int DT, bool NK, bool GATED, int ROWS, int BLK, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, BLK == 8 ? 2 : 4) few_kernel(Args a) {
  static_assert(NK || BLK == (GATED ? 8 : 4), "K x N: four columns a lane");
  constexpr int MB = (ROWS + 15) / 16;
  constexpr int STEP = NK ? 64 : 32, H = STEP / 32;
  constexpr int ROW = STEP * 2, LPR = ROW / 16, RPL = 64 / LPR; // bytes of a step's row, lanes to a row, rows of a load
  constexpr int L = 16 / RPL, XL = ROWS < 16 && RPL == 8 ? 1 : MB * L; // loads of 16 rows; loads of x
  // Steps in flight. Calls replayed over six matrices in turn: 16 x 4096 x 2 * 8192 gated fp16 28.8 us, with three 30.7; 1 x 4096 x
  // 4096 bf16 7.8, with two 8.0.
  constexpr int D = !NK || GATED || ROWS > 16 ? 2 : 4;
  constexpr int OUT = GATED ? BLK / 2 : BLK; // blocks of y's columns
  typedef typename fast::Frag<DT>::t frag_t;
  typedef typename Traits<DT>::out_t out_t;
  constexpr int TURN = 16 * ROW * (MB + (NK ? BLK : 0)), JOIN = BLK * MB * 64 * 16; // LDS bytes of a wave
  __shared__ __attribute__((aligned(1024))) uint8_t lds[WAVES * (TURN > JOIN ? TURN : JOIN)];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, s = lane & 15;
  const int n0 = blockIdx.x * 16 * OUT, m0 = blockIdx.y * ROWS, N = a.N, K = a.K, M = a.M;

  // Column that output position `at` of block c of y stands for; K x N lanes at the edge start at N - 4, and
  // what is then computed twice is stored once.
  auto column = [&](int c, int at, bool* mine) __attribute__((always_inline)) {
    if constexpr (NK) {
      const int n = n0 + 16 * c + at;
      *mine = n < N;
      return n;
    } else {
      const int from = n0 + 4 * at, n = min(from, N - 4) + c;
      *mine = from < N && n >= from;
      return n;
    }
  };
  auto half_word = [](const uint16_t* p) __attribute__((always_inline)) {
    float f[8];
    moe::unpack<DT>(u32x4{*p, 0, 0, 0}, f);
    return f[0];
  };
  constexpr int ITEMS = OUT * MB * 64, TURNS = (ITEMS + WAVES * 64 - 1) / (WAVES * 64);
  static_assert(TURNS == 1, "a thread finishes one group of four outputs");
  const int fl = tid & 63, fb = (tid >> 6) % MB, fc = (tid >> 6) / MB, fm = m0 + 16 * fb + (fl & 15);
  const bool finisher = tid < ITEMS && 16 * fb + (fl & 15) < ROWS && fm < M;
  float bias[4] = {0, 0, 0, 0}, bias_up[4] = {0, 0, 0, 0}, residual[4] = {0, 0, 0, 0};
  if (finisher) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      bool mine;
      const int n = column(fc, 4 * (fl >> 4) + r, &mine);
      if (!mine) continue;
      if (a.bias) {
        bias[r] = half_word(a.bias + n);
        if constexpr (GATED) bias_up[r] = half_word(a.bias + N + n);
      }
      if (a.residual) residual[r] = half_word(a.residual + fm * a.ldr + n);
    }
  }

  const int row = lane / LPR, chunk = lane % LPR;
  const uint16_t* x[XL];
#pragma unroll
  for (int i = 0; i < XL; ++i) x[i] = a.a + min(m0 + RPL * i + row, M - 1) * a.lda + 8 * chunk;
  constexpr int WP = NK ? BLK * L : GATED ? 2 : 1;
  const uint16_t* w[WP];
#pragma unroll
  for (int i = 0; i < WP; ++i) {
    const int up = GATED && (NK ? i / L >= OUT : i == 1);
    const int64_t from = up ? a.half : 0;
    const int c = RPL * i - up * 16 * OUT + row;
    w[i] = a.b + from + (NK ? min(n0 + c, N - 1) * a.ldb + 8 * chunk : 8 * g * a.ldb + min(n0 + 4 * s, N - 4));
  }

  struct Slot { // what a step reads
    u32x4 x[XL];
    u32x4 w[NK ? BLK * L : 4 * WP]; // K x N: rows 2i and 2i + 1, four columns each
  };
  auto load = [&](Slot& t, int step) __attribute__((always_inline)) {
    const int64_t k0 = (int64_t)step * STEP;
    if constexpr (NK) {
#pragma unroll
      for (int i = 0; i < BLK * L; ++i) t.w[i] = moe::load8<moe::kAnyAddress>(w[i] + k0);
    } else {
#pragma unroll
      for (int p = 0; p < WP; ++p) {
        const uint16_t* r = w[p] + k0 * a.ldb;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const u32x2 lo = *reinterpret_cast<const u32x2_any*>(r + 2 * i * a.ldb);
          const u32x2 hi = *reinterpret_cast<const u32x2_any*>(r + (2 * i + 1) * a.ldb);
          t.w[4 * p + i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
      }
    }
#pragma unroll
    for (int i = 0; i < XL; ++i) t.x[i] = moe::load8<moe::kAnyAddress>(x[i] + k0);
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
    for (int i = 0; i < XL; ++i) *reinterpret_cast<u32x4*>(turn_x + turn_at<ROW>(RPL * i + row, chunk)) = t.x[i];
    if constexpr (NK) {
#pragma unroll
      for (int i = 0; i < BLK * L; ++i) *reinterpret_cast<u32x4*>(turn_w + turn_at<ROW>(RPL * i + row, chunk)) = t.w[i];
    }
    wave_fence();
#pragma unroll
    for (int h = 0; h < H; ++h) {
      frag_t xf[MB];
#pragma unroll
      for (int b = 0; b < MB; ++b) // fewer than 16 rows: they fill the operand twice
        xf[b] = *reinterpret_cast<const frag_t*>(turn_x + turn_at<ROW>(XL * RPL < 16 ? s % 8 : 16 * b + s, 4 * h + g));
#pragma unroll
      for (int c = 0; c < BLK; ++c) {
        frag_t f;
        if constexpr (NK) {
          f = *reinterpret_cast<const frag_t*>(turn_w + turn_at<ROW>(16 * c + s, 4 * h + g));
        } else {
          u32x4 v;
#pragma unroll
          for (int i = 0; i < 4; ++i) { // column c of rows 2i and 2i + 1
            const u32x4 d = t.w[4 * (c / 4) + i];
            v[i] = __builtin_amdgcn_perm(d[2 + c % 4 / 2], d[c % 4 / 2], c % 2 ? 0x07060302u : 0x05040100u);
          }
          f = __builtin_bit_cast(frag_t, v);
        }
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[b][c] = mfma(f, xf[b], acc[b][c]);
      }
    }
  };

  const int whole = K / STEP;
  const int mine = (whole - wave + WAVES - 1) / WAVES; // steps wave, wave + WAVES, ... (none if not positive)
  stream_steps<D, Slot>(mine, [&](Slot& t, int i) __attribute__((always_inline)) { load(t, wave + WAVES * i); }, multiply);
  if (whole * STEP < K && wave == whole % WAVES) { // the partial step, zeros past K
    const int k0 = whole * STEP;
    Slot t;
    if constexpr (NK) {
#pragma unroll
      for (int i = 0; i < BLK * L; ++i) t.w[i] = load_upto(w[i] + k0, K - k0 - 8 * chunk, K);
    } else {
      const int left = K - k0 - 8 * g;
#pragma unroll
      for (int p = 0; p < WP; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint16_t* r = w[p] + (k0 + 2 * i) * a.ldb;
          u32x2 lo = {0, 0}, hi = {0, 0};
          if (2 * i < left) lo = *reinterpret_cast<const u32x2_any*>(r);
          if (2 * i + 1 < left) hi = *reinterpret_cast<const u32x2_any*>(r + a.ldb);
          t.w[4 * p + i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
    }
#pragma unroll
    for (int i = 0; i < XL; ++i) t.x[i] = load_upto(x[i] + k0, K - k0 - 8 * chunk, K);
    multiply(t);
  }

  __syncthreads(); // every wave is through with its part of the LDS
  floatx4_t* join = reinterpret_cast<floatx4_t*>(lds);
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int c = 0; c < BLK; ++c) join[(wave * BLK * MB + c * MB + b) * 64 + lane] = acc[b][c];
  __syncthreads();
  if (!finisher) return;
  floatx4_t v = join[tid], u = floatx4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int o = 1; o < WAVES; ++o) v += join[o * BLK * MB * 64 + tid];
  if constexpr (GATED) {
    u = join[ITEMS + tid];
#pragma unroll
    for (int o = 1; o < WAVES; ++o) u += join[o * BLK * MB * 64 + ITEMS + tid];
  }
  const act::Consts k = act::consts_of(a.act);
  auto bits = [](float f) __attribute__((always_inline)) { return __builtin_bit_cast(uint16_t, to_out(f, (out_t*)nullptr)); };
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    bool keep;
    const int n = column(fc, 4 * (fl >> 4) + r, &keep);
    if (!keep) continue;
    float y = v[r] + bias[r];
    const float up = u[r] + bias_up[r];
    if (a.z) {
      uint16_t* z = a.z + (int64_t)fm * (GATED ? 2 : 1) * N;
      z[n] = bits(z_value<DT>(y));
      if constexpr (GATED) z[N + n] = bits(z_value<DT>(up));
    }
    act::with_path(k, [&](auto path) __attribute__((always_inline)) { y = act::value<decltype(path)::value>(y, k); });
    if constexpr (GATED) y *= up;
    a.c[(int64_t)fm * N + n] = bits(a.residual ? y + residual[r] : y);
  }
}

} // namespace dense
} // namespace pgemm
