// Few rows times 4-bit weights: y[m][n] = sum_k x[m][k] * dec(q[n][k]), with
//   dec = (code - z[n][k / group]) * s[n][k / group]   (int4; z = 8 without zero points)
//   dec = e2m1(code) * s[n][k / group]                 (sign, two exponent bits, one mantissa bit)
// Codes lie along K, two to a byte, the lower nibble first.
//
// The codes' bytes bound it: each is read once and used for every row of x.
// A wave owns CB blocks of 16 columns and a range of K; lane (g, s), s < 16,
// loads 16 bytes (32 codes) of column s at a time, so the four lanes of a
// column read 64 bytes in a row, straight into registers: no weight is used
// by two waves, so LDS would only add a copy. Two swaps between lane groups
// then give lane group g the codes 8g..8g+7 of each 32, the operand layout of
// the 16x16x32 MFMA, whose 32 products all lie in one scale group.
//
// Codes become operands without rounding: code - z is a whole number up to
// 15 and an e2m1 value has two significant bits, so both are exact in either
// type, and the MFMA sums exact products in fp32. The group's scale multiplies
// that sum, also in fp32; a weight is never rounded to 16 bits.
//
// The waves of a workgroup split K between them (K is long and the rows are
// few) and their sums are joined in LDS in a fixed order.
#pragma once

#include "device_common.h"

namespace pgemm {
namespace w4 {

enum Fmt : int { kInt4 = 0, kInt4Zero = 1, kE2M1 = 2 };
constexpr int kStep = 128; // k of one load: 4 lane groups x 16 bytes
constexpr int kWaves = 8;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

struct Args {
  const uint16_t* x; // [M, K], rows ldx apart
  int64_t ldx;
  const uint8_t* q;       // [E][N][row_bytes]
  const uint16_t* scales; // [E][N][groups]
  const uint8_t* zeros;   // [E][N][groups]
  const int* offsets;     // E + 1 row bounds, or null: one expert with every row
  uint16_t* y;            // [M, N]
  int M, N, K, E;
  int row_bytes, groups;
};

template <int DT>
struct Frag;
template <>
struct Frag<kF16> { typedef half8_t t; };
template <>
struct Frag<kBF16> { typedef bf16x8_t t; };

__device__ inline uint32_t pair(uint32_t lo_from, uint32_t hi_from, bool high) {
  // the low (or high) halves of two registers as one
  return __builtin_amdgcn_perm(hi_from, lo_from, high ? 0x07060302u : 0x05040100u);
}

// The eight codes of a register as an MFMA operand, in the order in which
// they come out cheapest; order_x puts x's elements into the same order.
//   int4, fp16: (0,4) (1,5) (2,6) (3,7)   a nibble under the bits of 1024.0 is 1024 + code;
//               adding -(1024 + z) is exact
//   int4, bf16: (0,2) (4,6) (1,3) (5,7)   bytes of sign and magnitude are e4m3 codes of
//               (code - z) / 512, as e4m3 counts in 1/512 up to 15/512; the conversion
//               multiplies by 512
//   e2m1:       in order, by the conversion instruction
template <int DT, int FMT>
__device__ inline u32x4 decode(uint32_t d, uint32_t zz) {
  u32x4 o;
  if constexpr (FMT == kE2M1) {
    if constexpr (DT == kF16) {
      o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 0));
      o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 1));
      o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 2));
      o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 3));
    } else {
      o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 0));
      o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 1));
      o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 2));
      o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 3));
    }
  } else if constexpr (DT == kF16) {
    const half2_t c = __builtin_bit_cast(half2_t, zz); // -(1024 + z), twice
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const half2_t h = __builtin_bit_cast(half2_t, ((d >> (4 * p)) & 0x000F000Fu) | 0x64006400u);
      o[p] = __builtin_bit_cast(uint32_t, h + c);
    }
  } else {
    uint32_t b[2] = {d & 0x0F0F0F0Fu, (d >> 4) & 0x0F0F0F0Fu};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t t = (b[i] | 0x80808080u) - zz; // 128 + code - z in each byte
      const uint32_t neg = ~t & 0x80808080u, ones = neg >> 7;
      b[i] = ((t ^ (neg - ones)) + ones) ^ 0x80808080u; // sign bit and magnitude
      o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b[i], 512.0f, false));
      o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b[i], 512.0f, true));
    }
  }
  return o;
}

template <int DT, int FMT>
__device__ inline u32x4 order_x(u32x4 v) {
  if constexpr (FMT == kE2M1) return v;
  else if constexpr (DT == kF16)
    return u32x4{pair(v[0], v[2], false), pair(v[0], v[2], true), pair(v[1], v[3], false), pair(v[1], v[3], true)};
  else
    return u32x4{pair(v[0], v[1], false), pair(v[2], v[3], false), pair(v[0], v[1], true), pair(v[2], v[3], true)};
}

// The operand of the subtraction for zero point z (four bits).
template <int DT, int FMT>
__device__ inline uint32_t zero_operand(uint32_t z) {
  if constexpr (FMT == kE2M1) return 0;
  else if constexpr (DT == kF16) return (0xE400u + z) * 0x00010001u;
  else return z * 0x01010101u;
}

template <int DT>
__device__ inline float scale_value(uint16_t b) {
  if constexpr (DT == kF16) return (float)__builtin_bit_cast(_Float16, b);
  else return __builtin_bit_cast(float, (uint32_t)b << 16);
}

template <int DT, int FMT, int GROUP, int MB, int CB>
__global__ void __launch_bounds__(kWaves * 64) w4_kernel(Args a) {
  constexpr int GPS = kStep / GROUP; // scale groups of a step
  constexpr int SPG = GROUP / 32;    // MFMA k-groups of a scale group
  constexpr int SR = (GPS + 1) / 2;  // registers that hold a step's scales
  constexpr int XD = MB == 1 ? 4 : MB == 2 ? 2 : 1; // 32-k pieces of x read ahead
  typedef typename Frag<DT>::t frag_t;
  typedef typename Traits<DT>::out_t out_t;
  __shared__ floatx4_t red[kWaves][CB * MB * 64];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, s = lane & 15;
  const int n0 = blockIdx.x * 16 * CB;
  int m0, m1, e = 0;
  if (a.offsets) {
    e = blockIdx.y;
    if (e == a.E) { // rows of no expert are zeros
      const int lo = min(max(a.offsets[0], 0), a.M), hi = min(max(a.offsets[a.E], lo), a.M);
      for (int64_t i = tid; i < (int64_t)(a.M - (hi - lo)) * 16 * CB; i += kWaves * 64) {
        const int r = (int)(i / (16 * CB)), n = n0 + (int)(i % (16 * CB));
        if (n < a.N) a.y[(int64_t)(r < lo ? r : r + hi - lo) * a.N + n] = 0;
      }
      return;
    }
    m0 = min(max(a.offsets[e], 0), a.M);
    m1 = min(max(a.offsets[e + 1], m0), a.M);
  } else {
    m0 = blockIdx.y * 16 * MB;
    m1 = min(m0 + 16 * MB, a.M);
  }
  if (m0 >= m1) return;

  const uint8_t* wrow[CB];
  const uint16_t* srow[CB];
  const uint8_t* zrow[CB];
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    const int n = min(n0 + 16 * c + s, a.N - 1); // columns past N read the last one and are not stored
    const int64_t col = (int64_t)e * a.N + n;
    wrow[c] = a.q + col * a.row_bytes + 16 * g;
    srow[c] = a.scales + col * a.groups;
    zrow[c] = FMT == kInt4Zero ? a.zeros + col * a.groups : nullptr;
  }
  // the waves share the whole steps of K evenly; the last wave also takes the partial one
  const int whole = a.K / kStep;
  const int first = (int)((int64_t)wave * whole / kWaves), last = (int)((int64_t)(wave + 1) * whole / kWaves);
  const bool tail = wave == kWaves - 1 && whole * kStep < a.K;

  for (; m0 < m1; m0 += 16 * MB) {
    floatx4_t acc[MB][CB], d[MB][CB];
    const uint16_t* xrow[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) { // rows past the last read the last one and are not stored
      xrow[b] = a.x + (int64_t)min(m0 + 16 * b + s, m1 - 1) * a.ldx + 8 * g;
#pragma unroll
      for (int c = 0; c < CB; ++c) acc[b][c] = d[b][c] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    }

    struct Step { // what one step reads of the weights
      u32x4 w[CB];
      uint32_t sc[CB][SR], z[CB];
    };
    auto load = [&](Step& t, int step) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        t.w[c] = *reinterpret_cast<const u32x4_any*>(wrow[c] + (int64_t)step * (kStep / 2));
        __builtin_memcpy(t.sc[c], srow[c] + (int64_t)step * GPS, 2 * GPS);
        if constexpr (FMT == kInt4Zero) __builtin_memcpy(&t.z[c], zrow[c] + (int64_t)step * GPS, GPS);
      }
    };
    // 32 k of x, k0 = 32 * sub
    auto load_x = [&](u32x4 (&x)[MB], int sub) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < MB; ++b) x[b] = *reinterpret_cast<const u32x4_any*>(xrow[b] + (int64_t)sub * 32);
    };
    // 4 x 4 transpose of a step's registers over the lane groups
    auto transpose = [&](Step& t) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        auto r = __builtin_amdgcn_permlane32_swap(t.w[c][0], t.w[c][2], false, false);
        auto u = __builtin_amdgcn_permlane32_swap(t.w[c][1], t.w[c][3], false, false);
        auto lo = __builtin_amdgcn_permlane16_swap(r[0], u[0], false, false);
        auto hi = __builtin_amdgcn_permlane16_swap(r[1], u[1], false, false);
        t.w[c] = u32x4{lo[0], lo[1], hi[0], hi[1]};
      }
    };
    // sub-step I of a step: 32 k of every block; a scale group's last one adds its sum to acc
    auto sub_step = [&](Step& t, u32x4 (&x)[MB], auto ic) __attribute__((always_inline)) {
      constexpr int I = decltype(ic)::value, P = I / SPG;
      frag_t xo[MB];
#pragma unroll
      for (int b = 0; b < MB; ++b) xo[b] = __builtin_bit_cast(frag_t, order_x<DT, FMT>(x[b]));
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        const uint32_t zz = zero_operand<DT, FMT>(FMT == kInt4Zero ? (t.z[c] >> (8 * P)) & 15u : 8u);
        const frag_t w = __builtin_bit_cast(frag_t, decode<DT, FMT>(t.w[c][I], zz));
#pragma unroll
        for (int b = 0; b < MB; ++b) d[b][c] = mfma(xo[b], w, I % SPG ? d[b][c] : floatx4_t{0.f, 0.f, 0.f, 0.f});
        if constexpr (I % SPG == SPG - 1) {
          const float sc = scale_value<DT>((uint16_t)(t.sc[c][P / 2] >> (16 * (P & 1))));
#pragma unroll
          for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[b][c][r] = __builtin_fmaf(sc, d[b][c][r], acc[b][c][r]);
        }
      }
    };
    typedef std::integral_constant<int, 0> I0;
    typedef std::integral_constant<int, 1> I1;
    typedef std::integral_constant<int, 2> I2;
    typedef std::integral_constant<int, 3> I3;

    if (first < last) {
      u32x4 x[XD][MB]; // the next XD sub-steps of x
      const int last_sub = 4 * last - 1;
#pragma unroll
      for (int i = 0; i < XD; ++i) load_x(x[i], 4 * first + i);
      auto compute = [&](Step& t, int step) __attribute__((always_inline)) {
        transpose(t);
        auto sub = [&](auto ic) __attribute__((always_inline)) {
          constexpr int I = decltype(ic)::value;
          sub_step(t, x[I % XD], ic);
          // past the range the last one is read again, and not used
          load_x(x[I % XD], min(4 * step + I + XD, last_sub));
          __builtin_amdgcn_sched_barrier(0); // one sub-step's operands live at a time
        };
        sub(I0{});
        sub(I1{});
        sub(I2{});
        sub(I3{});
      };
      Step p, q;
      load(p, first);
      int t = first;
      for (; t + 1 < last; t += 2) {
        load(q, t + 1);
        compute(p, t);
        load(p, min(t + 2, last - 1));
        compute(q, t + 1);
      }
      if (t < last) compute(p, t);
    }
    if (tail) {
      // 32 k at a time, each lane its own four bytes and eight elements: nothing past a row's end
      // is read, and codes past K meet zeros of x
#pragma unroll 1
      for (int sub = 4 * whole; sub * 32 < a.K; ++sub) {
        const int xn = a.K - 32 * sub - 8 * g, wn = a.row_bytes - 16 * sub - 4 * g;
        u32x4 x[MB];
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t v = 0;
            if (2 * j < xn) v = xrow[b][32 * sub + 2 * j];
            if (2 * j + 1 < xn) v |= (uint32_t)xrow[b][32 * sub + 2 * j + 1] << 16;
            x[b][j] = v;
          }
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          const uint8_t* w = wrow[c] - 16 * g + 16 * sub + 4 * g;
          uint32_t v = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < wn) v |= (uint32_t)w[j] << (8 * j);
          uint32_t z = 8;
          if constexpr (FMT == kInt4Zero) z = zrow[c][sub / SPG] & 15u;
          const frag_t wf = __builtin_bit_cast(frag_t, decode<DT, FMT>(v, zero_operand<DT, FMT>(z)));
          const float sc = scale_value<DT>(srow[c][sub / SPG]);
#pragma unroll
          for (int b = 0; b < MB; ++b) {
            const floatx4_t one = mfma(__builtin_bit_cast(frag_t, order_x<DT, FMT>(x[b])), wf, floatx4_t{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[b][c][r] = __builtin_fmaf(sc, one[r], acc[b][c][r]);
          }
        }
      }
    }

#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < CB; ++c) red[wave][(c * MB + b) * 64 + lane] = acc[b][c];
    __syncthreads();
    for (int i = tid; i < CB * MB * 64; i += kWaves * 64) {
      floatx4_t v = red[0][i];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += red[w][i];
      const int l = i & 63, b = (i >> 6) % MB, c = (i >> 6) / MB;
      const int n = n0 + 16 * c + (l & 15), m = m0 + 16 * b + 4 * (l >> 4);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n < a.N && m + r < m1)
          a.y[(int64_t)(m + r) * a.N + n] = __builtin_bit_cast(uint16_t, to_out(v[r], (out_t*)nullptr));
    }
    __syncthreads();
  }
}

typedef void (*kernel_fn)(Args);
// The kernel for a format, group size, row blocks mb (1, 2 or 4) and column blocks cb (1, 2 or 4; up to 2 with mb = 4).
kernel_fn pick_f16(int fmt, int group, int mb, int cb);
kernel_fn pick_bf16(int fmt, int group, int mb, int cb);

template <int DT, int FMT, int GROUP>
kernel_fn pick_shape(int mb, int cb) {
  if (mb == 1) return cb == 1 ? w4_kernel<DT, FMT, GROUP, 1, 1> : cb == 2 ? w4_kernel<DT, FMT, GROUP, 1, 2> : w4_kernel<DT, FMT, GROUP, 1, 4>;
  if (mb == 2) return cb == 1 ? w4_kernel<DT, FMT, GROUP, 2, 1> : cb == 2 ? w4_kernel<DT, FMT, GROUP, 2, 2> : w4_kernel<DT, FMT, GROUP, 2, 4>;
  return cb == 1 ? w4_kernel<DT, FMT, GROUP, 4, 1> : w4_kernel<DT, FMT, GROUP, 4, 2>;
}
template <int DT, int FMT>
kernel_fn pick_group(int group, int mb, int cb) {
  return group == 32 ? pick_shape<DT, FMT, 32>(mb, cb) : group == 64 ? pick_shape<DT, FMT, 64>(mb, cb) : pick_shape<DT, FMT, 128>(mb, cb);
}
template <int DT>
kernel_fn pick(int fmt, int group, int mb, int cb) {
  return fmt == kInt4 ? pick_group<DT, kInt4>(group, mb, cb) : fmt == kInt4Zero ? pick_group<DT, kInt4Zero>(group, mb, cb) : pick_group<DT, kE2M1>(group, mb, cb);
}

} // namespace w4
} // namespace pgemm
