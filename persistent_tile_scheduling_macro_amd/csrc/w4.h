// Few rows times 4-bit weights: y[m][n] = sum_k x[m][k] * dec(q[n][k]), with
//   dec = (code - z[n][k / group]) * s[n][k / group]   (int4; z = 8 without zero points)
//   dec = e2m1(code) * s[n][k / group]                 (sign, two exponent bits, one mantissa bit)
// Codes lie along K, two to a byte, the lower nibble first.
//
// The codes' bytes bound it: each is read once and used for up to 32 rows of
// x. A wave owns CB blocks of 16 columns and a range of K, 128 k a step. The
// MFMA wants column s in lane (g, s), but loads in that layout make every
// lane a request of its own (consecutive lanes lie a row apart), and the
// address unit then bounds it (16 x 16384 x 8192: 41 us). So loads of codes,
// x and scales run along the rows, and each wave turns them in its own LDS:
//   codes   four lanes read 64 bytes of a column; lane (g, s) takes the four
//           bytes 16 i + 4 g of column s for sub-step i, 32 k in one MFMA, all
//           in one scale group;
//   x       16 lanes read 256 bytes of a row; operands of 16 bytes;
//   scales, zero points   read for 32 groups at a time.
// 16 x 16384 x 8192 with zero points now takes 22 us (3.6 TB/s), e2m1 without 18.8
// us; decoding and the turns through LDS keep it from the reads' own 13 us.
//
// Codes become operands without rounding: code - z is a whole number up to
// 15 and an e2m1 value has two significant bits, so both are exact in either
// type, and the MFMA sums exact products in fp32. The group's scale multiplies
// that sum, also in fp32; a weight is never rounded to 16 bits.
//
// The waves of a workgroup split K between them (K is long and the rows are
// few) and their sums are joined in LDS in a fixed order.
#pragma once

#include "moe_rows.h"

namespace pgemm {
namespace w4 {

enum Fmt : int { kInt4 = 0, kInt4Zero = 1, kE2M1 = 2 };
constexpr int kStep = 128; // k of one load: 4 lane groups x 16 bytes
// Waves of a workgroup: with 32 rows a wave's operands take 160 registers, and three workgroups of four waves fit a CU
// where one of eight would.
constexpr int waves_of(int rows) { return rows == 32 ? 4 : 8; }

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(1)));
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

// ROWS: rows of x taken at once, 4, 16 or 32 (4 reads only those; the MFMA always has 16).
template <int DT, int FMT, int GROUP, int ROWS, int CB>
__global__ void __launch_bounds__(waves_of(ROWS) * 64, ROWS == 32 ? 3 : 4) w4_kernel(Args a) {
  constexpr int kWaves = waves_of(ROWS);
  constexpr int MB = (ROWS + 15) / 16, XL = ROWS / 4; // row blocks; loads of x a step
  constexpr int GPS = kStep / GROUP;                  // scale groups of a step
  constexpr int SPG = GROUP / 32;                     // MFMA k-groups of a scale group
  constexpr int GC = 32, CHUNK = GC / GPS;            // scale groups kept at a time, their steps
  constexpr int D = ROWS == 32 ? 1 : 2; // steps in registers; with 32 rows a step is loaded again as soon as it is in LDS
  constexpr int XH = ROWS == 32 ? 2 : 1;              // parts in which x goes through LDS
  constexpr int SROW = 2 * GC + 4, ZROW = GC + 4;     // LDS rows of scales and zero points, off the banks' period
  constexpr int XROW = 256 / XH, XB = ROWS * XROW, WB = CB * 1024, SB = CB * 16 * SROW, ZB = FMT == kInt4Zero ? CB * 16 * ZROW : 0;
  constexpr int TURN = (XB + WB + SB + ZB + 15) / 16 * 16, JOIN = CB * MB * 1024;
  typedef typename Frag<DT>::t frag_t;
  typedef typename Traits<DT>::out_t out_t;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kWaves * (TURN > JOIN ? TURN : JOIN)];

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
    m0 = blockIdx.y * ROWS;
    m1 = min(m0 + ROWS, a.M);
  }
  if (m0 >= m1) return;

  uint8_t *turn_x = lds + wave * TURN, *turn_w = turn_x + XB, *turn_s = turn_w + WB, *turn_z = turn_s + SB;
  // a load's lanes: four to a column (codes, scales), 16 to a row of x (8 where x goes in two parts)
  constexpr int XC = 16 / XH, XR = 64 / XC; // chunks of a row part, rows of a load
  const int wcol = lane >> 2, wpart = lane & 3, xr = lane / XC, xpart = lane % XC;
  const uint8_t* wp[CB];
  auto column = [&](int c) __attribute__((always_inline)) { // columns past N read the last one and are not stored
    return (int64_t)e * a.N + min(n0 + 16 * c + wcol, a.N - 1);
  };
#pragma unroll
  for (int c = 0; c < CB; ++c) wp[c] = a.q + column(c) * a.row_bytes + 16 * wpart;
  // the waves share the whole steps of K evenly; the 32-k pieces behind them go to one wave each
  const int whole = a.K / kStep;
  const int first = (int)((int64_t)wave * whole / kWaves), last = (int)((int64_t)(wave + 1) * whole / kWaves);

  auto x_swizzle = [](int row) __attribute__((always_inline)) { return XROW == 256 ? 2 * (row & 7) : row & 7; };
  auto wave_fence = [&]() __attribute__((always_inline)) { // LDS serves a wave in order: only the compiler has to be held
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };

  for (; m0 < m1; m0 += ROWS) {
    floatx4_t acc[MB][CB], d[MB][CB];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < CB; ++c) acc[b][c] = d[b][c] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    const uint16_t* xp[XL / XH];
#pragma unroll
    for (int i = 0; i < XL / XH; ++i) // rows past the last read the last one and are not stored
      xp[i] = a.x + min(m0 + XR * i + xr, m1 - 1) * a.ldx + 8 * xpart;

    struct Step { // what one step reads
      u32x4 w[CB], x[XH][XL / XH];
    };
    auto load = [&](Step& t, int step) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < CB; ++c) t.w[c] = *reinterpret_cast<const u32x4_any*>(wp[c] + (int64_t)step * (kStep / 2));
#pragma unroll
      for (int h = 0; h < XH; ++h)
#pragma unroll
        for (int i = 0; i < XL / XH; ++i)
          t.x[h][i] = *reinterpret_cast<const u32x4_any*>(xp[i] + (int64_t)step * kStep + h * (kStep / XH));
    };
    // scales and zero points of the GC groups from step's first on
    auto refill = [&](int step) __attribute__((always_inline)) {
      const int g0 = step * GPS + 8 * wpart, left = a.groups - g0;
#pragma unroll 1 // not in a hurry, and its registers are needed elsewhere
      for (int c = 0; c < CB; ++c) {
        const uint16_t* sp = a.scales + column(c) * a.groups + g0;
        u32x4 v = {0, 0, 0, 0};
        if (left >= 8) v = *reinterpret_cast<const u32x4_any*>(sp);
        else if (left > 0) v = moe::load_part(sp, left);
        uint32_t* at = reinterpret_cast<uint32_t*>(turn_s + (16 * c + wcol) * SROW + 16 * wpart);
#pragma unroll
        for (int j = 0; j < 4; ++j) at[j] = v[j];
        if constexpr (FMT == kInt4Zero) {
          const uint8_t* zp = a.zeros + column(c) * a.groups + g0;
          uint32_t z[2] = {0, 0};
          if (left >= 8) {
            __builtin_memcpy(z, zp, 8);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j < left) z[j >> 2] |= (uint32_t)zp[j] << (8 * (j & 3));
          }
          uint32_t* to = reinterpret_cast<uint32_t*>(turn_z + (16 * c + wcol) * ZROW + 8 * wpart);
          to[0] = z[0];
          to[1] = z[1];
        }
      }
    };
    auto compute = [&](Step& t, int step) __attribute__((always_inline)) {
      auto write_x = [&](int h) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < XL / XH; ++i) {
          const int r = XR * i + xr;
          *reinterpret_cast<u32x4*>(turn_x + r * XROW + 16 * (xpart ^ x_swizzle(r))) = t.x[h][i];
        }
      };
      wave_fence(); // the last step's reads come first
      write_x(0);
#pragma unroll
      for (int c = 0; c < CB; ++c)
        *reinterpret_cast<u32x4*>(turn_w + c * 1024 + wcol * 64 + 16 * (wpart ^ (wcol >> 2))) = t.w[c];
      if ((step - first) % CHUNK == 0) refill(step);
      wave_fence();
      const int gr = (step - first) % CHUNK * GPS;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (XH == 2 && i == 2) {
          wave_fence();
          write_x(1);
          load(t, min(step + D, last - 1)); // past the range the last one again, not used
          wave_fence();
        }
        frag_t xo[MB];
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          const int r = ROWS == 4 ? s & 3 : 16 * b + s, chunk = 4 * (i % (4 / XH)) + g;
          xo[b] = __builtin_bit_cast(
              frag_t, order_x<DT, FMT>(*reinterpret_cast<const u32x4*>(turn_x + r * XROW + 16 * (chunk ^ x_swizzle(r)))));
        }
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          const int p = gr + i / SPG;
          const uint32_t v = *reinterpret_cast<const uint32_t*>(turn_w + c * 1024 + s * 64 + 16 * (i ^ (s >> 2)) + 4 * g);
          const uint32_t zz = zero_operand<DT, FMT>(FMT == kInt4Zero ? turn_z[(16 * c + s) * ZROW + p] & 15u : 8u);
          const frag_t w = __builtin_bit_cast(frag_t, decode<DT, FMT>(v, zz));
#pragma unroll
          for (int b = 0; b < MB; ++b) d[b][c] = mfma(xo[b], w, i % SPG ? d[b][c] : floatx4_t{0.f, 0.f, 0.f, 0.f});
          if (i % SPG == SPG - 1) { // a scale group is complete
            const float sc = scale_value<DT>(*reinterpret_cast<const uint16_t*>(turn_s + (16 * c + s) * SROW + 2 * p));
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[b][c][r] = __builtin_fmaf(sc, d[b][c][r], acc[b][c][r]);
          }
        }
      }
    };

    if (first < last) {
      Step t[D];
#pragma unroll
      for (int j = 0; j < D; ++j) load(t[j], min(first + j, last - 1));
      for (int i = first; i < last; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
          if (i + j < last) compute(t[j], i + j);
          if (XH == 1) load(t[j], min(i + j + D, last - 1));
        }
      }
    }
    // each lane its own four bytes and eight elements of a piece: nothing past a row's end is read,
    // and codes past K meet zeros of x
    for (int sub = 4 * whole + kWaves - 1 - wave; sub * 32 < a.K; sub += kWaves) {
      const int xn = a.K - 32 * sub - 8 * g, wn = a.row_bytes - 16 * sub - 4 * g;
      u32x4 x[MB];
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const uint16_t* xrow = a.x + min(m0 + 16 * b + s, m1 - 1) * a.ldx + 32 * sub + 8 * g;
        x[b] = xn >= 8 ? *reinterpret_cast<const u32x4_any*>(xrow) : xn > 0 ? moe::load_part(xrow, xn) : u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        const int64_t n = (int64_t)e * a.N + min(n0 + 16 * c + s, a.N - 1);
        const uint8_t* w = a.q + n * a.row_bytes + 16 * sub + 4 * g;
        uint32_t v = 0;
        if (wn >= 4) {
          __builtin_memcpy(&v, w, 4);
        } else {
#pragma unroll
          for (int j = 0; j < 3; ++j)
            if (j < wn) v |= (uint32_t)w[j] << (8 * j);
        }
        const int64_t at = n * a.groups + sub / SPG;
        const uint32_t z = FMT == kInt4Zero ? a.zeros[at] & 15u : 8u;
        const frag_t wf = __builtin_bit_cast(frag_t, decode<DT, FMT>(v, zero_operand<DT, FMT>(z)));
        const float sc = scale_value<DT>(a.scales[at]);
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          const floatx4_t one = mfma(__builtin_bit_cast(frag_t, order_x<DT, FMT>(x[b])), wf, floatx4_t{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[b][c][r] = __builtin_fmaf(sc, one[r], acc[b][c][r]);
        }
      }
    }

    __syncthreads(); // every wave is through with its part of the LDS
    floatx4_t* join = reinterpret_cast<floatx4_t*>(lds);
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < CB; ++c) join[(wave * CB * MB + c * MB + b) * 64 + lane] = acc[b][c];
    __syncthreads();
    const int end = min(m1, m0 + ROWS); // of this pass: with four rows at once the MFMA's other twelve repeat them
    for (int i = tid; i < CB * MB * 64; i += kWaves * 64) {
      floatx4_t v = join[i];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += join[w * CB * MB * 64 + i];
      const int l = i & 63, b = (i >> 6) % MB, c = (i >> 6) / MB;
      const int n = n0 + 16 * c + (l & 15), m = m0 + 16 * b + 4 * (l >> 4);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n < a.N && m + r < end)
          a.y[(int64_t)(m + r) * a.N + n] = __builtin_bit_cast(uint16_t, to_out(v[r], (out_t*)nullptr));
    }
    __syncthreads();
  }
}

typedef void (*kernel_fn)(Args);
// The kernel for a format, group size, rows at once (4, 16 or 32) and column blocks (1 or 2).
kernel_fn pick_f16(int fmt, int group, int rows, int cb);
kernel_fn pick_bf16(int fmt, int group, int rows, int cb);

template <int DT, int FMT, int GROUP>
kernel_fn pick_shape(int rows, int cb) {
  if (rows == 4) return cb == 1 ? w4_kernel<DT, FMT, GROUP, 4, 1> : w4_kernel<DT, FMT, GROUP, 4, 2>;
  if (rows == 16) return cb == 1 ? w4_kernel<DT, FMT, GROUP, 16, 1> : w4_kernel<DT, FMT, GROUP, 16, 2>;
  return cb == 1 ? w4_kernel<DT, FMT, GROUP, 32, 1> : w4_kernel<DT, FMT, GROUP, 32, 2>;
}
template <int DT, int FMT>
kernel_fn pick_group(int group, int rows, int cb) {
  return group == 32   ? pick_shape<DT, FMT, 32>(rows, cb)
         : group == 64 ? pick_shape<DT, FMT, 64>(rows, cb)
                       : pick_shape<DT, FMT, 128>(rows, cb);
}
template <int DT>
kernel_fn pick(int fmt, int group, int rows, int cb) {
  return fmt == kInt4       ? pick_group<DT, kInt4>(group, rows, cb)
         : fmt == kInt4Zero ? pick_group<DT, kInt4Zero>(group, rows, cb)
                            : pick_group<DT, kE2M1>(group, rows, cb);
}

} // namespace w4
} // namespace pgemm
