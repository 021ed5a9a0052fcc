// The linear layer: products of rows with one matrix, with what follows them
// in the epilogue, and the gradients.
//   z = x W + bias                      W: [K, C] ("K x N") or transposed, [C, K] ("N x K")
//   y = act(z) + residual               C = N
//   y = act(z[:, :N]) * z[:, N:] + residual   gated: C = 2N, gate columns first
//   dz = dy * act'(z)                   gated: dy * up * act'(gate) and dy * act(gate)
//   dbias = column sums of dz,  dx = dz W^T,  dW = x^T dz (or its transpose)
// Sums, activations and column sums are fp32; z, dz and the outputs are
// rounded once to the operands' 16 bits. Two of these roundings are not the
// outputs' own: dz's, which the matrix unit's operands need, and z's, the copy
// that the backward pass reads (in 32 bits it would double that traffic). In
// bf16 they take the gradients' error from 0.0017, one rounding's, to 0.0024,
// gated to 0.0030 (the gate's and up's rounding meet in one product).
//
// The products' bodies:
//   few   (dense_few.h)    up to 128 rows, in groups of 8, 16 or 32: reading W bounds it
//   tile  (dense_tile.h)   tiles of 128 (or 64) x 128 in two to six LDS stages, whole or cut along the sum
//   both  (dense_tile.h)   dx and dW of one backward pass as such tiles in one launch
//   ping  (dense_pp.h)     256 x 256 ping-pong tiles for large products
// tile and ping copy 16-byte chunks directly to LDS, so rows at other
// addresses are first moved to padded rows in the workspace (one pass over
// the operand; a body that loads odd rows itself runs at half the rate).
#pragma once

#include "dense_act.h"
#include "gemm_fast.h"
#include "moe_rows.h"

namespace pgemm {
namespace dense {

using moe::u32x4;

struct Args {
  const uint16_t *a, *b; // rows of x and W; weight gradient: rows of both operands
  int64_t lda, ldb;      // distance of two rows
  int64_t half;          // gated: elements between a gate column's and its up column's first
  uint16_t* c;           // [M][N], contiguous
  uint16_t* z;           // pre-activations [M][N or 2N], or null
  const uint16_t* bias;  // [N or 2N] or null
  const uint16_t* residual; // rows ldr apart, or null
  int64_t ldr;
  int M, N, K; // rows and columns of c, length of the sum
  int act;
  int n_m, n_n; // tiles
  int split;    // pieces the sum is cut into
  float* part;  // split > 1: their sums [split][M][columns of part_ld()]
};

// Columns of a piece's row: gate and up halves each a multiple of 8.
__host__ __device__ inline int64_t part_ld(const Args& a, bool gated) { return (int64_t)(gated ? 2 : 1) * ((a.N + 7) / 8 * 8); }

// Eight fp32 values to 16 bits, to the nearest, ties to even; a pair's conversion is one instruction for bf16.
template <int DT>
__device__ inline u32x4 pack(const float* f) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef typename Traits<DT>::out_t out2 __attribute__((ext_vector_type(2)));
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{f[2 * i], f[2 * i + 1]}), out2));
  return v;
}

// A pre-activation as the backward pass gets it. A finite one beyond fp16's range is stored as the type's largest value, not as
// an infinity: past 100 every activation's slope is 1 or 0, so it keeps its gradient (as 0 times infinity that would be NaN, for
// all of its row of dx and column of dW).
template <int DT>
__device__ inline float z_value(float v) {
  if constexpr (DT == kF16) return __builtin_fabsf(v) < __builtin_huge_valf() ? __builtin_amdgcn_fmed3f(v, -65504.0f, 65504.0f) : v;
  return v;
}

// Eight elements of a row, those past its end zeros.
__device__ inline u32x4 load8_upto(const uint16_t* row, int64_t n, int64_t N) {
  return n + 8 <= N ? moe::load8<moe::kAnyAddress>(row + n) : moe::load_part(row + n, (int)(N - n));
}

// What follows the sums of eight columns n .. n+7 of row m (n < N): v the sums
// (gated: of the gate), u those of up. The activation's path is chosen around
// the loops over a tile's rows (act::with_path), so that what runs lies together.
// EVEN: N is a multiple of 8.
template <int DT, bool GATED, bool EVEN = false>
struct Epilogue {
  const Args& a;
  const act::Consts k;
  __device__ explicit Epilogue(const Args& a_) : a(a_), k(act::consts_of(a_.act)) {}

  __device__ inline u32x4 load(const uint16_t* row, int n) const {
    return EVEN ? moe::load8<moe::kAnyAddress>(row + n) : load8_upto(row, n, a.N);
  }
  __device__ inline void store(uint16_t* row, int n, const float* v) const {
    if constexpr (EVEN) moe::store8<moe::kAnyAddress>(row + n, pack<DT>(v));
    else moe::store_row<moe::kAnyAddress>(row, n, a.N, pack<DT>(v));
  }

  // One test for the eight costs nothing that can be measured (4096 x 4096 x 2048 gated: 123.6 us without any, 123.9 with it);
  // putting each value right by itself costs 2%.
  __device__ inline void store_z(uint16_t* row, int n, const float* v) const {
    if constexpr (DT == kF16) {
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) most = __builtin_fmaxf(most, __builtin_fabsf(v[i]));
      if (__builtin_expect(__any(most > 65504.0f), 0)) {
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = z_value<DT>(v[i]);
        return store(row, n, z);
      }
    }
    store(row, n, v);
  }

  __device__ inline void bias_of(int n, float* bv, float* bu) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) bv[i] = 0.0f;
    if constexpr (GATED) {
#pragma unroll
      for (int i = 0; i < 8; ++i) bu[i] = 0.0f;
    }
    if (!a.bias || n >= a.N) return;
    moe::unpack<DT>(load(a.bias, n), bv);
    if constexpr (GATED) moe::unpack<DT>(load(a.bias + a.N, n), bu);
  }

  template <int PATH>
  __device__ inline void finish(int m, int n, float* v, float* u, const float* bv, const float* bu) const {
    const int64_t N = a.N;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] += bv[i];
      if constexpr (GATED) u[i] += bu[i];
    }
    if (a.z) {
      uint16_t* z = a.z + (int64_t)m * (GATED ? 2 * N : N);
      store_z(z, n, v);
      if constexpr (GATED) store_z(z + N, n, u);
    }
    u32x4 res = {0, 0, 0, 0};
    if (a.residual) res = load(a.residual + m * a.ldr, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = act::value<PATH>(v[i], k);
      if constexpr (GATED) v[i] *= u[i];
    }
    if (a.residual) {
      float r[8];
      moe::unpack<DT>(res, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    moe::store_row<moe::kAnyAddress>(a.c + (int64_t)m * N, n, (int)N, pack<DT>(v));
  }
};

// Steps 0 .. n-1 with D of them in flight (two where there are fewer than D): load(slot, step) into registers,
// multiply(slot). Loads past the last step are of that step again and not used: after a branch around a load the
// compiler would wait for more than it has to.
template <int D, class Slot, class L, class F>
__device__ inline void stream_loop(int n, L load, F multiply) {
  Slot t[D];
#pragma unroll
  for (int j = 0; j < D; ++j) load(t[j], min(j, n - 1));
  for (int i = 0; i < n; i += D) {
#pragma unroll
    for (int j = 0; j < D; ++j) {
      if (i + j < n) multiply(t[j]);
      load(t[j], min(i + j + D, n - 1));
    }
  }
}
template <int D, class Slot, class L, class F>
__device__ inline void stream_steps(int n, L load, F multiply) {
  if (n >= D) stream_loop<D, Slot>(n, load, multiply);
  else if (n > 0) stream_loop<D < 2 ? D : 2, Slot>(n, load, multiply);
}

// load16_to_lds as an instruction of its own: of the builtin the compiler knows that it writes LDS, but not which stage,
// and it waits ahead of a stage's reads for copies in flight into another, which leaves one step in flight (128 steps of a
// 128 x 128 tile on every CU: 73.6 us, now 69.3). The kernel's own waits cover every copy; M0 holds the wave's LDS address.
__device__ inline void copy16(intx4_t rsrc, uint32_t lds, uint32_t voffset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voffset), "s"(rsrc)
               : "memory", "m0");
}
__device__ inline intx4_t rsrc_words(const void* base) { // make_rsrc's four words
  const uint64_t p = (uint64_t)base;
  return intx4_t{(int)(uint32_t)p, (int)((uint32_t)(p >> 32) & 0xFFFFu), 0x7FFFFFFF, kRsrcWord3};
}

// The step range of piece `piece`: first step and steps of 64.
__device__ inline void piece_steps(int K, int split, int piece, int* first, int* count) {
  const int steps = (K + 63) / 64;
  const int lo = (int)((int64_t)steps * piece / split), hi = (int)((int64_t)steps * (piece + 1) / split);
  *first = lo;
  *count = hi - lo;
}

// Rows form: W as K x N or N x K; gradient form: c = a^T b over the rows of both.
enum Form : int { kRowsKN = 0, kRowsNK = 1, kGrad = 2 };
// kTile64 has six LDS stages and kTile128 five, and a CU to itself; kTile128Pair has two, two workgroups to a CU.
enum Body : int { kFew8, kFew16, kFew32, kTile64, kTile128, kTile128Pair, kPing };
typedef void (*kernel_fn)(Args);

// dz and the column sums of it (dense_rows.h).
struct ActGradArgs {
  const uint16_t* dy; // rows lddy apart
  int64_t lddy;
  const uint16_t* z;  // [M][C] contiguous (null for act none)
  uint16_t* dz;       // null: only the sums are wanted
  int64_t lddz;
  float* part;        // null: no sums
  uint16_t* db;
  int M, N, act;
  int stretches;
  int stream; // N a multiple of 8: read dy and z past the memory-side cache
};
// Rows of `halves` x `cols` elements, ld apart, to rows in which each half starts at a multiple of 8 and is
// filled up with zeros.
struct PadArgs {
  const uint16_t* from;
  int64_t ld;
  uint16_t* to;
  int rows, cols, halves;
  int chunks; // of a half, eight elements each
};
// What goes into one launch ahead of the products: up to two operands moved, the column sums joined.
struct SideArgs {
  PadArgs pad[2];
  int pad_blocks[2]; // 256 chunks each
  ActGradArgs sums;
  int C; // columns to sum, 64 a block; 0: none
};

struct Kernels {
  kernel_fn (*pick)(int body, int form, bool gated);
  kernel_fn join[2]; // by gated
  void (*(*pick_both)(int body, int form))(Args, Args, int, int);
  void (*join_both)(Args, Args, int);
  void (*act_grad[2])(ActGradArgs);
  void (*side)(SideArgs);
};
Kernels kernels_f16();
Kernels kernels_bf16();

} // namespace dense
} // namespace pgemm
