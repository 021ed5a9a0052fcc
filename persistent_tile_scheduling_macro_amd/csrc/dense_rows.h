// What stands around the linear layer's products: the pieces' sums joined, dz
// with the bias' column sums, rows moved to padded ones.
#pragma once

#include "dense.h"

namespace pgemm {
namespace dense {

// c = epilogue(sum of the pieces' sums), eight columns a thread, pieces in order.
template <int DT, bool GATED>
__device__ inline void join_pieces(const Args& a, int block) {
  const int chunks = (a.N + 7) / 8;
  const int64_t i = (int64_t)block * 256 + threadIdx.x, m = i / chunks;
  if (m >= a.M) return;
  const int n = (int)(i - m * chunks) * 8;
  const int64_t ld = part_ld(a, GATED), stride = a.M * ld;
  const float* p = a.part + m * ld + n;
  const Epilogue<DT, GATED> epilogue(a);
  float bv[8], bu[8];
  epilogue.bias_of(n, bv, bu);
  floatx4_t s[GATED ? 4 : 2];
#pragma unroll
  for (int j = 0; j < (GATED ? 4 : 2); ++j) s[j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int o = 0; o < a.split; ++o) {
    const float* r = p + o * stride;
    s[0] += *reinterpret_cast<const floatx4_t*>(r);
    s[1] += *reinterpret_cast<const floatx4_t*>(r + 4);
    if constexpr (GATED) {
      s[2] += *reinterpret_cast<const floatx4_t*>(r + ld / 2);
      s[3] += *reinterpret_cast<const floatx4_t*>(r + ld / 2 + 4);
    }
  }
  float v[8], u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = s[j / 4][j % 4];
    if constexpr (GATED) u[j] = s[2 + j / 4][j % 4];
  }
  act::with_path(epilogue.k, [&](auto path) __attribute__((always_inline)) {
    epilogue.template finish<decltype(path)::value>((int)m, n, v, u, bv, bu);
  });
}
template <int DT, bool GATED>
__global__ void __launch_bounds__(256) join_kernel(Args a) {
  join_pieces<DT, GATED>(a, blockIdx.x);
}
// Of two products, the first one in `head` workgroups.
template <int DT>
__global__ void __launch_bounds__(256) join_both_kernel(Args a, Args b, int head) {
  if ((int)blockIdx.x < head) join_pieces<DT, false>(a, blockIdx.x);
  else join_pieces<DT, false>(b, blockIdx.x - head);
}

// dz and the column sums of it. A workgroup takes 512 columns of y (a wave's
// reads are 1 KiB of a row) and a stretch of the rows, a thread eight columns and every fourth row; the
// threads' sums meet in LDS, the stretches' in `part` [stretches][C], which
// side_kernel adds in order. dz rows are ldz apart (a multiple of 8),
// filled up with zeros: they are the operands of the two products that follow.
// dy and z that the memory-side cache cannot hold beside dz are read past it (8192 x 8192 with dz: 12 us less; 4096 x 2048
// would take 26 us for 22). The bytes bound it: 8192 x 8192 with dz 80 us, 5.1 TB/s; the column sums alone 49 us, with 256
// columns a workgroup 61.
template <int DT, bool GATED>
__global__ void __launch_bounds__(256) act_grad_kernel(ActGradArgs a) {
  __shared__ float sums[4][GATED ? 2 : 1][512];
  const int tid = threadIdx.x, lane = tid & 63, strip = tid >> 6;
  const int n = blockIdx.x * 512 + 8 * lane;
  const int64_t C = GATED ? 2 * (int64_t)a.N : a.N;
  const int lo = (int)((int64_t)a.M * blockIdx.y / a.stretches), hi = (int)((int64_t)a.M * (blockIdx.y + 1) / a.stretches);
  const act::Consts k = act::consts_of(a.act);
  const bool live = n < a.N;
  float sv[8], su[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sv[i] = su[i] = 0.0f;
  // A row's eight columns: d the gradient, v (and u) the pre-activations, then dz.
  auto one_row = [&](auto path, auto with_z, int m, u32x4 dr, u32x4 vr, u32x4 ur) __attribute__((always_inline)) {
    float d[8], v[8], u[8];
    moe::unpack<DT>(dr, d);
    if constexpr (decltype(with_z)::value) {
      moe::unpack<DT>(vr, v);
      if constexpr (GATED) moe::unpack<DT>(ur, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float slope;
        const float value = act::value_and_slope<decltype(path)::value>(v[i], k, &slope);
        if constexpr (GATED) {
          v[i] = d[i] * u[i] * slope;
          u[i] = d[i] * value;
        } else {
          v[i] = d[i] * slope;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = d[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sv[i] += v[i];
      if constexpr (GATED) su[i] += u[i];
    }
    if (a.dz) {
      uint16_t* to = a.dz + m * a.lddz;
      moe::store_row<moe::kAnyAddress>(to, n, a.N, pack<DT>(v));
      if constexpr (GATED) moe::store_row<moe::kAnyAddress>(to + a.N, n, a.N, pack<DT>(u));
      if (n + 8 >= a.N) // the row's last thread fills it up
        for (int64_t j = C; j < a.lddz; ++j) to[j] = 0;
    }
  };
  auto rows = [&](auto path, auto with_z, auto stream) __attribute__((always_inline)) {
    auto eight = [&](const uint16_t* row) __attribute__((always_inline)) {
      if constexpr (decltype(stream)::value) return __builtin_nontemporal_load(reinterpret_cast<const moe::u32x4_any*>(row + n));
      else return load8_upto(row, n, a.N);
    };
    constexpr bool Z = decltype(with_z)::value;
    const u32x4 none = {0, 0, 0, 0};
#pragma unroll 2
    for (int64_t m = lo + strip; m < hi; m += 4)
      one_row(path, with_z, (int)m, eight(a.dy + m * a.lddy), Z ? eight(a.z + m * C) : none, Z && GATED ? eight(a.z + m * C + a.N) : none);
  };
  if (live) {
    if (GATED || a.z) {
      act::with_path(k, [&](auto path) __attribute__((always_inline)) {
        if (a.stream) rows(path, std::true_type{}, std::true_type{});
        else rows(path, std::true_type{}, std::false_type{});
      });
    } else {
      rows(std::integral_constant<int, act::kCopy>{}, std::false_type{}, std::false_type{});
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sums[strip][0][8 * lane + i] = sv[i];
    if constexpr (GATED) sums[strip][1][8 * lane + i] = su[i];
  }
  __syncthreads();
#pragma unroll
  for (int c = tid; c < 512; c += 256) {
    const int col = blockIdx.x * 512 + c;
    if (col >= a.N) break;
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
      float t = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) t += sums[j][h][c];
      a.part[(int64_t)blockIdx.y * C + (int64_t)h * a.N + col] = t;
    }
  }
}

// What the products wait for, in one launch (each would take some 5 us of its own): rows moved, one chunk of eight a
// thread; db as the sum of the stretches' sums, four threads a column.
template <int DT>
__global__ void __launch_bounds__(256) side_kernel(SideArgs a) {
  typedef typename Traits<DT>::out_t out_t;
  __shared__ float sums[4][64];
  int block = blockIdx.x;
  for (int k = 0; k < 2; ++k) {
    if (block < a.pad_blocks[k]) {
      const PadArgs& p = a.pad[k];
      const int per = p.chunks * p.halves;
      const int64_t i = (int64_t)block * 256 + threadIdx.x, r = i / per;
      if (r >= p.rows) return;
      const int at = (int)(i - r * per), h = at >= p.chunks ? 1 : 0, c = 8 * (at - h * p.chunks);
      const u32x4 v = load8_upto(p.from + r * p.ld + (int64_t)h * p.cols, c, p.cols);
      *reinterpret_cast<u32x4*>(p.to + 8 * i) = v;
      return;
    }
    block -= a.pad_blocks[k];
  }
  const int i = threadIdx.x & 63, col = block * 64 + i, part = threadIdx.x >> 6;
  float t = 0.0f;
  if (col < a.C) {
#pragma unroll 4
    for (int j = part; j < a.sums.stretches; j += 4) t += a.sums.part[(int64_t)j * a.C + col];
  }
  sums[part][i] = t;
  __syncthreads();
  if (part || col >= a.C) return;
  t = (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
  a.sums.db[col] = __builtin_bit_cast(uint16_t, to_out(t, (out_t*)nullptr));
}

} // namespace dense
} // namespace pgemm
