// Kernels that take token rows to their experts and back.
//
// Slot s = t*k + j is choice j of token t. Its key is the expert it names,
// or E when it names none (a dropped slot). The sorted position of a slot is
//   p(s) = #{s' : key(s') < key(s)} + #{s' < s : key(s') = key(s)},
// a stable counting sort, so no result depends on the order in which
// workgroups run. Everything here moves rows or sums at most a few of them:
// the bytes of the sorted rows bound every kernel. 8192 tokens x 8 of 64
// experts, rows of 4096 bf16: the sort 6 + 10 us, the rows moved 103 us (5.9
// TB/s of reads and writes), gathered and summed 109 to 112 us (5.4 to 5.6),
// both gradients of combine 221 us (5.2); a large copy reaches 5.2.
#pragma once

#include "device_common.h"

namespace pgemm {
namespace moe {

constexpr int kThreads = 256;
constexpr int kMaxExperts = 1024;  // LDS counters of the sort: four waves' worth
constexpr int kTile = 1024;        // slots a workgroup of the sort takes at a time
constexpr int kMaxChunks = 256;    // workgroups of the sort (each reads all of their counts)

// Eight 16-bit elements. Rows whose length is no multiple of 8 start at any
// even address; gfx950 serves wide global accesses at such addresses, so
// both forms move 16 bytes a lane (AL only tells the compiler the alignment).
// kStream marks accesses that the memory-side cache should not keep: sorted
// rows of more bytes than it holds (256 MiB) are gone before anyone reads them
// again, but on their way push out what would be, and their writing back
// delays the next kernel. 65536 rows of 4096 bf16, dispatch and its gradient:
// 104 + 162 us with plain accesses, 105 + 109 us streamed; combine and its
// gradients 143 + 216 and 112 + 222. Rows that fit are faster kept (12297 of
// 2056 fp16: 13.5 + 21.6 us against 16.5 + 25.6).
enum Access : int { kAnyAddress = 0, kAligned = 1, kStream = 2 };
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <int AL>
__device__ inline u32x4 load8(const uint16_t* p) {
  if constexpr (AL == kStream) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  else if constexpr (AL) return *reinterpret_cast<const u32x4*>(p);
  else return *reinterpret_cast<const u32x4_any*>(p);
}
template <int AL>
__device__ inline void store8(uint16_t* p, u32x4 v) {
  if constexpr (AL == kStream) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
  else if constexpr (AL) *reinterpret_cast<u32x4*>(p) = v;
  else *reinterpret_cast<u32x4_any*>(p) = v;
}
// The last elements of a row: n < 8 of them, the rest read as zeros.
__device__ inline u32x4 load_part(const uint16_t* p, int n) {
  uint16_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : (uint16_t)0;
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = e[2 * i] | (uint32_t)e[2 * i + 1] << 16;
  return v;
}
// The elements from `by` (0..7) on, moved down, zeros behind them.
__device__ inline u32x4 shift_down(u32x4 v, int by) {
  uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
  if (by & 4) {
    lo = hi;
    hi = 0;
  }
  const int bits = 16 * (by & 3);
  if (bits) lo = lo >> bits | hi << (64 - bits);
  hi >>= bits;
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}
__device__ inline void store_part(uint16_t* p, u32x4 v, int n) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
}
template <int AL>
__device__ inline u32x4 load_row(const uint16_t* row, int h, int H) {
  return AL || h + 8 <= H ? load8<AL>(row + h) : load_part(row + h, H - h);
}
template <int AL>
__device__ inline void store_row(uint16_t* row, int h, int H, u32x4 v) {
  if (AL || h + 8 <= H) store8<AL>(row + h, v);
  else store_part(row + h, v, H - h);
}

template <int DT>
__device__ inline void unpack(u32x4 v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == kBF16) {
      f[2 * i] = __builtin_bit_cast(float, v[i] << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xFFFF0000u);
    } else {
      f[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)v[i]);
      f[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(v[i] >> 16));
    }
  }
}
// fp32 -> 16 bits, to the nearest, ties to even
template <int DT>
__device__ inline u32x4 pack(const float* f) {
  typedef typename Traits<DT>::out_t out_t;
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __builtin_bit_cast(uint16_t, to_out(f[2 * i], (out_t*)nullptr)) |
           (uint32_t)__builtin_bit_cast(uint16_t, to_out(f[2 * i + 1], (out_t*)nullptr)) << 16;
  return v;
}

struct SortArgs {
  const void* ids; // [T, k] contiguous
  int n, E;        // slots, experts
  int chunk;       // slots per workgroup, a multiple of kTile
  int* counts;     // [chunks][E + 1]
  int *offsets, *order, *pos;
};

template <class ID>
__device__ inline int key_of(const void* ids, int64_t s, int E) {
  const ID e = static_cast<const ID*>(ids)[s];
  return e >= 0 && e < E ? (int)e : E;
}

// Lanes of the wave that hold the same key (keys below 2^bits).
__device__ inline uint64_t same_key(int key, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b) & 1;
    const uint64_t v = __ballot(one);
    m &= one ? v : ~v;
  }
  return m;
}

// Counts of this wave's quarter of the chunk, in its row of cnt. Each key's
// first lane adds the whole wave's number, so no counter is shared and no
// atomic is needed, however few experts the slots go to.
template <class ID>
__device__ inline void count_quarter(const SortArgs& a, int64_t first, int64_t last, int* cnt, int bits) {
  const int lane = threadIdx.x & 63;
  for (int64_t s0 = first; s0 < last; s0 += 64) {
    const int64_t s = s0 + lane;
    const int key = s < last ? key_of<ID>(a.ids, s, a.E) : a.E + 1;
    const uint64_t m = same_key(key, bits);
    if (key <= a.E && (m & ((1ull << lane) - 1)) == 0) cnt[key] += __popcll(m);
  }
}

template <class ID>
__global__ void __launch_bounds__(kThreads) sort_count_kernel(SortArgs a) {
  __shared__ int cnt[4][kMaxExperts + 1];
  const int wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e <= a.E; e += kThreads) cnt[0][e] = cnt[1][e] = cnt[2][e] = cnt[3][e] = 0;
  __syncthreads();
  const int bits = 32 - __clz(a.E + 1);
  const int64_t first = (int64_t)blockIdx.x * a.chunk + (int64_t)wave * (a.chunk / 4);
  const int64_t last = first + a.chunk / 4 < a.n ? first + a.chunk / 4 : a.n;
  count_quarter<ID>(a, first, last, cnt[wave], bits);
  __syncthreads();
  for (int e = threadIdx.x; e <= a.E; e += kThreads)
    a.counts[(int64_t)blockIdx.x * (a.E + 1) + e] = cnt[0][e] + cnt[1][e] + cnt[2][e] + cnt[3][e];
}

// Exclusive sum over the workgroup's 256 threads.
__device__ inline int block_scan(int v, int* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(s, d);
    if (lane >= d) s += u;
  }
  if (lane == 63) part[wave] = s;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < 3; ++w)
    if (w < wave) before += part[w];
  return before + s - v;
}

// Places every slot of a chunk. A workgroup needs, per expert, how many
// slots all chunks and how many the chunks before its own hold; it sums
// those columns itself (chunks x E counts, some 16 KB at 65536 slots and 64
// experts, from the L2), which is cheaper than another launch. With few
// experts several threads share a column: one thread a column, its loads in
// a row, took 20 of the kernel's 22 us there.
template <class ID>
__global__ void __launch_bounds__(kThreads) sort_place_kernel(SortArgs a, int chunks) {
  __shared__ int run[4][kMaxExperts + 1];
  __shared__ int sum[2][kMaxExperts + 1]; // [0] all chunks, [1] those before this one, by share and key
  __shared__ int part[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e <= a.E; e += kThreads) run[0][e] = run[1][e] = run[2][e] = run[3][e] = 0;
  __syncthreads();
  const int bits = 32 - __clz(a.E + 1);
  const int64_t first = (int64_t)blockIdx.x * a.chunk + (int64_t)wave * (a.chunk / 4);
  const int64_t last = first + a.chunk / 4 < a.n ? first + a.chunk / 4 : a.n;
  count_quarter<ID>(a, first, last, run[wave], bits);
  const int keys = a.E + 1, shares = keys < kThreads ? kThreads / keys : 1;
  for (int i = tid; i < keys * shares; i += kThreads) {
    const int e = i % keys;
    int all = 0, before = 0;
#pragma unroll 8
    for (int c = i / keys; c < chunks; c += shares) {
      const int v = a.counts[(int64_t)c * keys + e];
      all += v;
      before += c < (int)blockIdx.x ? v : 0;
    }
    sum[0][i] = all;
    sum[1][i] = before;
  }
  __syncthreads();
  // thread i owns experts i*per .. i*per + per - 1 (keys in order, so one scan orders them)
  constexpr int kPer = (kMaxExperts + kThreads) / kThreads;
  const int per = (a.E + kThreads) / kThreads;
  int total[kPer], before[kPer], mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * per + i;
    total[i] = before[i] = 0;
    if (i < per && e <= a.E) {
      for (int c = 0; c < shares; ++c) {
        total[i] += sum[0][c * keys + e];
        before[i] += sum[1][c * keys + e];
      }
    }
    mine += total[i];
  }
  int base = block_scan(mine, part);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * per + i;
    if (i < per && e <= a.E) {
      if (blockIdx.x == 0) a.offsets[e] = base;
      int at = base + before[i];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int v = run[w][e];
        run[w][e] = at;
        at += v;
      }
    }
    base += total[i];
  }
  __syncthreads();
  for (int64_t s0 = first; s0 < last; s0 += 64) {
    const int64_t s = s0 + lane;
    const int key = s < last ? key_of<ID>(a.ids, s, a.E) : a.E + 1;
    const uint64_t m = same_key(key, bits);
    if (key <= a.E) {
      const uint64_t below = m & ((1ull << lane) - 1);
      const int p = run[wave][key] + __popcll(below);
      const bool kept = key < a.E;
      a.pos[s] = kept ? p : -1;
      a.order[p] = kept ? (int)s : -1;
    }
    __builtin_amdgcn_wave_barrier(); // every lane has read its counter
    if (key <= a.E && (m & ((1ull << lane) - 1)) == 0) run[wave][key] += __popcll(m);
    __builtin_amdgcn_wave_barrier();
  }
}

struct MoveArgs {
  const uint16_t* x;
  int64_t ldx;
  uint16_t* xs;
  const int* pos;
  const int* offsets;
  int T, k, E, H, n;
  int token_blocks; // workgroups that move tokens; those behind them clear dropped rows
};

// Rows [offsets[E], n) belong to no slot: zeros. One contiguous range.
__device__ inline void clear_tail(uint16_t* rows, const int* offsets, int E, int n, int H, int part, int parts) {
  int kept = offsets[E];
  kept = kept < 0 ? 0 : kept > n ? n : kept;
  const int64_t from = (int64_t)kept * H, to = (int64_t)n * H;
  for (int64_t i = from + ((int64_t)part * kThreads + threadIdx.x) * 8; i < to; i += (int64_t)parts * kThreads * 8) {
    if (i + 8 <= to) store8<kAnyAddress>(rows + i, u32x4{0, 0, 0, 0});
    else store_part(rows + i, u32x4{0, 0, 0, 0}, (int)(to - i));
  }
}

// LANES lanes carry one token: its row is read once and written to the
// position of each of its slots.
template <int AL, int LANES>
__global__ void __launch_bounds__(kThreads) move_kernel(MoveArgs a) {
  if ((int)blockIdx.x >= a.token_blocks) {
    clear_tail(a.xs, a.offsets, a.E, a.n, a.H, blockIdx.x - a.token_blocks, gridDim.x - a.token_blocks);
    return;
  }
  const int64_t t = (int64_t)blockIdx.x * (kThreads / LANES) + __builtin_amdgcn_readfirstlane(threadIdx.x / LANES);
  if (t >= a.T) return;
  const uint16_t* row = a.x + t * a.ldx;
  const int* pos = a.pos + t * a.k;
  for (int h = (threadIdx.x % LANES) * 8; h < a.H; h += LANES * 8) {
    const u32x4 v = load_row<AL != 0>(row, h, a.H);
    for (int j = 0; j < a.k; ++j) {
      const int p = pos[j];
      if ((unsigned)p < (unsigned)a.n) store_row<AL>(a.xs + (int64_t)p * a.H, h, a.H, v);
    }
  }
}

// The whole of dispatch in one launch, for few slots: a workgroup per token
// finds the positions of its own slots by comparing them with every other
// (n*k/256 compares a thread, no wait for another workgroup), then moves the
// row. The last workgroup writes the offsets.
template <class ID, int AL>
__global__ void __launch_bounds__(kThreads) dispatch_small_kernel(SortArgs s, MoveArgs a) {
  __shared__ int cnt[kMaxExperts + 1];
  __shared__ int part[4];
  __shared__ int found[4][8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = a.n, E = a.E, k = a.k;
  if ((int)blockIdx.x == a.T) {
    for (int e = tid; e <= E; e += kThreads) cnt[e] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) atomicAdd(&cnt[key_of<ID>(s.ids, i, E)], 1);
    __syncthreads();
    const int per = (E + kThreads) / kThreads;
    int mine = 0;
    for (int i = 0; i < per; ++i)
      if (tid * per + i <= E) mine += cnt[tid * per + i];
    int base = block_scan(mine, part);
    for (int i = 0; i < per; ++i) {
      const int e = tid * per + i;
      if (e <= E) {
        s.offsets[e] = base;
        base += cnt[e];
      }
    }
    return;
  }
  const int t = blockIdx.x;
  const uint16_t* row = a.x + (int64_t)t * a.ldx;
  for (int j0 = 0; j0 < k; j0 += 8) {
    int key[8], c[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      key[u] = j0 + u < k ? key_of<ID>(s.ids, t * k + j0 + u, E) : -1;
      c[u] = 0;
    }
    for (int i = tid; i < n; i += kThreads) {
      const int o = key_of<ID>(s.ids, i, E);
#pragma unroll
      for (int u = 0; u < 8; ++u) c[u] += (o < key[u] || (o == key[u] && i < t * k + j0 + u)) ? 1 : 0;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
#pragma unroll
      for (int d = 32; d; d >>= 1) c[u] += __shfl_xor(c[u], d);
      if (lane == u) found[wave][u] = c[u];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 8; ++u) c[u] = found[0][u] + found[1][u] + found[2][u] + found[3][u];
    if (tid == 0) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (j0 + u < k) {
          s.pos[t * k + j0 + u] = key[u] < E ? c[u] : -1;
          s.order[c[u]] = key[u] < E ? t * k + j0 + u : -1;
        }
    }
    for (int h = tid * 8; h < a.H; h += kThreads * 8) {
      const u32x4 v = load_row<AL>(row, h, a.H);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (j0 + u < k) store_row<AL>(a.xs + (int64_t)c[u] * a.H, h, a.H, key[u] < E ? v : u32x4{0, 0, 0, 0});
    }
    __syncthreads();
  }
}

struct SumArgs {
  const uint16_t* rows; // [n, H] sorted rows
  int64_t ld;
  const float* w; // [T, k] (weighted form)
  const int* pos;
  uint16_t* out; // [T, H]
  int T, k, H, n;
};

// out[t] = sum over kept slots of w[t,j] * rows[pos[t,j]] (w = 1 in the
// unweighted form, the gradient of dispatch): fp32, in the order of j,
// rounded once. KU rows are read at a time; a dropped slot reads row 0 (which
// stays in the caches) and counts as zero whatever its weight or that row
// hold, so that the loads of a group need no branch between them.
template <int DT, int AL, int LANES, int KU, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads) gather_sum_kernel(SumArgs a) {
  const int64_t t = (int64_t)blockIdx.x * (kThreads / LANES) + __builtin_amdgcn_readfirstlane(threadIdx.x / LANES);
  if (t >= a.T) return;
  const int* pos = a.pos + t * a.k;
  const float* wt = WEIGHTED ? a.w + t * a.k : nullptr;
  uint16_t* out = a.out + t * a.H;
  for (int h = (threadIdx.x % LANES) * 8; h < a.H; h += LANES * 8) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < a.k; j0 += KU) {
      u32x4 v[KU];
      float w[KU];
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        const int j = j0 + u < a.k ? j0 + u : a.k - 1;
        const int p = pos[j];
        const bool ok = j0 + u < a.k && (unsigned)p < (unsigned)a.n;
        v[u] = load_row<AL>(a.rows + (ok ? (int64_t)p * a.ld : 0), h, a.H);
        if (!ok) v[u] = u32x4{0, 0, 0, 0};
        if constexpr (WEIGHTED) w[u] = ok ? wt[j] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        float f[8];
        unpack<DT>(v[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = WEIGHTED ? __builtin_fmaf(w[u], f[i], acc[i]) : acc[i] + f[i];
      }
    }
    store_row<AL != 0>(out, h, a.H, pack<DT>(acc));
  }
}

struct BackArgs {
  const uint16_t* dout; // [T, H]
  int64_t lddout;
  const uint16_t* ys; // [n, H]
  int64_t ldys;
  const float* w;
  const int *pos, *offsets;
  const int* order; // null: only the rows behind the last kept one are known to belong to no slot
  uint16_t* dys; // [n, H]
  float* dw;     // [T, k]
  int T, k, E, H, n;
  int token_blocks;
};

// Kept rows whose slot has been taken out of the plan since the sort (its pos names no row): zeros. Each lane looks at a
// row, a wave clears what it finds. The looks are two loads a row beside the H elements that a kept one costs: 8192 tokens
// x 8 level with and without them (rows of 4096 222 us, of 64 12.7), 131072 x 8 rows of 64 190 to 193 us, 600000 x 8 890
// to 936.
template <int AL>
__device__ inline void clear_orphans(const BackArgs& a, int part, int parts) {
  const int lane = threadIdx.x & 63;
  const int kept = min(max(a.offsets[a.E], 0), a.n);
  for (int64_t p0 = (int64_t)part * kThreads + (threadIdx.x & ~63); p0 < kept; p0 += (int64_t)parts * kThreads) {
    const int64_t p = p0 + lane;
    bool orphan = false;
    if (p < kept) {
      const int s = a.order[p];
      orphan = (unsigned)s >= (unsigned)a.n || (unsigned)a.pos[s] >= (unsigned)a.n;
    }
    for (uint64_t m = __ballot(orphan); m; m &= m - 1) {
      uint16_t* row = a.dys + (p0 + __builtin_ctzll(m)) * a.H;
      for (int h = lane * 8; h < a.H; h += 64 * 8) store_row<AL>(row, h, a.H, u32x4{0, 0, 0, 0});
    }
  }
}

// dys[pos[t,j]] = w[t,j] * dout[t] and dw[t,j] = <ys[pos[t,j]], dout[t]>: the
// token's gradient is read once for up to KU slots, each slot's row of ys
// once. The products of a dot are added in fp32 in a fixed order (lane,
// wave, workgroup).
template <int DT, int AL, int LANES, int KU>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(BackArgs a) {
  __shared__ float part[kThreads / 64][KU];
  if ((int)blockIdx.x >= a.token_blocks) {
    clear_tail(a.dys, a.offsets, a.E, a.n, a.H, blockIdx.x - a.token_blocks, gridDim.x - a.token_blocks);
    if (a.order) clear_orphans<AL>(a, blockIdx.x - a.token_blocks, gridDim.x - a.token_blocks);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / LANES) + __builtin_amdgcn_readfirstlane(threadIdx.x / LANES);
  const bool live = t < a.T; // a workgroup of several tokens keeps its barriers to the end
  const int* pos = a.pos + t * a.k;
  const uint16_t* dout = a.dout + t * a.lddout;
  for (int j0 = 0; j0 < a.k; j0 += KU) {
    int p[KU];
    float w[KU], dot[KU];
    bool ok[KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      ok[u] = live && j0 + u < a.k;
      p[u] = ok[u] ? pos[j0 + u] : -1;
      ok[u] = ok[u] && (unsigned)p[u] < (unsigned)a.n;
      w[u] = ok[u] ? a.w[t * a.k + j0 + u] : 0.f;
      dot[u] = 0.f;
    }
    if (live) {
      for (int h = (threadIdx.x % LANES) * 8; h < a.H; h += LANES * 8) {
        u32x4 y[KU];
        const u32x4 g = load_row<AL != 0>(dout, h, a.H);
#pragma unroll
        for (int u = 0; u < KU; ++u) {
          y[u] = load_row<AL>(a.ys + (ok[u] ? (int64_t)p[u] * a.ldys : 0), h, a.H);
          if (!ok[u]) y[u] = u32x4{0, 0, 0, 0};
        }
        float d[8];
        unpack<DT>(g, d);
#pragma unroll
        for (int u = 0; u < KU; ++u) {
          if (!ok[u]) continue;
          float f[8], o[8];
          unpack<DT>(y[u], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[u] = __builtin_fmaf(f[i], d[i], dot[u]);
            o[i] = w[u] * d[i];
          }
          store_row<AL>(a.dys + (int64_t)p[u] * a.H, h, a.H, pack<DT>(o));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < KU; ++u) {
#pragma unroll
      for (int d = 32; d; d >>= 1) dot[u] += __shfl_xor(dot[u], d);
    }
    if constexpr (LANES > 64) {
#pragma unroll
      for (int u = 0; u < KU; ++u)
        if (lane == u) part[wave][u] = dot[u];
      __syncthreads();
#pragma unroll
      for (int u = 0; u < KU; ++u) dot[u] = (part[0][u] + part[1][u]) + (part[2][u] + part[3][u]);
      __syncthreads();
    }
    if (live && threadIdx.x % LANES == 0) {
#pragma unroll
      for (int u = 0; u < KU; ++u)
        if (j0 + u < a.k) a.dw[t * a.k + j0 + u] = ok[u] ? dot[u] : 0.f;
    }
  }
}

} // namespace moe
} // namespace pgemm
