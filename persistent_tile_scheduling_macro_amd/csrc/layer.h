// A whole routed layer for the few tokens of a decoding batch, in two launches:
//   h[s] = act(x[t] W_in[e]^T)            gated: act(gate) * up of its 2I columns
//   out[t] = sum over t's slots s of weights[s] * (h[s] W_out[e]^T)
// with e = ids[s]. Reading the matrices of the experts that some token takes
// bounds it; each is read once for every group of tokens that take it.
//
// A group is up to 16 * MB of the tokens that take one expert. MB (1, 2 or 4) is
// chosen by their mean number so that nearly every expert is one group; another
// group reads the matrices again, four times in all at most. A token that names
// an expert twice is one row with the sum of its weights.
//
// up_kernel: one workgroup for a group and 16 columns of h. It counts the tokens
// of every expert from the ids and finds its group by a scan, so no sort and no
// launch goes before it; the scheme of the product is that of dense_few.h. The
// workgroups of the first columns also write the plan that the second launch
// reads: for each group its expert, slots and weights.
//
// down_kernel: one workgroup for 16 columns of out and a share of all groups'
// work (the whole of it where H / 16 workgroups fill the card). The groups'
// sums of I are laid end to end, in steps of 64, and cut evenly between
// workgroups and their waves, which read ahead across groups. At a group's end a
// wave adds its sums, times the rows' weights, in fp32 to its own [T][16] part of
// LDS; the waves' parts are added in order, and where several workgroups share
// the columns, the last one to come adds all their parts in order. So no sum
// depends on the order of atomics (but the ids of all tokens fix where the
// groups' sums are cut: a token's last bits may depend on the others' ids), no
// row of any expert's output goes through memory, and h is the only intermediate
// value that is rounded (to 16 bits: it is an MFMA operand; bf16 outputs are off
// by 0.0023 instead of one rounding's 0.0017).
//
// 32 tokens, 4 of 32 experts, 4096 x 2048 gated bf16: 182 and 122 us, 6.0 and 4.4
// TB/s; one token, 8 of 64, 2048 x 1024 gated: 20 and 10 us, of each 3.9 the
// launch.
#pragma once

#include "dense.h"
#include "grouped_few.h"

namespace pgemm {
namespace layer {

using grouped::load_upto;
using grouped::turn_at;
using moe::u32x4;

constexpr int kTokens = 64; // of one pass
constexpr int kMaxSlots = 2048;

struct Args {
  const uint16_t* x; // rows ldx apart
  int64_t ldx;
  const void* ids;   // [T, k] contiguous, 32 or 64 bits
  int ids64;
  const float* weights;  // [T, k]
  const uint16_t* w_in;  // [E][I or 2I][H]
  const uint16_t* w_out; // [E][H][I]
  uint16_t* h;           // [T * k][I]
  int* groups;           // number of groups, then {expert | rows << 16} of each
  int* slots;            // [group][kTokens]
  float* shares;         // [group][kTokens]
  int* arrived;          // [ceil(H / 16)] workgroups that have written their part
  float* parts;          // [ceil(H / 16)][sharers][T][16]
  uint16_t* out;         // [T, H]
  int T, k, E, H, I, act;
  int most;    // groups there can be
  int sharers; // workgroups that share 16 columns of out
};

__device__ inline void wave_fence() { // LDS serves a wave in order: only the compiler has to be held
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// LOOP: several turns of 16 columns a workgroup, for short rows, where finding the group (some 3 us) is most of a turn's
// work (21 experts, 286 x 4056: 86 us, looped 66; 128 experts, 1024 x 512 gated: 45 and 41). With long rows other workgroups' turns overlap it, and
// turns one after another do not (32 experts, 4096 x 2048 gated: 288 us and 326).
template <int DT, bool GATED, int MB, bool LOOP>
__global__ void __launch_bounds__(512, MB == 4 || (LOOP && MB == 2) ? 2 : 4) up_kernel(Args a) {
  constexpr int WAVES = 8, BLK = GATED ? 2 : 1, D = MB > 1 ? 2 : GATED ? 3 : 4, XL = 2 * MB;
  constexpr int TURN = 2048 * (MB + BLK), JOIN = BLK * MB * 1024;
  typedef typename fast::Frag<DT>::t frag_t;
  typedef typename Traits<DT>::out_t out_t;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[WAVES * (TURN > JOIN ? TURN : JOIN)];
  __shared__ short s_ids[kMaxSlots];
  __shared__ int s_count[moe::kMaxExperts];
  __shared__ int s_row[16 * MB];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = a.T * a.k, H = a.H, I = a.I;
  const bool writes = blockIdx.x == 0;

  // ---- the tokens of every expert, and this workgroup's group
  for (int i = tid; i < a.E; i += WAVES * 64) s_count[i] = 0;
  if (writes && blockIdx.y == 0)
    for (int i = tid; i < (H + 15) / 16; i += WAVES * 64) a.arrived[i] = 0;
  for (int i = tid; i < n; i += WAVES * 64)
    s_ids[i] = (short)(a.ids64 ? moe::key_of<int64_t>(a.ids, i, a.E) : moe::key_of<int32_t>(a.ids, i, a.E));
  __syncthreads();
  for (int i = tid; i < n; i += WAVES * 64) {
    const int e = s_ids[i], t = i / a.k;
    bool first = e < a.E; // of its token's choices
    for (int j = t * a.k; j < i; ++j) first &= s_ids[j] != e;
    if (first) atomicAdd(&s_count[e], 1);
  }
  __syncthreads();
  const int per = (a.E + 63) / 64; // experts a lane counts
  int mine_groups = 0;
  for (int i = 0; i < per; ++i)
    if (per * lane + i < a.E) mine_groups += (s_count[per * lane + i] + 16 * MB - 1) / (16 * MB);
  int upto = mine_groups;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  const int which = blockIdx.y, groups = __builtin_amdgcn_readfirstlane(__shfl(upto, 63));
  if (writes && which == 0 && tid == 0) a.groups[0] = groups;
  if (which >= groups) return;
  const int owner = (int)__builtin_ctzll(__ballot(upto > which));
  int left = which - __builtin_amdgcn_readfirstlane(__shfl(upto - mine_groups, owner)); // groups before it in owner's experts
  int e = per * owner;
  for (;; ++e) {
    const int c = (s_count[e] + 16 * MB - 1) / (16 * MB);
    if (left < c) break;
    left -= c;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  const int first_row = __builtin_amdgcn_readfirstlane(left) * 16 * MB;

  // every wave finds the rows for itself: lane t looks through its token's choices, and the tokens that
  // have one move to the front
  const int row = lane >> 3, chunk = lane & 7;
  int slot = -1;
  float share = 0.0f;
  if (lane < a.T) {
    for (int j = a.k - 1; j >= 0; --j)
      if (s_ids[lane * a.k + j] == e) slot = lane * a.k + j;
    if (writes && wave == 0)
      for (int j = 0; j < a.k; ++j)
        if (s_ids[lane * a.k + j] == e) share += a.weights[lane * a.k + j];
  }
  const uint64_t taken = __ballot(slot >= 0), below = (1ull << lane) - 1;
  const int all_rows = (int)__popcll(taken), rows = min(all_rows - first_row, 16 * MB);
  const int rank = slot >= 0 ? (int)__popcll(taken & below) : all_rows + (int)__popcll(~taken & below);
  const int slot_at = __builtin_amdgcn_ds_permute(4 * rank, slot); // lane r: the slot of the expert's row r
  if (wave == 0 && slot >= 0 && rank >= first_row && rank < first_row + rows) {
    s_row[rank - first_row] = slot; // read after the next barrier
    if (writes) {
      a.slots[which * kTokens + rank - first_row] = slot;
      a.shares[which * kTokens + rank - first_row] = share;
    }
  }
  if (writes && tid == 0) a.groups[1 + which] = e | rows << 16;

  // ---- the product
  const int x_loads = __builtin_amdgcn_readfirstlane((rows + 7) >> 3), blocks = (x_loads + 1) >> 1;
  const uint16_t* x_kept[XL];
#pragma unroll
  for (int i = 0; i < XL; ++i) x_kept[i] = a.x + __shfl(slot_at, first_row + min(8 * i + row, rows - 1)) / a.k * a.ldx + 8 * chunk;
  const act::Consts k = act::consts_of(a.act);
  int n0 = blockIdx.x * 16;
  do {
    // opaque, or the turn's addresses would all be kept in registers from turn to turn, and spilled
    int lane_v = tid & 63;
    asm volatile("" : "+v"(lane_v));
    const int row = lane_v >> 3, chunk = lane_v & 7, g = lane_v >> 4, s = lane_v & 15;
    const uint16_t* x[XL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      x[i] = x_kept[i];
      asm volatile("" : "+v"(x[i]));
    }
    const uint16_t* w[BLK * 2];
#pragma unroll
    for (int i = 0; i < BLK * 2; ++i)
      w[i] = a.w_in + ((int64_t)e * I * BLK + (i >= 2 ? I : 0) + min(n0 + 8 * (i & 1) + row, I - 1)) * H + 8 * chunk;
    struct Slot { u32x4 x[XL], w[BLK * 2]; };
    auto load = [&](Slot& t, int step) __attribute__((always_inline)) {
      const int64_t k0 = (int64_t)step * 64;
#pragma unroll
      for (int i = 0; i < BLK * 2; ++i) t.w[i] = moe::load8<moe::kAnyAddress>(w[i] + k0);
#pragma unroll
      for (int i = 0; i < XL; ++i)
        if (i == 0 || i < x_loads) t.x[i] = moe::load8<moe::kAnyAddress>(x[i] + k0);
    };
    floatx4_t acc[MB][BLK];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < BLK; ++c) acc[b][c] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    uint8_t *turn_x = lds + wave * TURN, *turn_w = turn_x + 2048 * MB;
    auto multiply = [&](const Slot& t) __attribute__((always_inline)) {
      wave_fence(); // the last step's reads come first
#pragma unroll
      for (int i = 0; i < XL; ++i)
        if (i < x_loads) *reinterpret_cast<u32x4*>(turn_x + turn_at<128>(8 * i + row, chunk)) = t.x[i];
#pragma unroll
      for (int i = 0; i < BLK * 2; ++i) *reinterpret_cast<u32x4*>(turn_w + turn_at<128>(8 * i + row, chunk)) = t.w[i];
      wave_fence();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        frag_t f[BLK];
#pragma unroll
        for (int c = 0; c < BLK; ++c) f[c] = *reinterpret_cast<const frag_t*>(turn_w + turn_at<128>(16 * c + s, 4 * h + g));
#pragma unroll
        for (int b = 0; b < MB; ++b)
          if (b < blocks) {
            // an odd number of loads leaves the block's upper half to repeat its lower one
            const int r = 16 * b + (2 * b + 1 < x_loads ? s : s & 7);
            const frag_t xf = *reinterpret_cast<const frag_t*>(turn_x + turn_at<128>(r, 4 * h + g));
#pragma unroll
            for (int c = 0; c < BLK; ++c) acc[b][c] = mfma(f[c], xf, acc[b][c]);
          }
      }
    };
    const int whole = H / 64, mine = (whole - wave + WAVES - 1) / WAVES;
    dense::stream_steps<D, Slot>(
        mine, [&](Slot& t, int i) __attribute__((always_inline)) { load(t, wave + WAVES * i); }, multiply);
    if (whole * 64 < H && wave == whole % WAVES) { // the partial step, zeros past H
      const int k0 = whole * 64;
      Slot t;
#pragma unroll
      for (int i = 0; i < BLK * 2; ++i) t.w[i] = load_upto(w[i] + k0, H - k0 - 8 * chunk, H);
#pragma unroll
      for (int i = 0; i < XL; ++i)
        if (i < x_loads) t.x[i] = load_upto(x[i] + k0, H - k0 - 8 * chunk, H);
      multiply(t);
    }

    __syncthreads(); // every wave is through with its part of the LDS
    floatx4_t* join = reinterpret_cast<floatx4_t*>(lds);
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < BLK; ++c) join[(wave * BLK * MB + c * MB + b) * 64 + lane] = acc[b][c];
    __syncthreads();
    const int b = tid >> 6, m = 16 * b + s;
    if (b < MB && m < rows) {
      floatx4_t v = join[tid], u = floatx4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int o = 1; o < WAVES; ++o) v += join[o * BLK * MB * 64 + tid];
      if constexpr (GATED) {
        u = join[MB * 64 + tid];
#pragma unroll
        for (int o = 1; o < WAVES; ++o) u += join[o * BLK * MB * 64 + MB * 64 + tid];
      }
      uint16_t* to = a.h + (int64_t)s_row[m] * I;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int c = n0 + 4 * g + r;
        if (c >= I) continue;
        float y = v[r];
        act::with_path(k, [&](auto path) __attribute__((always_inline)) { y = act::value<decltype(path)::value>(y, k); });
        if constexpr (GATED) y *= u[r];
        to[c] = __builtin_bit_cast(uint16_t, to_out(y, (out_t*)nullptr));
      }
    }
    if constexpr (LOOP) __syncthreads(); // the next turn writes the LDS that this one read
    n0 += gridDim.x * 16;
  } while (LOOP && n0 < I);
}

// Waves of a workgroup of down_kernel, as many as LDS holds: there are few workgroups (16 columns of 2048 rows and eight
// experts of I = 1024: 17 us with eight waves, 12.5 us with 16).
constexpr int down_waves(int blocks) { return blocks == 1 ? 16 : 8; }

// The last step's chunks past a row's end are read as the row's last eight elements and put right on the way to LDS, and
// the first eight rows of h are always read: of the loads on all paths the compiler counts the fewest, and with a path
// that has none it would wait for every load in flight. SHORT: I < 8.
template <int DT, int MB, bool SHORT>
__global__ void __launch_bounds__(64 * down_waves(MB), MB == 4 ? 2 : 4) down_kernel(Args a) {
  constexpr int WAVES = down_waves(MB), D = MB == 1 ? 4 : 2, XL = 2 * MB, RING = MB == 1 ? 8 : 4, R = 16 * MB;
  static_assert(D < RING, "a ring entry lasts from a group's first load to its last product");
  constexpr int TURN = 2048 * (MB + 1);
  typedef typename fast::Frag<DT>::t frag_t;
  typedef typename Traits<DT>::out_t out_t;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[WAVES * TURN];
  __shared__ floatx4_t s_out[WAVES][kTokens * 4]; // [token][16 columns]
  __shared__ int s_token[WAVES][RING][R];         // of a group's rows
  __shared__ float s_share[WAVES][RING][R];
  __shared__ int s_last;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, s = lane & 15, row = lane >> 3, chunk = lane & 7;
  const int tile = blockIdx.x, n0 = tile * 16, H = a.H, I = a.I;
  const int infos = a.groups[min(lane, a.most)]; // lane 0: how many; then the first groups
  for (int i = lane; i < a.T * 4; i += 64) s_out[wave][i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  const int groups = __builtin_amdgcn_readfirstlane(infos);
  const int steps = (I + 63) / 64, runs = WAVES * a.sharers, run = blockIdx.y * WAVES + wave;
  const int64_t units = (int64_t)groups * steps;
  const int64_t from = units * run / runs, to = units * (run + 1) / runs;
  const int mine = (int)(to - from);

  // ---- the load cursor: group, step, the slots and shares of its rows in the lanes (fetched a group ahead)
  int l_at = (int)(from / steps), l_step = (int)(from - (int64_t)l_at * steps), l_loads = 0;
  bool fresh = true; // group l_at has not been entered
  int next_slot = 0;
  float next_share = 0.0f;
  auto fetch = [&](int at) __attribute__((always_inline)) { // lanes past the rows read what nobody uses
    const int i = min(at, groups - 1) * kTokens + lane;
    next_slot = a.slots[i];
    next_share = a.shares[i];
  };
  const uint16_t* w[2];
  int x[XL], l_rows = 0; // element offsets in h
  struct Slot { u32x4 x[XL], w[2]; int loads, rest; };
  int left = mine;
  auto load = [&](Slot& t) __attribute__((always_inline)) {
    if (left <= 0) return;
    --left;
    if (fresh) {
      const int info = __builtin_amdgcn_readfirstlane(l_at < 63 ? __shfl(infos, l_at + 1) : a.groups[1 + l_at]);
      l_rows = info >> 16;
      l_loads = (l_rows + 7) >> 3;
#pragma unroll
      for (int i = 0; i < 2; ++i) w[i] = a.w_out + ((int64_t)(info & 0xFFFF) * H + min(n0 + 8 * i + row, H - 1)) * I + 8 * chunk;
    }
    const int at = min(l_step * 64, I - 8 - 8 * chunk); // from the lane's own chunk of the row's start
    t.rest = I - l_step * 64;
    auto chunk_of = [&](const uint16_t* p) __attribute__((always_inline)) {
      if constexpr (SHORT) return load_upto(p, I - 8 * chunk, I);
      else return moe::load8<moe::kAnyAddress>(p + at);
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) t.w[i] = chunk_of(w[i]);
    if (fresh) { // the slots come in while the matrix is read
      const int slot = next_slot;
      const float share = next_share;
      if (lane < R) {
        s_token[wave][l_at % RING][lane] = lane < l_rows ? slot / a.k : -1;
        s_share[wave][l_at % RING][lane] = share;
      }
#pragma unroll
      for (int i = 0; i < XL; ++i) x[i] = __shfl(slot, min(8 * i + row, l_rows - 1)) * I + 8 * chunk;
      fetch(l_at + 1);
      fresh = false;
    }
    t.loads = l_loads;
#pragma unroll
    for (int i = 0; i < XL; ++i)
      if (i == 0 || i < l_loads) t.x[i] = chunk_of(a.h + x[i]);
    if (++l_step == steps) {
      l_step = 0;
      ++l_at;
      fresh = true;
    }
  };

  // ---- the compute cursor
  int c_at = l_at, c_step = l_step;
  floatx4_t acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  auto flush = [&]() __attribute__((always_inline)) { // group c_at's sums to their tokens
    wave_fence();
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      const int token = s_token[wave][c_at % RING][16 * b + s];
      const float share = s_share[wave][c_at % RING][16 * b + s];
      if (token >= 0) {
        floatx4_t* o = &s_out[wave][token * 4 + g];
        floatx4_t v = *o;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(share, acc[b][r], v[r]);
        *o = v;
      }
      acc[b] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    }
  };
  uint8_t *turn_x = lds + wave * TURN, *turn_w = turn_x + 2048 * MB;
  auto multiply = [&](Slot& t) __attribute__((always_inline)) {
    if (!SHORT && t.rest < 64) { // the row's end
      const int own = t.rest - 8 * chunk;
      auto cut = [&](u32x4 v) __attribute__((always_inline)) {
        return own >= 8 ? v : own <= 0 ? u32x4{0, 0, 0, 0} : moe::shift_down(v, 8 - own);
      };
#pragma unroll
      for (int i = 0; i < 2; ++i) t.w[i] = cut(t.w[i]);
#pragma unroll
      for (int i = 0; i < XL; ++i)
        if (i < t.loads) t.x[i] = cut(t.x[i]);
    }
    wave_fence(); // the last step's reads come first
#pragma unroll
    for (int i = 0; i < XL; ++i)
      if (i < t.loads) *reinterpret_cast<u32x4*>(turn_x + turn_at<128>(8 * i + row, chunk)) = t.x[i];
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4*>(turn_w + turn_at<128>(8 * i + row, chunk)) = t.w[i];
    wave_fence();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const frag_t f = *reinterpret_cast<const frag_t*>(turn_w + turn_at<128>(s, 4 * h + g));
#pragma unroll
      for (int b = 0; b < MB; ++b)
        if (2 * b < t.loads) {
          // an odd number of loads leaves the block's upper half to repeat its lower one
          const int r = 16 * b + (2 * b + 1 < t.loads ? s : s & 7);
          acc[b] = mfma(f, *reinterpret_cast<const frag_t*>(turn_x + turn_at<128>(r, 4 * h + g)), acc[b]);
        }
    }
    if (++c_step == steps) {
      flush();
      c_step = 0;
      ++c_at;
    }
  };
  if (mine > 0) {
    fetch(l_at);
    Slot t[D];
#pragma unroll
    for (int j = 0; j < D; ++j) load(t[j]);
    for (int i = 0; i < mine; i += D) {
#pragma unroll
      for (int j = 0; j < D; ++j)
        if (i + j < mine) {
          multiply(t[j]);
          load(t[j]);
        }
    }
    if (c_step) flush(); // the next wave has the rest of this group's sum
  }
  __syncthreads();
  const float* waves = reinterpret_cast<const float*>(s_out);
  auto store = [&](int i, float v) __attribute__((always_inline)) {
    const int c = n0 + i % 16;
    if (c < H) a.out[(int64_t)(i / 16) * H + c] = __builtin_bit_cast(uint16_t, to_out(v, (out_t*)nullptr));
  };
  // Parts pass through agent-scope accesses, which go past the XCD's own L2: waiting for them (the barrier does) makes them
  // visible before the arrival is counted. (Plain stores and a fence, which writes back the whole L2, cost 80 us.)
  float* part = a.parts + (int64_t)tile * a.sharers * a.T * 16;
  for (int i = tid; i < a.T * 16; i += WAVES * 64) {
    float v = waves[i];
#pragma unroll
    for (int o = 1; o < WAVES; ++o) v += waves[o * kTokens * 16 + i];
    if (a.sharers == 1) store(i, v);
    else __hip_atomic_store(part + blockIdx.y * a.T * 16 + i, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (a.sharers == 1) return;
  __builtin_amdgcn_s_waitcnt(0); // every counter
  __syncthreads();
  if (tid == 0) s_last = __hip_atomic_fetch_add(a.arrived + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.sharers - 1;
  __syncthreads();
  if (!s_last) return;
  for (int i = tid; i < a.T * 16; i += WAVES * 64) {
    float v = 0.0f;
    for (int z = 0; z < a.sharers; ++z) v += __hip_atomic_load(part + z * a.T * 16 + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    store(i, v);
  }
}

typedef void (*kernel_fn)(Args);
kernel_fn up_f16(bool gated, int blocks, bool loop);
kernel_fn up_bf16(bool gated, int blocks, bool loop);
kernel_fn down_f16(int blocks, bool is_short);
kernel_fn down_bf16(int blocks, bool is_short);

template <int DT, bool GATED, bool LOOP>
kernel_fn pick_up_blocks(int blocks) {
  return blocks == 1 ? up_kernel<DT, GATED, 1, LOOP> : blocks == 2 ? up_kernel<DT, GATED, 2, LOOP> : up_kernel<DT, GATED, 4, LOOP>;
}
template <int DT>
kernel_fn pick_up(bool gated, int blocks, bool loop) {
  if (loop) return gated ? pick_up_blocks<DT, true, true>(blocks) : pick_up_blocks<DT, false, true>(blocks);
  return gated ? pick_up_blocks<DT, true, false>(blocks) : pick_up_blocks<DT, false, false>(blocks);
}
template <int DT>
kernel_fn pick_down(int blocks, bool is_short) {
  if (is_short) return blocks == 1 ? down_kernel<DT, 1, true> : blocks == 2 ? down_kernel<DT, 2, true> : down_kernel<DT, 4, true>;
  return blocks == 1 ? down_kernel<DT, 1, false> : blocks == 2 ? down_kernel<DT, 2, false> : down_kernel<DT, 4, false>;
}

} // namespace layer
} // namespace pgemm
