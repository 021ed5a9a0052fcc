// Entry points that sort token rows by expert and bring them back.
#include "context.h"
#include "moe_rows.h"

using namespace pgemm;

namespace {

// Up to this many slots dispatch is one launch (dispatch_small_kernel), above it three.
constexpr int64_t kSmallSlots = 2048;
// Workgroups that clear the rows of dropped slots (they leave at once if there are none).
constexpr int kClearBlocks = 128;

// One wave carries a row of up to 1024 elements (two passes of 16 bytes a lane), four waves a longer one.
int lanes_of(int64_t H) { return H > 1024 ? 256 : 64; }
unsigned token_blocks(int64_t T, int64_t H) {
  const int64_t per = moe::kThreads / lanes_of(H);
  return (unsigned)((T + per - 1) / per);
}

int check_rows(pgemm_ctx* h, int64_t T, int64_t k, int64_t H, int dtype) {
  if (T < 0 || k < 1 || H < 0)
    return fail(h, PGEMM_ERR_INVALID_ARG, "sizes T=%lld k=%lld H=%lld", (long long)T, (long long)k, (long long)H);
  if (T > INT32_MAX || k > INT32_MAX || T * k > (int64_t)1 << 30 || H > (int64_t)1 << 30)
    return fail(h, PGEMM_ERR_UNSUPPORTED, "T * k and H must not exceed 2^30");
  if (dtype != PGEMM_F16 && dtype != PGEMM_BF16)
    return fail(h, PGEMM_ERR_INVALID_ARG, "dtype %d is not fp16 or bf16", dtype);
  if (((int64_t)token_blocks(T, H) + kClearBlocks) * moe::kThreads > UINT32_MAX) // threads of a launch
    return fail(h, PGEMM_ERR_UNSUPPORTED, "T=%lld tokens of H=%lld are more than one launch takes", (long long)T, (long long)H);
  return PGEMM_OK;
}

int check_experts(pgemm_ctx* h, int64_t E) {
  if (E < 1) return fail(h, PGEMM_ERR_INVALID_ARG, "E=%lld experts", (long long)E);
  if (E > moe::kMaxExperts)
    return fail(h, PGEMM_ERR_UNSUPPORTED, "E=%lld experts, at most %d", (long long)E, moe::kMaxExperts);
  return PGEMM_OK;
}

// How the kernels touch the n sorted rows.
int access_of(bool aligned, int64_t n, int64_t H) {
  constexpr int64_t cache = (int64_t)256 << 20; // the memory-side cache
  return !aligned ? moe::kAnyAddress : n * H * 2 > cache && H > 1024 ? moe::kStream : moe::kAligned;
}

bool aligned16(const void* p) { return ((uintptr_t)p % 16) == 0; }

// Slots a workgroup of the sort takes: kTile, or more where that would make too many workgroups.
int64_t sort_chunk(int64_t n) {
  const int64_t tiles = (n + moe::kTile - 1) / moe::kTile;
  return (tiles + moe::kMaxChunks - 1) / moe::kMaxChunks * moe::kTile;
}

template <class ID>
hipError_t launch_dispatch(pgemm_ctx* h, const moe::SortArgs& s, moe::MoveArgs a, int access) {
  const hipStream_t st = h->stream;
  if (s.n <= kSmallSlots) {
    auto kern = access ? moe::dispatch_small_kernel<ID, moe::kAligned> : moe::dispatch_small_kernel<ID, moe::kAnyAddress>;
    return enqueue(st, dim3((unsigned)a.T + 1), dim3(moe::kThreads), kern, s, a);
  }
  const int chunks = (int)((s.n + s.chunk - 1) / s.chunk);
  hipError_t e = enqueue(st, dim3(chunks), dim3(moe::kThreads), moe::sort_count_kernel<ID>, s);
  if (e == hipSuccess) e = enqueue(st, dim3(chunks), dim3(moe::kThreads), moe::sort_place_kernel<ID>, s, chunks);
  if (e != hipSuccess || a.H == 0) return e;
  a.token_blocks = (int)token_blocks(a.T, a.H);
  const dim3 grid((unsigned)a.token_blocks + kClearBlocks);
  const bool wide = lanes_of(a.H) == 256;
  auto kern = access == moe::kStream    ? moe::move_kernel<moe::kStream, 256>
              : access == moe::kAligned ? (wide ? moe::move_kernel<moe::kAligned, 256> : moe::move_kernel<moe::kAligned, 64>)
                                        : (wide ? moe::move_kernel<moe::kAnyAddress, 256> : moe::move_kernel<moe::kAnyAddress, 64>);
  return enqueue(st, grid, dim3(moe::kThreads), kern, a);
}

template <int DT, int AL, int LANES, bool WEIGHTED>
hipError_t launch_sum_k(pgemm_ctx* h, const moe::SumArgs& a, unsigned grid) {
  auto kern = a.k >= 8   ? moe::gather_sum_kernel<DT, AL, LANES, 8, WEIGHTED>
              : a.k >= 3 ? moe::gather_sum_kernel<DT, AL, LANES, 4, WEIGHTED>
                         : moe::gather_sum_kernel<DT, AL, LANES, 2, WEIGHTED>;
  return enqueue(h->stream, dim3(grid), dim3(moe::kThreads), kern, a);
}

template <int DT, bool WEIGHTED>
hipError_t launch_sum(pgemm_ctx* h, const moe::SumArgs& a, int access) {
  const unsigned grid = token_blocks(a.T, a.H);
  const bool wide = lanes_of(a.H) == 256;
  if (access == moe::kStream) return launch_sum_k<DT, moe::kStream, 256, WEIGHTED>(h, a, grid);
  if (access == moe::kAligned)
    return wide ? launch_sum_k<DT, moe::kAligned, 256, WEIGHTED>(h, a, grid) : launch_sum_k<DT, moe::kAligned, 64, WEIGHTED>(h, a, grid);
  return wide ? launch_sum_k<DT, moe::kAnyAddress, 256, WEIGHTED>(h, a, grid)
              : launch_sum_k<DT, moe::kAnyAddress, 64, WEIGHTED>(h, a, grid);
}

template <int DT, int AL, int LANES>
hipError_t launch_back_k(pgemm_ctx* h, const moe::BackArgs& a, unsigned grid) {
  auto kern = a.k >= 8   ? moe::combine_backward_kernel<DT, AL, LANES, 8>
              : a.k >= 3 ? moe::combine_backward_kernel<DT, AL, LANES, 4>
                         : moe::combine_backward_kernel<DT, AL, LANES, 2>;
  return enqueue(h->stream, dim3(grid), dim3(moe::kThreads), kern, a);
}

template <int DT>
hipError_t launch_back(pgemm_ctx* h, const moe::BackArgs& a, int access) {
  // with the plan's order every sorted row is looked at: more workgroups for many rows, as far as a launch has room
  const unsigned room = UINT32_MAX / moe::kThreads - (unsigned)a.token_blocks;
  const unsigned looks = a.order ? (unsigned)a.n / 1024 : 0, clear = looks < kClearBlocks ? kClearBlocks : looks < 2048 ? looks : 2048;
  const unsigned grid = (unsigned)a.token_blocks + (clear < room ? clear : room);
  const bool wide = lanes_of(a.H) == 256;
  if (access == moe::kStream) return launch_back_k<DT, moe::kStream, 256>(h, a, grid);
  if (access == moe::kAligned)
    return wide ? launch_back_k<DT, moe::kAligned, 256>(h, a, grid) : launch_back_k<DT, moe::kAligned, 64>(h, a, grid);
  return wide ? launch_back_k<DT, moe::kAnyAddress, 256>(h, a, grid) : launch_back_k<DT, moe::kAnyAddress, 64>(h, a, grid);
}

int sum_impl(pgemm_handle_t h, const void* rows, int64_t ld, const float* w, const int32_t* pos, int64_t T, int64_t k,
             int64_t H, int dtype, void* out, bool weighted) {
  if (!h) return PGEMM_ERR_INVALID_ARG;
  h->last_error[0] = 0;
  const int rc = check_rows(h, T, k, H, dtype);
  if (rc != PGEMM_OK) return rc;
  if (T == 0 || H == 0) return PGEMM_OK;
  if (!rows || !pos || !out || (weighted && !w)) return fail(h, PGEMM_ERR_INVALID_ARG, "a pointer is NULL");
  if (ld < 0) return fail(h, PGEMM_ERR_INVALID_ARG, "row stride %lld", (long long)ld);
  DeviceScope dev(h->device);
  if (!dev.ok()) return fail(h, PGEMM_ERR_HIP, "hipSetDevice failed");
  moe::SumArgs a;
  a.rows = static_cast<const uint16_t*>(rows);
  a.ld = ld;
  a.w = w;
  a.pos = pos;
  a.out = static_cast<uint16_t*>(out);
  a.T = (int)T;
  a.k = (int)k;
  a.H = (int)H;
  a.n = (int)(T * k);
  const bool al = H % 8 == 0 && ld % 8 == 0 && aligned16(rows) && aligned16(out);
  const int access = access_of(al, T * k, H);
  const bool bf16 = dtype == PGEMM_BF16;
  if (weighted)
    return launch_status(h, bf16 ? launch_sum<kBF16, true>(h, a, access) : launch_sum<kF16, true>(h, a, access), "combine");
  return launch_status(h, bf16 ? launch_sum<kBF16, false>(h, a, access) : launch_sum<kF16, false>(h, a, access),
                       "dispatch backward");
}

int back_impl(pgemm_handle_t h, const void* dout, int64_t lddout, const void* ys, int64_t ldys, const float* w,
              const int32_t* offsets, const int32_t* order, const int32_t* pos, int64_t T, int64_t k, int64_t E, int64_t H,
              int dtype, void* dys, float* dw) {
  if (!h) return PGEMM_ERR_INVALID_ARG;
  h->last_error[0] = 0;
  int rc = check_rows(h, T, k, H, dtype);
  if (rc == PGEMM_OK) rc = check_experts(h, E);
  if (rc != PGEMM_OK) return rc;
  if (T == 0) return PGEMM_OK;
  if (!w || !offsets || !pos || !dw || (H > 0 && (!dout || !ys || !dys)))
    return fail(h, PGEMM_ERR_INVALID_ARG, "a pointer is NULL");
  if (lddout < 0 || ldys < 0)
    return fail(h, PGEMM_ERR_INVALID_ARG, "row strides %lld, %lld", (long long)lddout, (long long)ldys);
  DeviceScope dev(h->device);
  if (!dev.ok()) return fail(h, PGEMM_ERR_HIP, "hipSetDevice failed");
  moe::BackArgs a;
  a.dout = static_cast<const uint16_t*>(dout);
  a.lddout = lddout;
  a.ys = static_cast<const uint16_t*>(ys);
  a.ldys = ldys;
  a.w = w;
  a.pos = pos;
  a.offsets = offsets;
  a.order = order;
  a.dys = static_cast<uint16_t*>(dys);
  a.dw = dw;
  a.T = (int)T;
  a.k = (int)k;
  a.E = (int)E;
  a.H = (int)H;
  a.n = (int)(T * k);
  a.token_blocks = (int)token_blocks(T, H);
  const bool al = H % 8 == 0 && lddout % 8 == 0 && ldys % 8 == 0 && aligned16(dout) && aligned16(ys) && aligned16(dys);
  const int access = access_of(al, T * k, H);
  return launch_status(h, dtype == PGEMM_BF16 ? launch_back<kBF16>(h, a, access) : launch_back<kF16>(h, a, access),
                       "combine backward");
}

} // namespace

extern "C" {

int pgemm_moe_dispatch_workspace(int64_t T, int64_t k, int64_t E, int64_t* bytes) {
  if (!bytes || T < 0 || k < 1 || E < 1) return PGEMM_ERR_INVALID_ARG;
  *bytes = 0;
  if (T > INT32_MAX || k > INT32_MAX || T * k > (int64_t)1 << 30 || E > moe::kMaxExperts) return PGEMM_ERR_UNSUPPORTED;
  const int64_t n = T * k;
  if (n > kSmallSlots) {
    const int64_t chunk = sort_chunk(n);
    *bytes = (n + chunk - 1) / chunk * (E + 1) * (int64_t)sizeof(int);
  }
  return PGEMM_OK;
}

int pgemm_moe_dispatch(pgemm_handle_t h, const void* x, int64_t ldx, const void* ids, int ids_type, int64_t T, int64_t k,
                       int64_t E, int64_t H, int dtype, int32_t* offsets, int32_t* order, int32_t* pos, void* xs,
                       void* work, int64_t work_bytes) {
  if (!h) return PGEMM_ERR_INVALID_ARG;
  h->last_error[0] = 0;
  int rc = check_rows(h, T, k, H, dtype);
  if (rc == PGEMM_OK) rc = check_experts(h, E);
  if (rc != PGEMM_OK) return rc;
  if (ids_type != PGEMM_IDS_I32 && ids_type != PGEMM_IDS_I64)
    return fail(h, PGEMM_ERR_INVALID_ARG, "unknown ids type %d", ids_type);
  if (ldx < 0) return fail(h, PGEMM_ERR_INVALID_ARG, "row stride %lld", (long long)ldx);
  if (!offsets || (T > 0 && (!ids || !order || !pos || (H > 0 && (!x || !xs)))))
    return fail(h, PGEMM_ERR_INVALID_ARG, "a pointer is NULL");
  int64_t need = 0;
  rc = pgemm_moe_dispatch_workspace(T, k, E, &need);
  if (rc != PGEMM_OK) return rc;
  if (work_bytes < need || (need && !work))
    return fail(h, PGEMM_ERR_INVALID_ARG, "workspace of %lld bytes, %lld are needed", (long long)work_bytes,
                (long long)need);
  DeviceScope dev(h->device);
  if (!dev.ok()) return fail(h, PGEMM_ERR_HIP, "hipSetDevice failed");
  moe::SortArgs s;
  s.ids = ids;
  s.n = (int)(T * k);
  s.E = (int)E;
  s.chunk = (int)sort_chunk(T * k);
  s.counts = static_cast<int*>(work);
  s.offsets = offsets;
  s.order = order;
  s.pos = pos;
  moe::MoveArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.xs = static_cast<uint16_t*>(xs);
  a.pos = pos;
  a.offsets = offsets;
  a.T = (int)T;
  a.k = (int)k;
  a.E = (int)E;
  a.H = (int)H;
  a.n = s.n;
  a.token_blocks = 0;
  const bool al = H % 8 == 0 && ldx % 8 == 0 && aligned16(x) && aligned16(xs);
  const int access = access_of(al, T * k, H);
  const bool i32 = ids_type == PGEMM_IDS_I32;
  return launch_status(h, i32 ? launch_dispatch<int32_t>(h, s, a, access) : launch_dispatch<int64_t>(h, s, a, access), "dispatch");
}

int pgemm_moe_dispatch_backward(pgemm_handle_t h, const void* dxs, int64_t lddxs, const int32_t* pos, int64_t T,
                                int64_t k, int64_t H, int dtype, void* dx) {
  return sum_impl(h, dxs, lddxs, nullptr, pos, T, k, H, dtype, dx, false);
}

int pgemm_moe_combine(pgemm_handle_t h, const void* ys, int64_t ldys, const float* w, const int32_t* pos, int64_t T,
                      int64_t k, int64_t H, int dtype, void* out) {
  return sum_impl(h, ys, ldys, w, pos, T, k, H, dtype, out, true);
}

int pgemm_moe_combine_backward(pgemm_handle_t h, const void* dout, int64_t lddout, const void* ys, int64_t ldys,
                               const float* w, const int32_t* offsets, const int32_t* pos, int64_t T, int64_t k,
                               int64_t E, int64_t H, int dtype, void* dys, float* dw) {
  return back_impl(h, dout, lddout, ys, ldys, w, offsets, nullptr, pos, T, k, E, H, dtype, dys, dw);
}

int pgemm_moe_combine_backward_plan(pgemm_handle_t h, const void* dout, int64_t lddout, const void* ys, int64_t ldys,
                                    const float* w, const int32_t* offsets, const int32_t* order, const int32_t* pos,
                                    int64_t T, int64_t k, int64_t E, int64_t H, int dtype, void* dys, float* dw) {
  if (h && T > 0 && !order) return fail(h, PGEMM_ERR_INVALID_ARG, "order is NULL");
  return back_impl(h, dout, lddout, ys, ldys, w, offsets, order, pos, T, k, E, H, dtype, dys, dw);
}

} // extern "C"
