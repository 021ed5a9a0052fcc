// The handle behind pgemm_handle_t and its error detail, shared by the
// translation units that implement the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstdarg>
#include <cstdio>

#include "../../include/pgemm.h"
#include "kernels.h"
#include "launch.h"

struct pgemm_ctx {
  int device = 0;
  hipStream_t stream = nullptr;
  int cus = 0;
  int* counter = nullptr; // work counter of the claiming modes (device int32)
  int32_t* visits = nullptr;
  int64_t n_visits = 0;
  int32_t* owner = nullptr;
  int64_t n_owner = 0;
  int64_t* trace = nullptr;
  int64_t n_trace = 0;
  int b_nk = 0; // layout of B: 0 = K x N row-major, 1 = N x K row-major
  float scale_a = 1.0f, scale_b = 1.0f; // per-tensor scales of e4m3 A and B
  // Tile-order defaults measured on MI355X (8192^3 and 4096^3 fp16, round-robin
  // timing): GROUP_SIZE_M between 1 and 16 moved throughput by a few percent
  // at most. The XCD remap (-1 = automatic: on when a launch has more tiles
  // than CUs) leaves the time level at 8192^3 and cuts the L2-miss fetches
  // there by a third (each XCD reads fewer operand panels); with one wave of
  // tiles it fetches the same bytes and measured slightly slower, so it stays
  // off there.
  int group_m = 4;
  int xcd_remap = -1;
  int tile = PGEMM_TILE_AUTO; // macro-tile choice of the fast kernel
  int mainloop = PGEMM_MAINLOOP_AUTO; // lockstep, ping-pong or producer waves for the 256-row tile
  // Stream-K: shortest piece, in k-step pairs, a split may cut (tiles with
  // fewer pairs are not split).
  int sk_min_pairs = 4;
  float* work = nullptr; // stream-K partial tiles, grown on demand
  size_t work_bytes = 0;
  int occ_cache[3][5][pgemm::kNumBodies] = {}; // occupancy per (dtype, mode, body); 0 = not queried yet
  char last_error[512] = {0};
};

namespace pgemm {

inline int fail(pgemm_ctx* h, int status, const char* fmt, ...) {
  if (h) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(h->last_error, sizeof(h->last_error), fmt, ap);
    va_end(ap);
  }
  return status;
}

// Makes the handle's device current for the length of a call and gives the
// caller's back (the operators may be called between torch's own launches).
class DeviceScope {
 public:
  explicit DeviceScope(int device) {
    if (hipGetDevice(&before_) != hipSuccess) before_ = -1;
    ok_ = before_ == device || hipSetDevice(device) == hipSuccess;
    if (before_ == device) before_ = -1;
  }
  ~DeviceScope() {
    if (before_ >= 0) (void)hipSetDevice(before_);
  }
  DeviceScope(const DeviceScope&) = delete;
  DeviceScope& operator=(const DeviceScope&) = delete;
  bool ok() const { return ok_; }

 private:
  int before_ = -1;
  bool ok_ = false;
};

// Status of a call's launches (the first that failed), as a pgemm_status_t.
inline int launch_status(pgemm_ctx* h, hipError_t e, const char* what) {
  return e == hipSuccess ? PGEMM_OK : fail(h, PGEMM_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

} // namespace pgemm
