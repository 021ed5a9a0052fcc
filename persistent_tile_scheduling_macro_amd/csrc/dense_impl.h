// The linear layer's kernels of one element type, included by its translation unit only.
#pragma once

#include "dense_few.h"
#include "dense_pp.h"
#include "dense_rows.h"
#include "dense_tile.h"

namespace pgemm {
namespace dense {

template <int DT, int FORM, bool GATED>
kernel_fn pick_form(int body) {
  if constexpr (FORM != kGrad) {
    constexpr bool NK = FORM == kRowsNK;
    constexpr int BLK = NK ? (GATED ? 2 : 1) : (GATED ? 8 : 4);
    switch (body) {
      case kFew8: return few_kernel<DT, NK, GATED, 8, BLK, 8>;
      case kFew16: return few_kernel<DT, NK, GATED, 16, BLK, 8>;
      case kFew32: return few_kernel<DT, NK, GATED, 32, BLK, 8>;
      case kTile64: return tile_kernel<DT, FORM, GATED, 64, 6>;
    }
  }
  return body == kPing ? ping_kernel<DT, FORM, GATED> : body == kTile128Pair ? tile_kernel<DT, FORM, GATED, 128, 2>
                                                                            : tile_kernel<DT, FORM, GATED, 128, 5>;
}
template <int DT>
kernel_fn pick(int body, int form, bool gated) {
  if (form == kGrad) return pick_form<DT, kGrad, false>(body);
  if (form == kRowsNK) return gated ? pick_form<DT, kRowsNK, true>(body) : pick_form<DT, kRowsNK, false>(body);
  return gated ? pick_form<DT, kRowsKN, true>(body) : pick_form<DT, kRowsKN, false>(body);
}
template <int DT>
void (*pick_both(int body, int form))(Args, Args, int, int) {
  const bool pair = body == kTile128Pair;
  if (form == kRowsNK) return pair ? both_kernel<DT, kRowsNK, 2> : both_kernel<DT, kRowsNK, 4>;
  return pair ? both_kernel<DT, kRowsKN, 2> : both_kernel<DT, kRowsKN, 4>;
}
template <int DT>
Kernels kernels() {
  return {pick<DT>, {join_kernel<DT, false>, join_kernel<DT, true>}, pick_both<DT>, join_both_kernel<DT>,
          {act_grad_kernel<DT, false>, act_grad_kernel<DT, true>}, side_kernel<DT>};
}

} // namespace dense
} // namespace pgemm
