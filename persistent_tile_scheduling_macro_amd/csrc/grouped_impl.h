// The grouped kernels of one element type, included by its translation unit only.
#pragma once

#include "grouped_few.h"
#include "grouped_pp.h"

namespace pgemm {
namespace grouped {

template <int DT>
kernel_fn pick(int body, bool grad, bool nk) {
  switch (body) {
    case kPingPong:
      return grad ? grouped_pp_kernel<DT, true, false> : nk ? grouped_pp_kernel<DT, false, true> : grouped_pp_kernel<DT, false, false>;
    case kFew16: return nk ? grouped_few_kernel<DT, true, 1, 1> : grouped_few_kernel<DT, false, 1, 4>;
    case kFew16Wide: return nk ? grouped_few_kernel<DT, true, 1, 2> : grouped_few_kernel<DT, false, 1, 4>;
    case kFew32Wide: return nk ? grouped_few_kernel<DT, true, 2, 2> : grouped_few_kernel<DT, false, 2, 4>;
    case kFewGrad: return grad_few_kernel<DT>;
    default:
      return grad ? grouped_kernel<DT, true, false> : nk ? grouped_kernel<DT, false, true> : grouped_kernel<DT, false, false>;
  }
}

} // namespace grouped
} // namespace pgemm
