// The linear layer's kernels for f16 operands.
#include "dense_impl.h"

namespace pgemm {
namespace dense {
Kernels kernels_f16() { return kernels<kF16>(); }
} // namespace dense
} // namespace pgemm
