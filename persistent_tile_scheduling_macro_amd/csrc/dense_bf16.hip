// The linear layer's kernels for bf16 operands.
#include "dense_impl.h"

namespace pgemm {
namespace dense {
Kernels kernels_bf16() { return kernels<kBF16>(); }
} // namespace dense
} // namespace pgemm
