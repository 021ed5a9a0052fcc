// The routed layer's kernels for f16 operands.
#include "layer.h"

namespace pgemm {
namespace layer {
kernel_fn up_f16(bool gated, int blocks, bool loop) { return pick_up<kF16>(gated, blocks, loop); }
kernel_fn down_f16(int blocks, bool is_short) { return pick_down<kF16>(blocks, is_short); }
} // namespace layer
} // namespace pgemm
