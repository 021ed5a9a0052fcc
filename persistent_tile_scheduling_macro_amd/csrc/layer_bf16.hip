// The routed layer's kernels for bf16 operands.
#include "layer.h"

namespace pgemm {
namespace layer {
kernel_fn up_bf16(bool gated, int blocks, bool loop) { return pick_up<kBF16>(gated, blocks, loop); }
kernel_fn down_bf16(int blocks, bool is_short) { return pick_down<kBF16>(blocks, is_short); }
} // namespace layer
} // namespace pgemm
