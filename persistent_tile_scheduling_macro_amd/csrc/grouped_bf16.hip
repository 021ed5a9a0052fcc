// Instantiations of the grouped products for one element type.
#include "grouped.h"

pgemm::grouped::kernel_fn pgemm::grouped::pick_bf16(bool grad, bool nk) { return pick<kBF16>(grad, nk); }
