// Instantiations of the grouped products for one element type.
#include "grouped.h"

pgemm::grouped::kernel_fn pgemm::grouped::pick_f16(bool grad, bool nk) { return pick<kF16>(grad, nk); }
