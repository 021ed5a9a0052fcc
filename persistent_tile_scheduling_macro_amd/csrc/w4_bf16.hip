// Instantiations of the 4-bit product for one element type.
#include "w4.h"

pgemm::w4::kernel_fn pgemm::w4::pick_bf16(int fmt, int group, int rows, int cb) { return pick<kBF16>(fmt, group, rows, cb); }
