// Instantiations of the grouped products for one element type.
#include "grouped_impl.h"

pgemm::grouped::kernel_fn pgemm::grouped::pick_f16(int body, bool grad, bool nk) { return pick<kF16>(body, grad, nk); }
pgemm::grouped::kernel_fn pgemm::grouped::join_f16(bool shared) {
  return shared ? join_pieces_kernel<kF16, 8> : join_pieces_kernel<kF16, 1>;
}
