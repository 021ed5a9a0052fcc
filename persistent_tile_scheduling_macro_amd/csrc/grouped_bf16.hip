// Instantiations of the grouped products for one element type.
#include "grouped_impl.h"

pgemm::grouped::kernel_fn pgemm::grouped::pick_bf16(int body, bool grad, bool nk) { return pick<kBF16>(body, grad, nk); }
pgemm::grouped::kernel_fn pgemm::grouped::join_bf16(bool shared) {
  return shared ? join_pieces_kernel<kBF16, 8> : join_pieces_kernel<kBF16, 1>;
}
