// Kernel launches of the host code.
#pragma once

#include <hip/hip_runtime.h>

#include <tuple>

namespace pgemm {

// Enqueue a kernel and return this launch's own status. (The <<<>>> form gives none, and hipGetLastError returns the
// thread's last error, which an earlier call of anybody's may have left; that one is not read or cleared here.)
template <class... P, class... A>
hipError_t enqueue(hipStream_t stream, dim3 grid, dim3 block, void (*kernel)(P...), A... args) {
  std::tuple<P...> values(args...);
  return std::apply(
      [&](P&... p) {
        void* pointers[] = {&p...};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, pointers, 0, stream);
        if (e != hipSuccess) (void)hipGetLastError(); // reported by the caller, so not left behind
        return e;
      },
      values);
}

} // namespace pgemm
