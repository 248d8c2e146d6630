// Instantiations of the few-row attention kernel.
#include "attend_few.hpp"
#include "attend_kernels.hpp"

namespace sgemv_dev {
template <class T>
static AttendFn pick(int dim) {
  if (dim <= 64) return dim == 64 ? attend_few_kernel<T, 64, true> : attend_few_kernel<T, 64, false>;
  if (dim <= 128) return dim == 128 ? attend_few_kernel<T, 128, true> : attend_few_kernel<T, 128, false>;
  return dim == 256 ? attend_few_kernel<T, 256, true> : attend_few_kernel<T, 256, false>;
}
AttendFn get_attend_few(bool bf16, int dim) { return bf16 ? pick<__bf16>(dim) : pick<_Float16>(dim); }
}  // namespace sgemv_dev
