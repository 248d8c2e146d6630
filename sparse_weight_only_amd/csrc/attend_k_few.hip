// Instantiations of the few-row attention kernel.
#include "attend_few.hpp"
#include "attend_kernels.hpp"

namespace sgemv_dev {
AttendFn get_attend_few(bool bf16, int dp) {
  if (bf16) return dp == 64 ? attend_few_kernel<__bf16, 64> : dp == 128 ? attend_few_kernel<__bf16, 128> : attend_few_kernel<__bf16, 256>;
  return dp == 64 ? attend_few_kernel<_Float16, 64> : dp == 128 ? attend_few_kernel<_Float16, 128> : attend_few_kernel<_Float16, 256>;
}
}  // namespace sgemv_dev
