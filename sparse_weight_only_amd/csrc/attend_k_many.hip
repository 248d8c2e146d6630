// Instantiations of the many-row attention kernel and of the join of splits.
#include "attend_kernels.hpp"
#include "attend_many.hpp"

namespace sgemv_dev {
AttendFn get_attend_many(bool bf16, int dp) {
  if (bf16) return dp == 64 ? attend_many_kernel<__bf16, 64> : dp == 128 ? attend_many_kernel<__bf16, 128> : attend_many_kernel<__bf16, 256>;
  return dp == 64 ? attend_many_kernel<_Float16, 64> : dp == 128 ? attend_many_kernel<_Float16, 128> : attend_many_kernel<_Float16, 256>;
}
AttendJoinFn get_attend_join(bool bf16) { return bf16 ? attend_join_kernel<__bf16> : attend_join_kernel<_Float16>; }
}  // namespace sgemv_dev
