// Instantiations of the few-row attention kernel.
#include "attend_few.hpp"
#include "attend_kernels.hpp"

namespace sgemv_dev {
template <class T, int DP, bool WHOLE>
static AttendFn pick_waves(int waves) {
  if constexpr (DP < 256)
    if (waves == 8) return attend_few_kernel<T, DP, WHOLE, 8>;
  return waves == 4 ? attend_few_kernel<T, DP, WHOLE, 4> : nullptr;
}
template <class T>
static AttendFn pick(int dim, int waves) {
  if (dim <= 64) return dim == 64 ? pick_waves<T, 64, true>(waves) : pick_waves<T, 64, false>(waves);
  if (dim <= 128) return dim == 128 ? pick_waves<T, 128, true>(waves) : pick_waves<T, 128, false>(waves);
  return dim == 256 ? pick_waves<T, 256, true>(waves) : pick_waves<T, 256, false>(waves);
}
AttendFn get_attend_few(bool bf16, int dim, int waves) { return bf16 ? pick<__bf16>(dim, waves) : pick<_Float16>(dim, waves); }
}  // namespace sgemv_dev
