// Instantiations of the many-row attention kernel and of the join of splits.
#include "attend_join.hpp"
#include "attend_kernels.hpp"
#include "attend_many.hpp"

namespace sgemv_dev {
template <class T, int DP, bool WHOLE>
static AttendFn pick_halves(bool halves) {
  if constexpr (DP < 256)
    if (halves) return attend_many_kernel<T, DP, WHOLE, true>;
  return attend_many_kernel<T, DP, WHOLE, false>;
}
template <class T>
static AttendFn pick(int dim, bool halves) {
  if (dim <= 64) return dim == 64 ? pick_halves<T, 64, true>(halves) : pick_halves<T, 64, false>(halves);
  if (dim <= 128) return dim == 128 ? pick_halves<T, 128, true>(halves) : pick_halves<T, 128, false>(halves);
  return dim == 256 ? pick_halves<T, 256, true>(false) : pick_halves<T, 256, false>(false);
}
AttendFn get_attend_many(bool bf16, int dim, bool halves) { return bf16 ? pick<__bf16>(dim, halves) : pick<_Float16>(dim, halves); }

template <class T, int DP>
static AttendJoinFn join_rows(bool many) { return many ? attend_join_rows_kernel<T, DP> : attend_join_kernel<T, DP>; }
template <class T>
static AttendJoinFn pick_join(int dim, bool many) {
  return dim <= 64 ? join_rows<T, 64>(many) : dim <= 128 ? join_rows<T, 128>(many) : join_rows<T, 256>(many);
}
AttendJoinFn get_attend_join(bool bf16, int dim, bool many_rows) { return bf16 ? pick_join<__bf16>(dim, many_rows) : pick_join<_Float16>(dim, many_rows); }
}  // namespace sgemv_dev
