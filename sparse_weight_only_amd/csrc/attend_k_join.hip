// Instantiations of the join of split contexts.
#include "attend_join.hpp"
#include "attend_kernels.hpp"

namespace sgemv_dev {
template <class T, int DP, bool WINDOW>
static AttendJoinFn join_rows(bool many) { return many ? attend_join_rows_kernel<T, DP, WINDOW> : attend_join_kernel<T, DP, WINDOW>; }
template <class T, bool WINDOW>
static AttendJoinFn pick_join(int dim, bool many) {
  return dim <= 64 ? join_rows<T, 64, WINDOW>(many) : dim <= 128 ? join_rows<T, 128, WINDOW>(many) : join_rows<T, 256, WINDOW>(many);
}
template <class T>
static AttendJoinFn pick_window(int dim, bool many, bool window) { return window ? pick_join<T, true>(dim, many) : pick_join<T, false>(dim, many); }
AttendJoinFn get_attend_join(bool bf16, int dim, bool many_rows, bool window) {
  return bf16 ? pick_window<__bf16>(dim, many_rows, window) : pick_window<_Float16>(dim, many_rows, window);
}
}  // namespace sgemv_dev
