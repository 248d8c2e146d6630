// Which instantiation of the attention kernels a width asks for.
#pragma once
#include "attend_few.hpp"
#include "attend_kernels.hpp"
#include "attend_many.hpp"

namespace sgemv_dev {

template <class T, bool EIGHT, bool WINDOW>
AttendFn pick_few(int dim) {
  if (dim <= 64) return dim == 64 ? attend_few_kernel<T, 64, true, EIGHT, WINDOW> : attend_few_kernel<T, 64, false, EIGHT, WINDOW>;
  if (dim <= 128) return dim == 128 ? attend_few_kernel<T, 128, true, EIGHT, WINDOW> : attend_few_kernel<T, 128, false, EIGHT, WINDOW>;
  return dim == 256 ? attend_few_kernel<T, 256, true, EIGHT, WINDOW> : attend_few_kernel<T, 256, false, EIGHT, WINDOW>;
}
template <bool EIGHT, bool WINDOW>
AttendFn get_attend_few(bool bf16, int dim) { return bf16 ? pick_few<__bf16, EIGHT, WINDOW>(dim) : pick_few<_Float16, EIGHT, WINDOW>(dim); }

template <class T, int DP, bool WHOLE, bool EIGHT, bool WINDOW>
AttendFn pick_halves(bool halves) {
  if constexpr (DP < 256)
    if (halves) return attend_many_kernel<T, DP, WHOLE, true, EIGHT, WINDOW>;
  return attend_many_kernel<T, DP, WHOLE, false, EIGHT, WINDOW>;
}
template <class T, bool EIGHT, bool WINDOW>
AttendFn pick_many(int dim, bool halves) {
  if (dim <= 64) return dim == 64 ? pick_halves<T, 64, true, EIGHT, WINDOW>(halves) : pick_halves<T, 64, false, EIGHT, WINDOW>(halves);
  if (dim <= 128) return dim == 128 ? pick_halves<T, 128, true, EIGHT, WINDOW>(halves) : pick_halves<T, 128, false, EIGHT, WINDOW>(halves);
  return dim == 256 ? pick_halves<T, 256, true, EIGHT, WINDOW>(false) : pick_halves<T, 256, false, EIGHT, WINDOW>(false);
}
template <bool EIGHT, bool WINDOW>
AttendFn get_attend_many(bool bf16, int dim, bool halves) {
  return bf16 ? pick_many<__bf16, EIGHT, WINDOW>(dim, halves) : pick_many<_Float16, EIGHT, WINDOW>(dim, halves);
}

}  // namespace sgemv_dev
