// Attention kernels by type, head width (padded to 64, 128 or 256), cache and mask.
#pragma once
#include "attend_device.hpp"

namespace sgemv_dev {
typedef void (*AttendJoinFn)(AttendParams, int, int);
// EIGHT: over a cache in 8 bits; WINDOW: through a window
template <bool EIGHT, bool WINDOW> AttendFn get_attend_few(bool bf16, int dim);
template <bool EIGHT, bool WINDOW> AttendFn get_attend_many(bool bf16, int dim, bool halves);
AttendJoinFn get_attend_join(bool bf16, int dim, bool many_rows, bool window);
}  // namespace sgemv_dev
