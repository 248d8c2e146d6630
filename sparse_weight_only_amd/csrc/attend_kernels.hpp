// Attention kernels by type and head width (padded to 64, 128 or 256).
#pragma once
#include "attend_device.hpp"

namespace sgemv_dev {
typedef void (*AttendJoinFn)(AttendParams, int, int);
AttendFn get_attend_few(bool bf16, int dim);
AttendFn get_attend_many(bool bf16, int dim, bool halves);
AttendJoinFn get_attend_join(bool bf16, int dim, bool many_rows);
}  // namespace sgemv_dev
