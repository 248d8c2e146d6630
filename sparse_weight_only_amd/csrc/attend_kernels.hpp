// Attention kernels by type and padded head width (64, 128 or 256).
#pragma once
#include "attend_device.hpp"

namespace sgemv_dev {
typedef void (*AttendJoinFn)(AttendParams, int, int);
AttendFn get_attend_few(bool bf16, int dp);
AttendFn get_attend_many(bool bf16, int dp);
AttendJoinFn get_attend_join(bool bf16);
}  // namespace sgemv_dev
