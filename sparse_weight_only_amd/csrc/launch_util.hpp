// Launch helpers shared by the launchers.
#pragma once
#include <stdint.h>

namespace sgemv {

// Raises a kernel's dynamic LDS limit where a launch needs more than 64 KiB;
// SGEMV_OK or SGEMV_EHIP.
int ensure_lds(const void* fn, int64_t lds_bytes);

}  // namespace sgemv
