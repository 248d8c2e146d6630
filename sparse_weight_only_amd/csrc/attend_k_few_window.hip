// Instantiations of the few-row attention kernel, through a window.
#include "attend_pick.hpp"

namespace sgemv_dev {
template AttendFn get_attend_few<false, true>(bool, int);
}  // namespace sgemv_dev
