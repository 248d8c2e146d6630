// Instantiations of the many-row attention kernel, through a window.
#include "attend_pick.hpp"

namespace sgemv_dev {
template AttendFn get_attend_many<false, true>(bool, int, bool);
}  // namespace sgemv_dev
