// Instantiations of the few-row attention kernel.
#include "attend_pick.hpp"

namespace sgemv_dev {
template AttendFn get_attend_few<false, false>(bool, int);
}  // namespace sgemv_dev
