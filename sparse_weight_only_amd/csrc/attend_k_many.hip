// Instantiations of the many-row attention kernel.
#include "attend_pick.hpp"

namespace sgemv_dev {
template AttendFn get_attend_many<false, false>(bool, int, bool);
}  // namespace sgemv_dev
