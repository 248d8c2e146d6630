// Instantiations of the many-row attention kernel over a cache in 8 bits, through a window.
#include "attend_pick.hpp"

namespace sgemv_dev {
template AttendFn get_attend_many<true, true>(bool, int, bool);
}  // namespace sgemv_dev
