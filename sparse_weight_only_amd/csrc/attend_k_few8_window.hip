// Instantiations of the few-row attention kernel over a cache in 8 bits, through a window.
#include "attend_pick.hpp"

namespace sgemv_dev {
template AttendFn get_attend_few<true, true>(bool, int);
}  // namespace sgemv_dev
