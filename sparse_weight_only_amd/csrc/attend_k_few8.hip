// Instantiations of the few-row attention kernel over a cache in 8 bits.
#include "attend_pick.hpp"

namespace sgemv_dev {
template AttendFn get_attend_few<true, false>(bool, int);
}  // namespace sgemv_dev
