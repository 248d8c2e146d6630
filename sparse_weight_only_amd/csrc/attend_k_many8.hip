// Instantiations of the many-row attention kernel over a cache in 8 bits.
#include "attend_pick.hpp"

namespace sgemv_dev {
template AttendFn get_attend_many<true, false>(bool, int, bool);
}  // namespace sgemv_dev
