// The attention kernel for f16 caches.
#include "attend_dev.h"

namespace specdec {

void launch_attend_f16(const AttendArgs& a, const KvArgs& c, const AttendPlan& p) {
  launch_attend_type<_Float16>(a, c, p);
}

}  // namespace specdec
