// The attention kernel for f32 caches.
#include "attend_dev.h"

namespace specdec {

void launch_attend_f32(const AttendArgs& a, const KvArgs& c, const AttendPlan& p) {
  launch_attend_type<float>(a, c, p);
}

}  // namespace specdec
