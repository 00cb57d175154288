// The attention kernel for bf16 caches.
#include "attend_dev.h"

namespace specdec {

void launch_attend_bf16(const AttendArgs& a, const KvArgs& c, const AttendPlan& p) {
  launch_attend_type<__bf16>(a, c, p);
}

}  // namespace specdec
