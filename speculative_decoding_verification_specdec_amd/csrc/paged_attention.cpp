// gfx950 attention over the paged cache: the plan of a call and the join of what it cut.
//
//   x_j = c q.k_j,  out = sum_j exp(x_j) v_j / sum_j exp(x_j)
// in one pass over the cache with a running maximum and sum, the query rows of a kv head's group and of
// all the round's tokens together (so K and V are read once for all of them).
//
// Bound: the cache's bytes.  A round has few rows (tokens x heads of a group), 4 rows flops a byte of the
// cache, which the matrix cores do in a tenth of the time that the bytes take; so the work is cut by
// bytes.  Sequences differ in length and one long one must not decide the time: the 32-slot tiles of all
// (sequence, kv head, chunk of rows) segments are laid end to end and cut into equal contiguous ranges, one a
// wave.  A segment that lies in one range is written at once; the others leave one part a range (at most
// two a wave), which the join adds up.  A range ends in the first part of at most one cut segment, which
// it notes, so the join has as many segments to look at as there are ranges.
#include <hip/hip_runtime.h>

#include "attend_plan.h"

namespace specdec {
namespace {

// Up to 32 rows (16 of the widest heads, as their registers allow) every wave takes all rows of its own range:
// 1024 ranges, one wave a SIMD, four of them a workgroup where the LDS holds their parts.  (The kernel for more
// rows takes 130 us where this one takes 122, 64 x 500-4000 slots of 8 heads, 32 rows; 75 and 70 at 4 rows, head dim
// 64.)  More rows are shared
// out to the four waves of a workgroup, 64 or 128 a chunk, with a range for each workgroup that is resident: 512, or
// 256 where 128 rows of the widest heads allow one a CU (64 rows at 256 ranges: 157 us where 512 take 152, 64 x
// 500-4000 slots of 4 heads; 128 rows against 64 in two workgroups a CU: 558 and 697 us, 512 rows in all).
AttendPlan make_plan(int K, int q_heads, int kv_heads, int dim) {
  AttendPlan p{};
  const int rows = (K + 1) * (q_heads / kv_heads);
  p.dim = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
  p.wide = rows > (p.dim == 256 ? 16 : 32);
  if (p.wide) {
    p.rows = rows <= 64 ? 64 : 128;
    p.log_ranges = p.dim == 256 && p.rows == 128 ? 8 : 9;
  } else {
    p.rows = rows <= 16 ? 16 : 32;
    p.log_ranges = 10;
    p.log_waves = p.dim == 256 ? 0 : 2;
  }
  return p;
}

size_t align16(size_t x) { return (x + 15) & ~size_t{15}; }

}  // namespace

size_t attend_workspace_bytes(int K, int q_heads, int kv_heads, int dim) {
  const AttendPlan p = make_plan(K, q_heads, kv_heads, dim);
  const size_t groups = size_t{1} << (p.log_ranges - p.log_waves), part_rows = 2 * groups * p.rows;
  return groups * sizeof(CutSegment) + part_rows * p.dim * 4 + 2 * align16(part_rows * 4);
}

hipError_t launch_attend(const AttendArgs& a, const KvArgs& c, int dtype) {
  AttendPlan p = make_plan(a.K, a.q_heads, c.heads, c.dim);
  const size_t groups = size_t{1} << (p.log_ranges - p.log_waves), part_rows = 2 * groups * p.rows;
  char* ws = static_cast<char*>(a.workspace);
  p.cut = reinterpret_cast<CutSegment*>(ws);
  ws += groups * sizeof(CutSegment);
  p.part_o = reinterpret_cast<float*>(ws);
  ws += part_rows * p.dim * 4;
  p.part_m = reinterpret_cast<float*>(ws);
  ws += align16(part_rows * 4);
  p.part_l = reinterpret_cast<float*>(ws);
  p.page_shift = -1;
  if ((c.page_size & (c.page_size - 1)) == 0) p.page_shift = __builtin_ctz(c.page_size);
  p.scale_log2 = a.scale * 1.44269504088896340736f;
  if (dtype == 0)
    launch_attend_f32(a, c, p);
  else if (dtype == 1)
    launch_attend_bf16(a, c, p);
  else
    launch_attend_f16(a, c, p);
  return hipGetLastError();
}

}  // namespace specdec
