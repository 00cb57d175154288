// gfx950 attention over the paged cache: the plan of a call and the join of what it cut.
//
//   x_j = c q.k_j,  out = sum_j exp(x_j) v_j / sum_j exp(x_j)
// in one pass over the cache with a running maximum and sum, the query rows of a kv head's group and of
// all the round's tokens together (so K and V are read once for all of them).
//
// Bound: the cache's bytes.  A round has few rows (tokens x heads of a group), 4 rows flops a byte of the
// cache, which the matrix cores do in a tenth of the time that the bytes take; so the work is cut by
// bytes.  Sequences differ in length and one long one must not decide the time: the units of 128 slots of
// all (sequence, kv head, row chunk) segments are laid end to end and cut into equal contiguous ranges,
// one a workgroup.  A segment that lies in one range is written at once; the others leave one part a
// range (at most two a workgroup), which the join adds up.  A range ends in the first part of at most one
// cut segment, which it notes, so the join has as many workgroups to look at as there are ranges.
#include <hip/hip_runtime.h>

#include "attend_dev.h"

namespace specdec {
namespace {

// The row tiles and waves for the rows of a group: 16-row tiles a wave as needed up to what the
// registers hold (4; 1 for the widest heads), then more waves by rows, then chunks.
AttendPlan make_plan(int B, int K, int q_heads, int kv_heads, int dim, bool f32) {
  AttendPlan p{};
  const int rows = (K + 1) * (q_heads / kv_heads);
  p.dim = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
  p.tile_rows = rows <= 16 || p.dim == 256 ? 1 : rows <= 32 || (f32 && p.dim == 128) ? 2 : 4;
  const int wave_rows = 16 * p.tile_rows;
  p.row_waves = rows <= wave_rows ? 1 : rows <= 2 * wave_rows ? 2 : 4;
  p.rows = wave_rows * p.row_waves;
  p.chunks = (rows + p.rows - 1) / p.rows;
  p.groups = kAttendGroups;
  return p;
}

size_t align16(size_t x) { return (x + 15) & ~size_t{15}; }

}  // namespace

size_t attend_workspace_bytes(int B, int K, int q_heads, int kv_heads, int dim) {
  const AttendPlan p = make_plan(B, K, q_heads, kv_heads, dim, false);  // (f32 has no more rows)
  const size_t part_rows = 2 * static_cast<size_t>(p.groups) * p.rows;
  return p.groups * sizeof(CutSegment) + part_rows * p.dim * 4 + 2 * align16(part_rows * 4);
}

hipError_t launch_attend(const AttendArgs& a, const KvArgs& c, int dtype) {
  AttendPlan p = make_plan(a.B, a.K, a.q_heads, c.heads, c.dim, dtype == 0);
  const size_t part_rows = 2 * static_cast<size_t>(p.groups) * p.rows;
  char* ws = static_cast<char*>(a.workspace);
  p.cut = reinterpret_cast<CutSegment*>(ws);
  ws += p.groups * sizeof(CutSegment);
  p.part_o = reinterpret_cast<float*>(ws);
  ws += part_rows * p.dim * 4;
  p.part_m = reinterpret_cast<float*>(ws);
  ws += align16(part_rows * 4);
  p.part_l = reinterpret_cast<float*>(ws);
  p.page_shift = -1;
  if ((c.page_size & (c.page_size - 1)) == 0) p.page_shift = __builtin_ctz(c.page_size);
  p.scale_log2 = a.scale * kLog2e;
  if (dtype == 0)
    launch_attend_f32(a, c, p);
  else if (dtype == 1)
    launch_attend_bf16(a, c, p);
  else
    launch_attend_f16(a, c, p);
  return hipGetLastError();
}

}  // namespace specdec
