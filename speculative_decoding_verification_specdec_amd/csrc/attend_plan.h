// The plan of an attention call: how paged_attention.cpp cuts it and attend_dev.h's kernels follow it.
#pragma once

#include "paged.h"

namespace specdec {

// A segment that lies in the ranges of several workgroups: parts of workgroups w .. w + parts - 1 (parts 0:
// none); n: its sequence's new tokens.
struct alignas(32) CutSegment {
  int parts, b, seg, n;
};

// How a call is cut.  A segment is one (sequence, kv head, chunk of its query rows); its tiles, and those of all
// segments one after the other, are dealt out evenly to 1 << log_ranges waves in contiguous ranges.
struct AttendPlan {
  int log_ranges;
  int log_waves;        // log2(ranges a workgroup), neighbouring ones
  int wide;             // the kernel for many rows: one range a workgroup
  int rows;             // rows of a chunk: 16 a row tile
  int dim;              // kDim of the kernel
  int page_shift;       // log2(page_size), or -1
  float scale_log2;     // scale * log2(e)
  CutSegment* cut;      // [workgroups] the cut segment whose first part a workgroup holds
  float* part_o;        // [2 workgroups][rows][dim] unnormalised outputs: of the segment that comes from the
  float* part_m;        // [2 workgroups][rows]      workgroup before (0) and of the one that begins here (1);
  float* part_l;        // [2 workgroups][rows]      their bases (of scores * log2(e)) and sums
};

// The split and the join of a call, by the cache's element type.
void launch_attend_bf16(const AttendArgs& a, const KvArgs& c, const AttendPlan& p);
void launch_attend_f16(const AttendArgs& a, const KvArgs& c, const AttendPlan& p);
void launch_attend_f32(const AttendArgs& a, const KvArgs& c, const AttendPlan& p);

}  // namespace specdec
