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
// range (at most two a workgroup), which the join adds up.
#include <hip/hip_runtime.h>

#include "attend_dev.h"

namespace specdec {
namespace {

// One wave per output row: rows past the last new token are 0, those of an invalid sequence NaN, those
// of a cut segment the sum of its parts; the others are there already.
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, KvArgs c, AttendPlan plan,
                                                          int dtype) {
  const int lane = threadIdx.x & 63;
  const long long rows = static_cast<long long>(a.B) * (a.K + 1) * a.q_heads;
  const int group = a.q_heads / c.heads;
  const long long all = plan.prefix[a.B] * c.heads * plan.chunks;
  const int groups = active_groups(all, plan.groups);
  for (long long row = blockIdx.x * 4LL + (threadIdx.x >> 6); row < rows; row += gridDim.x * 4LL) {
    const long long token = row / a.q_heads;
    const int h = static_cast<int>(row - token * a.q_heads);
    const int b = static_cast<int>(token / (a.K + 1));
    const int i = static_cast<int>(token - static_cast<long long>(b) * (a.K + 1));
    const RoundRows r = round_rows(c, a.num_draft, a.kv_len, b, a.K);
    float o[kMaxHeadDim / 64] = {};
    float lse = -INFINITY;
    if (i < r.rows) {
      if (r.n > 0) {
        const int kvh = h / group;
        const int qrow = i * group + h - kvh * group, chunk = qrow / plan.rows;
        const int local = qrow - chunk * plan.rows;
        const long long units = units_of(r);
        const long long u0 = plan.prefix[b] * c.heads * plan.chunks + (kvh * plan.chunks + chunk) * units;
        const int w0 = owner_of(u0, all, groups), w1 = owner_of(u0 + units - 1, all, groups);
        if (w0 == w1) continue;
        // The first range holds its piece last unless the segment starts with it; the others start with it.
        const int slot0 = range_begin(w0, all, groups) == u0 ? 0 : 1;
        float top = -INFINITY, sum = 0.f;
        for (int w = w0; w <= w1; w += 64) {
          const int n = min(64, w1 - w + 1);
          float m = -INFINITY, l = 0.f;
          if (lane < n) {
            const long long at = (2LL * (w + lane) + (w + lane == w0 ? slot0 : 0)) * plan.rows + local;
            m = plan.part_m[at];
            l = plan.part_l[at];
          }
          const float now = fmaxf(top, wave_max_f(m)), base = now == -INFINITY ? 0.f : now;
          const float old = exp2_hw(top - base), f = exp2_hw(m - base);
          sum = sum * old + wave_sum_f(l * f);
#pragma unroll
          for (int e = 0; e < kMaxHeadDim / 64; ++e) o[e] *= old;
          for (int x = 0; x < n; ++x) {
            const float fx = __shfl(f, x, 64);
            const float* src =
                plan.part_o +
                ((2LL * (w + x) + (w + x == w0 ? slot0 : 0)) * plan.rows + local) * plan.dim;
#pragma unroll
            for (int e = 0; e < kMaxHeadDim / 64; ++e)
              if (lane + 64 * e < c.dim) o[e] += fx * src[lane + 64 * e];
          }
          top = now;
        }
        const float inv = 1.f / sum;
#pragma unroll
        for (int e = 0; e < kMaxHeadDim / 64; ++e) o[e] *= inv;
        lse = top == -INFINITY ? __builtin_nanf("") : top * kLn2 + logf(sum);
      } else {
        lse = __builtin_nanf("");
#pragma unroll
        for (int e = 0; e < kMaxHeadDim / 64; ++e) o[e] = lse;
      }
    }
#pragma unroll
    for (int e = 0; e < kMaxHeadDim / 64; ++e) {
      const int d = lane + 64 * e;
      if (d >= c.dim) continue;
      if (dtype == 0)
        static_cast<float*>(a.out)[row * c.dim + d] = o[e];
      else if (dtype == 1)
        static_cast<__bf16*>(a.out)[row * c.dim + d] = from_float<__bf16>(o[e]);
      else
        static_cast<_Float16*>(a.out)[row * c.dim + d] = from_float<_Float16>(o[e]);
    }
    if (lane == 0 && a.lse) a.lse[row] = lse;
  }
}

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
  return align16((static_cast<size_t>(B) + 1) * 8) + part_rows * p.dim * 4 + 2 * align16(part_rows * 4);
}

hipError_t launch_attend(const AttendArgs& a, const KvArgs& c, int dtype) {
  AttendPlan p = make_plan(a.B, a.K, a.q_heads, c.heads, c.dim, dtype == 0);
  const size_t part_rows = 2 * static_cast<size_t>(p.groups) * p.rows;
  char* ws = static_cast<char*>(a.workspace);
  p.prefix = reinterpret_cast<long long*>(ws);
  ws += align16((static_cast<size_t>(a.B) + 1) * 8);
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
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const long long rows = static_cast<long long>(a.B) * (a.K + 1) * a.q_heads;
  const long long blocks = (rows + 3) / 4;
  attend_join_kernel<<<static_cast<unsigned>(blocks < (1 << 20) ? blocks : 1 << 20), 256, 0, a.stream>>>(
      a, c, p, dtype);
  return hipGetLastError();
}

}  // namespace specdec
