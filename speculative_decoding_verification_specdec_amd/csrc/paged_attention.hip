// gfx950 kernel of the attention over the paged cache.
//
//   x_j = c q.k_j,  out = sum_j exp(x_j) v_j / sum_j exp(x_j)
// in one pass with a running maximum and sum.  One workgroup takes one query row and head; its waves
// take the keys in turn, a lane holds every 64th element of a row.
#include <hip/hip_runtime.h>

#include "paged.h"
#include "wave_ops.h"

namespace specdec {
namespace {

constexpr int kAttendWaves = 4;
constexpr int kPerLane = kMaxHeadDim / 64;

template <typename T>
__global__ __launch_bounds__(64 * kAttendWaves) void attend_kernel(AttendArgs a, KvArgs c) {
  __shared__ float sh_m[kAttendWaves], sh_l[kAttendWaves], sh_o[kAttendWaves][kMaxHeadDim];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int group = a.q_heads / c.heads;
  const long long rows = static_cast<long long>(a.B) * (a.K + 1) * a.q_heads;
  for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
    const long long token = row / a.q_heads;
    const int h = static_cast<int>(row - token * a.q_heads);
    const int b = static_cast<int>(token / (a.K + 1));
    const int i = static_cast<int>(token - static_cast<long long>(b) * (a.K + 1));
    const RoundRows r = round_rows(c, a.num_draft, a.kv_len, b, a.K);
    const T* q = static_cast<const T*>(a.q) + token * a.q_stride + h * static_cast<long long>(c.dim);
    float qv[kPerLane], o[kPerLane];
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) {
      qv[e] = i < r.n && lane + 64 * e < c.dim ? to_float(q[lane + 64 * e]) : 0.f;
      o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    bool good = r.n > 0;
    const int total = r.len + r.n;
    for (int j = wave; i < r.n && j < total; j += kAttendWaves) {
      const int page = page_of(c, b, j);
      good = good && page >= 0;
      if (page < 0 || j > r.len + i) continue;
      const long long at = row_at(c, page, j % c.page_size, h / group);
      const T* k = reinterpret_cast<const T*>(c.k) + at;
      const T* v = reinterpret_cast<const T*>(c.v) + at;
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < kPerLane; ++e)
        if (lane + 64 * e < c.dim) x += qv[e] * to_float(k[lane + 64 * e]);
      x = wave_sum_f(x) * a.scale;
      const float top = fmaxf(m, x);
      const float base = top == -INFINITY ? 0.f : top;
      const float old = expf(m - base), p = expf(x - base);
      l = l * old + p;
#pragma unroll
      for (int e = 0; e < kPerLane; ++e)
        if (lane + 64 * e < c.dim) o[e] = o[e] * old + p * to_float(v[lane + 64 * e]);
      m = top;
    }
    if (!good) {
      m = 0.f;
      l = __builtin_nanf("");
    }
    if (lane == 0) {
      sh_m[wave] = m;
      sh_l[wave] = l;
    }
#pragma unroll
    for (int e = 0; e < kPerLane; ++e)
      if (lane + 64 * e < c.dim) sh_o[wave][lane + 64 * e] = o[e];
    __syncthreads();
    float top = -INFINITY;
    for (int w = 0; w < kAttendWaves; ++w) top = fmaxf(top, sh_m[w]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int w = 0; w < kAttendWaves; ++w) sum += sh_l[w] * expf(sh_m[w] - base);
    T* out = static_cast<T*>(a.out) + row * c.dim;
    const bool pad = i >= r.rows;
    for (int d = threadIdx.x; d < c.dim; d += blockDim.x) {
      float x = 0.f;
      for (int w = 0; w < kAttendWaves; ++w) x += sh_o[w][d] * expf(sh_m[w] - base);
      out[d] = from_float<T>(pad ? 0.f : x / sum);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[row] = pad ? -INFINITY : base + logf(sum);
    __syncthreads();
  }
}

}  // namespace

size_t attend_workspace_bytes(int B, int K, int q_heads, int kv_heads, int dim) { return 16; }

hipError_t launch_attend(const AttendArgs& a, const KvArgs& c, int dtype) {
  const long long rows = static_cast<long long>(a.B) * (a.K + 1) * a.q_heads;
  const dim3 grid(static_cast<unsigned>(rows < (1 << 22) ? rows : 1 << 22)), block(64 * kAttendWaves);
  if (dtype == 0)
    attend_kernel<float><<<grid, block, 0, a.stream>>>(a, c);
  else if (dtype == 1)
    attend_kernel<__bf16><<<grid, block, 0, a.stream>>>(a, c);
  else
    attend_kernel<_Float16><<<grid, block, 0, a.stream>>>(a, c);
  return hipGetLastError();
}

}  // namespace specdec
