// gfx950 kernel of the accumulated attention weights.
//
//   weight_j += sum over accepted rows i and heads h of the group of exp(c q_ih.k_j - lse_ih)
// One wave takes one slot of one kv head and walks over the rows; a slot has one owner, so the sums
// need no atomics and come in a fixed order.
#include <hip/hip_runtime.h>

#include "paged.h"
#include "wave_ops.h"

namespace specdec {
namespace {

constexpr int kWeightWaves = 4;
constexpr int kWeightGroups = 64;  // workgroups per (sequence, head)
constexpr int kPerLane = kMaxHeadDim / 64;

template <typename T>
__global__ __launch_bounds__(64 * kWeightWaves) void kv_weights_kernel(WeightArgs a, KvArgs c) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int group = a.q_heads / c.heads;
  const long long pairs = static_cast<long long>(a.B) * c.heads;
  for (long long bh = blockIdx.y; bh < pairs; bh += gridDim.y) {
    const int b = static_cast<int>(bh / c.heads), g = static_cast<int>(bh - (bh / c.heads) * c.heads);
    const RoundRows r = round_rows(c, a.num_draft, a.kv_len, b, a.K);
    const int accepted = r.n == 0 ? -1 : a.accept_len ? a.accept_len[b] : r.n - 1;
    if (accepted < 0 || accepted >= r.n) continue;
    for (int j = blockIdx.x * kWeightWaves + wave; j <= r.len + accepted;
         j += gridDim.x * kWeightWaves) {
      const int page = page_of(c, b, j);
      if (page < 0) continue;
      const T* k = reinterpret_cast<const T*>(c.k) + row_at(c, page, j % c.page_size, g);
      float kv[kPerLane];
#pragma unroll
      for (int e = 0; e < kPerLane; ++e)
        kv[e] = lane + 64 * e < c.dim ? to_float(k[lane + 64 * e]) : 0.f;
      float sum = 0.f;
      for (int i = max(0, j - r.len); i <= accepted; ++i) {
        const long long token = static_cast<long long>(b) * (a.K + 1) + i;
        for (int h = g * group; h < (g + 1) * group; ++h) {
          const T* q = static_cast<const T*>(a.q) + token * a.q_stride + h * static_cast<long long>(c.dim);
          float x = 0.f;
#pragma unroll
          for (int e = 0; e < kPerLane; ++e)
            if (lane + 64 * e < c.dim) x += kv[e] * to_float(q[lane + 64 * e]);
          sum += expf(wave_sum_f(x) * a.scale - a.lse[token * a.q_heads + h]);
        }
      }
      if (lane == 0) c.weight[record_at(c, page, j % c.page_size, g)] += sum;
    }
  }
}

}  // namespace

hipError_t launch_kv_weights(const WeightArgs& a, const KvArgs& c, int dtype) {
  const long long pairs = static_cast<long long>(a.B) * c.heads;
  const dim3 grid(kWeightGroups, static_cast<unsigned>(pairs < 65535 ? pairs : 65535));
  const dim3 block(64 * kWeightWaves);
  if (dtype == 0)
    kv_weights_kernel<float><<<grid, block, 0, a.stream>>>(a, c);
  else if (dtype == 1)
    kv_weights_kernel<__bf16><<<grid, block, 0, a.stream>>>(a, c);
  else
    kv_weights_kernel<_Float16><<<grid, block, 0, a.stream>>>(a, c);
  return hipGetLastError();
}

}  // namespace specdec
