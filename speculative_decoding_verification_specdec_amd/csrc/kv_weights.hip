// gfx950 kernel of the accumulated attention weights.
//
//   weight_j += sum over accepted rows i and heads h of the group of exp(c q_ih.k_j - lse_ih)
// The scores come as matrix products S [rows x slots] = Q . K^T, so that a lane's four results belong to one slot
// (its column lane % 16) and four rows: the sum over rows is made in the lane, and at the end of a tile over the
// four lanes 16 apart.  A slot is one wave's, so there are no atomics and the order is fixed.
//
// Bound: the bytes of K and of the weights, which are read and written; each byte of K once, streamed from
// memory to registers.  The query rows, which all slots of a segment (one sequence and kv head) share, lie in LDS
// operand by operand.  (Plain loads: streaming ones, which are faster where nothing is written, took 543 us for
// 64 x 16380 slots of 8 heads where plain ones take 481, 391 of them without the weights' stores; holding stores back
// in LDS for 4-16 tiles changed that by 1%.)  The tiles of all segments, laid end to end and weighed by what they
// cost, are cut into equal ranges, one a workgroup, whose four waves take the range's tiles in turn.
// 64 x 500-4000 slots of 8 heads, up to 24 rows, bf16: 69 us, 4.4 TB/s; 4 x 50-65 k slots, up to 48 rows: 105 us.
#include <hip/hip_runtime.h>

#include "paged.h"
#include "paged_tiles.h"
#include "wave_ops.h"

namespace specdec {
namespace {

constexpr int kWeightWaves = 4;
constexpr int kQueryBytes = 32768;  // of LDS for query operands: four workgroups a CU
// What reading a tile costs, in units of the arithmetic on 16 rows of it: 8 KiB at a SIMD's share of the memory's
// rate take as long as the products and exponentials of ten row tiles.  (40 instead changed nothing at 24 rows and
// took 96 us for 92 at 512.)
constexpr int kTileCost = 10;

struct WeightPlan {
  int log_ranges;
  int chunk;         // row tiles that LDS holds at once
  int page_shift;    // log2(page_size), or -1
  float scale_log2;  // scale * log2(e)
};

// A sequence's part of the work: tiles of each of its kv heads, and what one costs.
struct WeightRows {
  int len, rows, accepted, tiles, cost;
};

template <int kKeys>
__device__ __forceinline__ WeightRows weight_rows(const WeightArgs& a, const KvArgs& c, int group, int b) {
  const RoundRows r = round_rows(c, a.num_draft, a.kv_len, b, a.K);
  const int accepted = r.n == 0 ? -1 : a.accept_len ? a.accept_len[b] : r.n - 1;
  WeightRows w{r.len, 0, accepted, 0, 0};
  if (accepted >= 0 && accepted < r.n) {
    w.rows = (accepted + 1) * group;
    w.tiles = (r.len + accepted) / kKeys + 1;
    w.cost = kTileCost + (w.rows + 15) / 16;
  }
  return w;
}
__device__ __forceinline__ long long weight_work(const WeightRows& w, int heads) {
  return static_cast<long long>(w.tiles) * heads * w.cost;
}

// floor(n / d) for 0 <= n < 2^52: an f64 quotient that is no integer stays away from the next one.
__device__ __forceinline__ long long quotient(long long n, long long d) {
  return static_cast<long long>(static_cast<double>(n) / static_cast<double>(d));
}

// kFast: head_dim is kDim, pages are whole groups of 16 slots and 16 slots lie within 2^32 bytes.
template <typename T, int kDim, bool kFast>
struct WeightWave {
  typedef Tile<T, kDim, kFast> L;

  const KvArgs& c;
  int page_shift, lane, col, g, head, last;
  const T* kpool;          // of the kv head
  const int32_t* table;    // of the sequence
  struct Keys {
    u32x4 f[L::kSub][L::kSteps];
    long long record;      // where the weight of slot lane % kKeys lies, -1: nowhere
  };

  __device__ __forceinline__ explicit WeightWave(const KvArgs& args) : c(args) {}

  __device__ __forceinline__ int page_index(int slot) const {
    return page_shift >= 0
               ? slot >> page_shift
               : static_cast<int>(static_cast<unsigned>(slot) / static_cast<unsigned>(c.page_size));
  }

  __device__ __forceinline__ void fetch(Keys& k, int tile) const {
    const int mine = lane & (L::kKeys - 1);  // the slot whose weight this lane keeps
    const bool used = tile * L::kKeys + mine <= last;
    if constexpr (kFast) {
      int page[L::kSub], off[L::kSub];
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub) {
        // (a group past the last slot takes the last slot's)
        const int slot = min(tile * L::kKeys + 16 * sub, last & ~15);
        const int idx = uniform(page_index(slot));
        off[sub] = slot - idx * c.page_size;
        page[sub] = table_at(table, idx);
      }
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub) {
        const bool good = static_cast<unsigned>(page[sub]) < static_cast<unsigned>(c.num_pages);
        L::template load_row<false>(
            k.f[sub], scalar_base(kpool + ((good ? page[sub] : 0) * c.page_stride + off[sub] * c.slot_stride)),
            static_cast<unsigned>(col) * static_cast<unsigned>(c.slot_stride), g, c.dim);
        if (mine >> 4 == sub) k.record = good && used ? record_at(c, page[sub], off[sub] + col, head) : -1;
      }
    } else {
      const int slot = min(tile * L::kKeys + mine, last);
      const int idx = page_index(slot), off = slot - idx * c.page_size, page = table[idx];
      const bool good = static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages);
      const long long row = (good ? page : 0) * c.page_stride + off * c.slot_stride;
      k.record = good && used ? record_at(c, page, off, head) : -1;
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub)
        L::template load_row<false>(k.f[sub], (GlobalBytes)(kpool + shfl64(row, 16 * sub + col)), 0u, g, c.dim);
    }
  }

  // exp(score - lse) of 16 rows, added up over the lane's four.  kMasked: rows that do not see the slot, and
  // those past the last one, add nothing whatever their score is.
  template <bool kMasked>
  __device__ __forceinline__ void add_rows(float (&sum)[L::kSub], const Keys& k, const u32x4 (*q)[64], const float* lse,
                                           const int* limit, float scale, int first) const {
    f32x4 x[L::kSub];
#pragma unroll
    for (int sub = 0; sub < L::kSub; ++sub) x[sub] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < L::kSteps; ++s) {
      const u32x4 rows = q[s][lane];
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub) x[sub] = mma16(rows, k.f[sub][s], x[sub], T{});
    }
    const f32x4 base = *reinterpret_cast<const f32x4*>(lse + 4 * g);
#pragma unroll
    for (int sub = 0; sub < L::kSub; ++sub) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[sub][r] = __builtin_amdgcn_exp2f(fmaf(x[sub][r], scale, -base[r]));
        if (kMasked && first + 16 * sub + col > limit[4 * g + r]) x[sub][r] = 0.f;
      }
      sum[sub] += (x[sub][0] + x[sub][1]) + (x[sub][2] + x[sub][3]);
    }
  }

  __device__ __forceinline__ void add_tile(const Keys& k, int tile, float old, const u32x4 (*q)[64],
                                           const float* lse, const int* limit, int rows, float scale, int len) const {
    float sum[L::kSub] = {};
    const int first = tile * L::kKeys;
    const int whole = first + L::kKeys - 1 > len ? 0 : rows / 16;  // row tiles of which every row sees every slot
    int t = 0;
    for (; t < whole; ++t) add_rows<false>(sum, k, q + t * L::kSteps, lse + 16 * t, limit, scale, first);
    for (; 16 * t < rows; ++t)
      add_rows<true>(sum, k, q + t * L::kSteps, lse + 16 * t, limit + 16 * t, scale, first);
    float all = row_sum(sum[0]);
    if constexpr (L::kSub == 2) {
      const float other = row_sum(sum[1]);
      all = lane & 16 ? other : all;
    }
    if (lane < L::kKeys && k.record >= 0) c.weight[k.record] = old + all;
  }

  __device__ __forceinline__ float old_weight(const Keys& k) const {
    return lane < L::kKeys && k.record >= 0 ? c.weight[k.record] : 0.f;
  }
};

template <typename T, int kDim, bool kFast>
__global__ __launch_bounds__(64 * kWeightWaves, kDim == 256 ? 2 : 4) void kv_weights_kernel(WeightArgs a, KvArgs c,
                                                                                          WeightPlan plan) {
  typedef WeightWave<T, kDim, kFast> Wave;
  typedef typename Wave::L L;
  extern __shared__ u32x4 sh_q[][64];                                  // [row tiles][steps][lane]
  float* sh_lse = reinterpret_cast<float*>(sh_q + plan.chunk * L::kSteps);  // lse * log2(e) of the rows
  int* sh_limit = reinterpret_cast<int*>(sh_lse + 16 * plan.chunk);    // the last slot that a row sees
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int group = a.q_heads / c.heads;

  // Work before each sequence: every lane sums a run of sequences, then a scan over the lanes.
  const int per = (a.B + 63) / 64;
  const int run0 = min(a.B, lane * per), run1 = min(a.B, run0 + per);
  long long mine = 0;
  for (int b = run0; b < run1; ++b) mine += weight_work(weight_rows<L::kKeys>(a, c, group, b), c.heads);
  const long long upto = scan_work(mine);
  const long long total = read_lane64(upto, 63);
  // The range takes the tiles that begin in it.
  const long long begin = blockIdx.x * total >> plan.log_ranges, end = (blockIdx.x + 1LL) * total >> plan.log_ranges;
  if (begin >= end) return;
  const int owner = __builtin_ctzll(__ballot(mine > 0 && begin < upto));
  long long before = read_lane64(upto - mine, owner);  // work before sequence b's head `head`
  int b = uniform(owner * per);
  WeightRows now = weight_rows<L::kKeys>(a, c, group, b);
  for (; begin >= before + weight_work(now, c.heads); now = weight_rows<L::kKeys>(a, c, group, ++b))
    before += weight_work(now, c.heads);
  long long segment = static_cast<long long>(now.tiles) * now.cost;
  int head = uniform(static_cast<int>(quotient(begin - before, segment)));
  before += head * segment;

  Wave s(c);
  s.page_shift = plan.page_shift;
  s.lane = lane;
  s.col = lane & 15;
  s.g = lane >> 4;
  for (;;) {
    const int first = uniform(static_cast<int>(quotient(max(0LL, begin - before) + now.cost - 1, now.cost)));
    const int stop =
        uniform(static_cast<int>(min<long long>(now.tiles, quotient(end - before + now.cost - 1, now.cost))));
    s.head = head;
    s.last = uniform(now.len + now.accepted);
    s.kpool = reinterpret_cast<const T*>(c.k) + head * c.head_stride;
    s.table = c.table + static_cast<long long>(b) * c.max_pages;
    const int len = uniform(now.len);
    for (int row0 = 0; first < stop && row0 < now.rows; row0 += 16 * plan.chunk) {
      typename Wave::Keys k0, k1;
      int tile = first + wave;
      if (tile < stop) s.fetch(k0, tile);
      // The rows' operands, and what their scores need.
      const int rows = uniform(min(now.rows - row0, 16 * plan.chunk));
      __syncthreads();  // (the rows before are done with)
      for (int u = wave; u < (rows + 15) / 16 * L::kSteps; u += kWeightWaves) {
        const int t = u / L::kSteps, row = row0 + 16 * t + s.col, i = row / group;
        u32x4 x = {0, 0, 0, 0};
        if (row < now.rows)
          x = L::template load_step<false>(
              (GlobalBytes)(static_cast<const T*>(a.q) + (static_cast<long long>(b) * (a.K + 1) + i) * a.q_stride +
                            static_cast<long long>(head * group + row - i * group) * c.dim),
              0u, u - t * L::kSteps, s.g, c.dim);
        sh_q[u][lane] = x;
      }
      for (int x = threadIdx.x; x < (rows + 15) / 16 * 16; x += 64 * kWeightWaves) {
        const int row = row0 + x, i = row / group;
        const bool real = row < now.rows;
        sh_limit[x] = real ? len + i : -1;
        sh_lse[x] = real ? a.lse[(static_cast<long long>(b) * (a.K + 1) + i) * a.q_heads + head * group + row -
                                 i * group] * kLog2e
                         : 0.f;
      }
      __syncthreads();
      // The next tile's keys are on their way while this one is computed on; the weight that it adds to is asked
      // for before them.
      while (tile < stop) {
        float old = s.old_weight(k0);
        if (tile + kWeightWaves < stop) s.fetch(k1, tile + kWeightWaves);
        s.add_tile(k0, tile, old, sh_q, sh_lse, sh_limit, rows, plan.scale_log2, len);
        tile += kWeightWaves;
        if (tile >= stop) break;
        old = s.old_weight(k1);
        if (tile + kWeightWaves < stop) s.fetch(k0, tile + kWeightWaves);
        s.add_tile(k1, tile, old, sh_q, sh_lse, sh_limit, rows, plan.scale_log2, len);
        tile += kWeightWaves;
      }
    }
    before += segment;
    if (before >= end) return;
    if (++head == c.heads) {
      head = 0;
      do now = weight_rows<L::kKeys>(a, c, group, ++b);
      while (now.tiles == 0);
      segment = static_cast<long long>(now.tiles) * now.cost;
    }
  }
}

template <typename T, int kDim, bool kFast>
void launch_weights_dim(const WeightArgs& a, const KvArgs& c, WeightPlan p) {
  const int steps = Tile<T, kDim, kFast>::kSteps;
  const int need = ((a.K + 1) * (a.q_heads / c.heads) + 15) / 16, most = kQueryBytes / (1024 * steps);
  p.chunk = need < most ? need : most;
  // As many workgroups as are resident.  (Half: 77 us for 74, and 102 for 92 at 512 rows; twice: 74 and 110.)
  p.log_ranges = kDim == 256 ? 9 : 10;
  const unsigned lds = p.chunk * (1024 * steps + 16 * 8);
  kv_weights_kernel<T, kDim, kFast><<<1u << p.log_ranges, 64 * kWeightWaves, lds, a.stream>>>(a, c, p);
}

template <typename T>
void launch_weights_type(const WeightArgs& a, const KvArgs& c, const WeightPlan& p) {
  const bool whole = c.page_size % 16 == 0 && c.slot_stride < (1LL << 25);
  if (c.dim <= 64)
    c.dim == 64 && whole ? launch_weights_dim<T, 64, true>(a, c, p) : launch_weights_dim<T, 64, false>(a, c, p);
  else if (c.dim <= 128)
    c.dim == 128 && whole ? launch_weights_dim<T, 128, true>(a, c, p) : launch_weights_dim<T, 128, false>(a, c, p);
  else
    c.dim == 256 && whole ? launch_weights_dim<T, 256, true>(a, c, p) : launch_weights_dim<T, 256, false>(a, c, p);
}

}  // namespace

hipError_t launch_kv_weights(const WeightArgs& a, const KvArgs& c, int dtype) {
  WeightPlan p{};
  p.page_shift = (c.page_size & (c.page_size - 1)) == 0 ? __builtin_ctz(c.page_size) : -1;
  p.scale_log2 = a.scale * kLog2e;
  if (dtype == 0)
    launch_weights_type<float>(a, c, p);
  else if (dtype == 1)
    launch_weights_type<__bf16>(a, c, p);
  else
    launch_weights_type<_Float16>(a, c, p);
  return hipGetLastError();
}

}  // namespace specdec
