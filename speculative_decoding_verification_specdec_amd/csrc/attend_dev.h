// The attention kernel over the paged cache (see paged_attention.hip for the split and the join),
// instantiated for one element type in each of attend_bf16.hip, attend_f16.hip and attend_f32.hip.
#pragma once

#include <hip/hip_runtime.h>

#include "paged_tiles.h"
#include "wave_ops.h"

namespace specdec {

constexpr int kAttendWaves = 4;
constexpr int kAttendThreads = 64 * kAttendWaves;
constexpr int kUnit = 128;          // slots of one unit of work
constexpr int kQueryRegs = 16;      // registers that a wave's query operands may take
constexpr int kAttendGroups = 512;  // workgroups at most (two a CU)

// A segment that lies in several ranges: parts of workgroups w .. w + parts - 1 (parts 0: none).
struct alignas(16) CutSegment {
  int parts, b, seg, first_slot;
};

// How a call is cut.  A segment is one (sequence, kv head, chunk of query rows); its units, and those of
// all segments one after the other, are dealt out evenly to `groups` workgroups in contiguous ranges.
struct AttendPlan {
  int groups;
  int row_waves;        // waves of a workgroup that hold different rows; the others split the slots
  int chunks;           // row chunks of a (sequence, kv head)
  int rows;             // rows of a chunk: 16 * row groups a wave * row_waves
  int tile_rows;        // 16-row groups a wave
  int dim;              // kDim of the kernel
  int page_shift;       // log2(page_size), or -1
  float scale_log2;     // scale * log2(e)
  CutSegment* cut;      // [groups] the segment that a workgroup's range ends in the first part of
  float* part_o;        // [2 groups][rows][dim] unnormalised outputs of cut segments
  float* part_m;        // [2 groups][rows] their maxima (of scores * log2(e))
  float* part_l;        // [2 groups][rows] their sums
};

__device__ __forceinline__ long long units_of(const RoundRows& r) {
  return r.n > 0 ? (static_cast<long long>(r.len) + r.n + kUnit - 1) / kUnit : 0;
}
// Workgroups that get a range: with fewer units than workgroups, one unit each.
__device__ __forceinline__ int active_groups(long long total, int groups) {
  return total < groups ? static_cast<int>(total) : groups;
}
// First unit of workgroup w, and the workgroup that holds a unit.
__device__ __forceinline__ long long range_begin(long long w, long long total, int groups) {
  return w * total / groups;
}
__device__ __forceinline__ int owner_of(long long unit, long long total, int groups) {
  return static_cast<int>(((unit + 1) * groups - 1) / total);
}

// Maximum and sum over the four lanes 16 apart that share a row.
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16, 64));
  return fmaxf(x, __shfl_xor(x, 32, 64));
}
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}

__device__ __forceinline__ long long shfl64(long long x, int src) {
  const int lo = __shfl(static_cast<int>(x), src, 64);
  const int hi = __shfl(static_cast<int>(x >> 32), src, 64);
  return static_cast<long long>(hi) << 32 | static_cast<unsigned>(lo);
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Where a tile's rows lie.  kPaged16: pages are whole 16-slot groups, so each group has one page and a
// wave-uniform address, and lanes add 32-bit offsets that stay the same for the whole walk; otherwise a
// lane looks up one slot and the others get its row by shuffles.
template <bool kPaged16, int kSub>
struct TileRows {
  long long at[kPaged16 ? kSub : 1];
};

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// A page-table entry at a wave-uniform place, by a scalar load.
__device__ __forceinline__ int table_at(const int32_t* table, long long i) {
  typedef const __attribute__((address_space(4))) int32_t* Scalar;
  return *(Scalar)(reinterpret_cast<uintptr_t>(table + i));
}

template <typename T, int kDim, bool kFast, int kRowTiles>
struct AttendWave {
  typedef Tile<T, kDim, kFast> L;
  // Query operands that would take over kQueryRegs registers are read from LDS for each tile instead.
  static constexpr bool kQueryLds = kRowTiles * L::kSteps > kQueryRegs / 4;
  static constexpr int kQueryTiles = kQueryLds ? 1 : kRowTiles;

  const KvArgs& c;
  const T *kpool, *vpool;   // of the kv head
  const int32_t* table;     // of the sequence
  int page_shift, len, total, lane, col, g;
  float scale;
  const u32x4 (*sh_q)[64];  // [row tile * steps][lane]
  u32x4 q[kQueryTiles][L::kSteps];
  u32x4 kf[L::kSub][L::kSteps];
  unsigned vf[L::kRowsV][L::kWords];
  f32x4 o[kRowTiles][L::kOut];
  float m[kRowTiles], l[kRowTiles];
  int limit[kRowTiles];     // last slot that the lane's row sees
  bool bad;

  __device__ __forceinline__ explicit AttendWave(const KvArgs& args) : c(args) {}

  typedef TileRows<kFast, L::kSub> Rows;
  struct Pages {
    int page[kFast ? L::kSub : 1], off[kFast ? L::kSub : 1];
  };

  __device__ __forceinline__ int page_index(int slot) const {
    return page_shift >= 0
               ? slot >> page_shift
               : static_cast<int>(static_cast<unsigned>(slot) / static_cast<unsigned>(c.page_size));
  }

  __device__ __forceinline__ Pages find(int tile) const {
    Pages p;
    if constexpr (kFast) {
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub) {
        // (a group past the last slot takes the last slot's)
        const int slot = min(tile * L::kKeys + 16 * sub, (total - 1) & ~15);
        const int idx = uniform(page_index(slot));
        p.off[sub] = slot - idx * c.page_size;
        p.page[sub] = table_at(table, idx);
      }
    } else {
      const int slot = min(tile * L::kKeys + (lane & (L::kKeys - 1)), total - 1);
      const int idx = page_index(slot);
      p.off[0] = slot - idx * c.page_size;
      p.page[0] = table[idx];
    }
    return p;
  }

  __device__ __forceinline__ Rows resolve(const Pages& p) {
    Rows r;
#pragma unroll
    for (int x = 0; x < (kFast ? L::kSub : 1); ++x) {
      const bool good = static_cast<unsigned>(p.page[x]) < static_cast<unsigned>(c.num_pages);
      bad = bad || !good;
      r.at[x] = (good ? p.page[x] : 0) * c.page_stride + p.off[x] * c.slot_stride;
    }
    return r;
  }

  __device__ __forceinline__ void load_k(const Rows& r) {
#pragma unroll
    for (int sub = 0; sub < L::kSub; ++sub) {
      if constexpr (kFast)
        L::template load_row<true>(kf[sub], kpool + r.at[sub],
                    static_cast<unsigned>(col) * static_cast<unsigned>(c.slot_stride), g, c.dim);
      else
        L::template load_row<true>(kf[sub], kpool + shfl64(r.at[0], 16 * sub + col), 0u, g, c.dim);
    }
  }

  __device__ __forceinline__ void load_v(const Rows& r) {
#pragma unroll
    for (int x = 0; x < L::kRowsV; ++x) {
      if constexpr (kFast)
        L::template load_v<true>(vf[x], vpool + r.at[x / 4],
                  static_cast<unsigned>(4 * g + x % 4) * static_cast<unsigned>(c.slot_stride), col,
                  c.dim);
      else
        L::template load_v<true>(vf[x], vpool + shfl64(r.at[0], L::slot_of(x / 4, x % 4, g)), 0u, col, c.dim);
    }
  }

  __device__ __forceinline__ void scores(f32x4 (&p)[kRowTiles][L::kSub]) const {
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      u32x4 qt[L::kSteps];
#pragma unroll
      for (int e = 0; e < L::kSteps; ++e)
        qt[e] = kQueryLds ? sh_q[t * L::kSteps + e][lane] : q[kQueryLds ? 0 : t][e];
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub) {
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < L::kSteps; ++e) x = mma16(kf[sub][e], qt[e], x, T{});
        p[t][sub] = x;
      }
    }
  }

  // Scores to probabilities relative to the running maximum (kept in units of log2), which moves on.
  __device__ __forceinline__ void softmax(f32x4 (&p)[kRowTiles][L::kSub]) {
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      float top = p[t][0][0];
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub)
#pragma unroll
        for (int x = 0; x < 4; ++x) top = fmaxf(top, p[t][sub][x]);
      top = fmaxf(m[t], row_max(top) * scale);
      if (__any(top > m[t])) {
        // (no slot yet: m = -inf, and everything that it would scale is 0)
        const float old = m[t] == -INFINITY ? 0.f : exp2_hw(m[t] - top);
        l[t] *= old;
#pragma unroll
        for (int x = 0; x < L::kOut; ++x) o[t][x] *= old;
        m[t] = top;
      }
      const float base = m[t] == -INFINITY ? 0.f : m[t];
      float sum = 0.f;
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          p[t][sub][x] = exp2_hw(fmaf(p[t][sub][x], scale, -base));
          sum += p[t][sub][x];
        }
      l[t] += sum;
    }
  }

  // acc + V^T P^T for output group x of one row tile; p the probabilities by (sub, r), packed for the
  // 16-bit types.  `keep`, where given, has the bits of the operands' slots that count.
  template <bool kMasked>
  __device__ __forceinline__ f32x4 product(const f32x4 (&p)[L::kSub], const u32x4& packed, int x,
                                           const u32x4& keep, f32x4 acc) const {
    if constexpr (L::kHalf) {
      unsigned select = x & 1 ? 0x07060302u : 0x05040100u;
      if (kMasked) asm volatile("" : "+s"(select));  // (keeps the turned block out of registers)
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = __builtin_amdgcn_perm(vf[2 * i + 1][x / 2], vf[2 * i][x / 2], select);
      return kMasked ? mma16(v & keep, packed & keep, acc, T{}) : mma16(v, packed, acc, T{});
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const unsigned pr = __float_as_uint(p[0][r]);
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(
            __uint_as_float(kMasked ? vf[r][x] & keep[r] : vf[r][x]),
            __uint_as_float(kMasked ? pr & keep[r] : pr), acc, 0, 0, 0);
      }
      return acc;
    }
  }

  // Probabilities of 16-bit types enter the product rounded to that type (half a step, 2^-8 or 2^-11
  // of each: as much as the rounding of the result itself); the row's sum l is of the unrounded ones.
  static __device__ __forceinline__ u32x4 packed(const f32x4 (&p)[L::kSub]) {
    u32x4 w = {0, 0, 0, 0};
    if constexpr (L::kHalf) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        w[2 * s] = pack2<T>(p[s][0], p[s][1]);
        w[2 * s + 1] = pack2<T>(p[s][2], p[s][3]);
      }
    }
    return w;
  }

  __device__ __forceinline__ void products(const f32x4 (&p)[kRowTiles][L::kSub]) {
    u32x4 pk[kRowTiles];
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) pk[t] = packed(p[t]);
#pragma unroll
    for (int x = 0; x < L::kOut; ++x)
#pragma unroll
      for (int t = 0; t < kRowTiles; ++t) o[t][x] = product<false>(p[t], pk[t], x, u32x4{}, o[t][x]);
  }

  static __device__ __forceinline__ bool word_finite(unsigned w) {
    if constexpr (sizeof(T) == 4) return (w & 0x7f800000u) != 0x7f800000u;
    constexpr unsigned e = __is_same(T, __bf16) ? 0x7f80u : 0x7c00u;
    return (w & e) != e && (w >> 16 & e) != e;
  }

  // A tile with slots that not every row sees.  A value that is not finite must not reach a row that does
  // not see its slot, not even as 0 * value: a tile with such values (stale slots past the last one
  // included) is done in several products, first of the slots that every row sees, then slot by slot,
  // each added only to the rows that see it.
  __device__ __forceinline__ void products_edge(const f32x4 (&p)[kRowTiles][L::kSub], int first) {
    bool finite = true;
#pragma unroll
    for (int x = 0; x < L::kRowsV; ++x)
#pragma unroll
      for (int y = 0; y < L::kWords; ++y) finite = finite && word_finite(vf[x][y]);
    const bool at_once = !__any(!finite);
    u32x4 pk[kRowTiles];
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) pk[t] = packed(p[t]);
    const int last = at_once ? len : min(first + L::kKeys, total) - 1;
    for (int only = len; only <= last; only = max(only + 1, first)) {
      u32x4 keep;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        unsigned bits = 0;
#pragma unroll
        for (int x = L::kHalf ? 2 * i : i; x <= (L::kHalf ? 2 * i + 1 : i); ++x) {
          const int slot = first + L::slot_of(x / 4, x % 4, g);
          const bool in = at_once || (only == len ? slot <= len : slot == only);
          bits |= in ? (L::kHalf ? 0xffffu << (x % 2 * 16) : 0xffffffffu) : 0u;
        }
        keep[i] = bits;
      }
#pragma unroll
      for (int t = 0; t < kRowTiles; ++t) {
        const bool sees = at_once || only <= limit[t];
#pragma unroll
        for (int x = 0; x < L::kOut; ++x) {
          const f32x4 add = product<true>(p[t], pk[t], x, keep, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int r = 0; r < 4; ++r) o[t][x][r] += sees ? add[r] : 0.f;
        }
      }
    }
  }

  // The wave's tiles first, first + step, .. before end.  The next tile's K is loaded while this one's
  // scores become probabilities, its V after the products, and its pages are looked up one tile earlier.
  __device__ __forceinline__ void walk(int tile, int end, int step) {
    if (tile >= end) return;
    Rows rows = resolve(find(tile));
    load_k(rows);
    load_v(rows);
    Pages next = find(min(tile + step, end - 1));
    const int whole_end = min(end, (len + 1) / L::kKeys);  // tiles of which every row sees every slot
    f32x4 p[kRowTiles][L::kSub];
    for (; tile < whole_end; tile += step) {
      scores(p);
      __builtin_amdgcn_sched_barrier(0);
      rows = resolve(next);  // (past the last tile: that one again)
      load_k(rows);
      next = find(min(tile + 2 * step, end - 1));
      __builtin_amdgcn_sched_barrier(0);
      softmax(p);
      products(p);
      __builtin_amdgcn_sched_barrier(0);
      load_v(rows);
      __builtin_amdgcn_sched_barrier(0);
    }
    for (; tile < end; tile += step) {
      const int first = tile * L::kKeys;
      scores(p);
      __builtin_amdgcn_sched_barrier(0);
      rows = resolve(next);
      load_k(rows);
      next = find(min(tile + 2 * step, end - 1));
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
        for (int sub = 0; sub < L::kSub; ++sub)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (first + L::slot_of(sub, x, g) > limit[t]) p[t][sub][x] = -INFINITY;
      softmax(p);
      products_edge(p, first);
      __builtin_amdgcn_sched_barrier(0);
      load_v(rows);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// Four elements from d on of an output row, and with the first its lse; a row past the last token is 0.
template <typename T>
__device__ __forceinline__ void write_row(const AttendArgs& a, const KvArgs& c, long long row, bool used,
                                          int d, f32x4 sum, float top, float total) {
  const float inv = 1.f / total;
  if (!used) sum = f32x4{0.f, 0.f, 0.f, 0.f};
  else sum *= inv;
  T* out = static_cast<T*>(a.out) + row * c.dim + d;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<u32x2*>(out) = u32x2{pack2<T>(sum[0], sum[1]), pack2<T>(sum[2], sum[3])};
  else
    *reinterpret_cast<f32x4*>(out) = sum;
  if (d == 0 && a.lse)
    a.lse[row] = !used ? -INFINITY : top == -INFINITY ? __builtin_nanf("") : top * kLn2 + logf(total);
}

// Adds up the parts of a cut segment: workgroup (w, y) the rows 16 y .. of the one whose first part
// workgroup w of the split holds.  dim / 4 lanes share a row, so a wave loads 256 / dim parts' worth at once,
// four of them ahead.
template <typename T, int kDim>
__global__ __launch_bounds__(kAttendThreads) void attend_join_kernel(AttendArgs a, KvArgs c,
                                                                     AttendPlan plan) {
  constexpr int kLanes = kDim / 4;                    // lanes of a row
  constexpr int kRowsOnce = kAttendThreads / kLanes;  // rows at once
  const int w = blockIdx.x;
  const CutSegment cut = plan.cut[w];
  if (cut.parts == 0) return;
  const RoundRows r = round_rows(c, a.num_draft, a.kv_len, cut.b, a.K);
  const int group = a.q_heads / c.heads;
  const int h = cut.seg / plan.chunks, chunk = cut.seg - h * plan.chunks;
  const int d = threadIdx.x % kLanes * 4;
  const int end = min(plan.rows, (a.K + 1) * group - chunk * plan.rows);
  for (int local = blockIdx.y * kRowsOnce + threadIdx.x / kLanes; local < end; local += gridDim.y * kRowsOnce) {
    const int qrow = chunk * plan.rows + local, i = qrow / group;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float top = -INFINITY, sum = 0.f;
    if (i < r.n) {
      constexpr int kAhead = 8;
      for (int p = 0; p < cut.parts; p += kAhead) {
        f32x4 x[kAhead];
        float m[kAhead], l[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          const int q = min(p + e, cut.parts - 1);
          const long long at = (2LL * (w + q) + (q == 0 ? cut.first_slot : 0)) * plan.rows + local;
          x[e] = *reinterpret_cast<const f32x4*>(plan.part_o + at * kDim + d);
          m[e] = plan.part_m[at];
          l[e] = plan.part_l[at];
        }
        float now = top;
#pragma unroll
        for (int e = 0; e < kAhead; ++e) now = fmaxf(now, m[e]);
        const float base = now == -INFINITY ? 0.f : now;
        const float old = exp2_hw(top - base);
        o *= old;
        sum *= old;
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          if (p + e >= cut.parts) break;
          const float f = exp2_hw(m[e] - base);
          o += x[e] * f;
          sum += l[e] * f;
        }
        top = now;
      }
    }
    if (d < c.dim)
      write_row<T>(a, c, (static_cast<long long>(cut.b) * (a.K + 1) + i) * a.q_heads + h * group + qrow - i * group,
                   i < r.n, d, o, top, sum);
  }
}

// kFast: head_dim is kDim, pages are whole groups of 16 slots and 16 slots lie within 2^32 bytes.
template <typename T, int kDim, bool kFast, int kRowTiles, int kOccupancy>
__global__ __launch_bounds__(kAttendThreads, kOccupancy) void attend_split_kernel(AttendArgs a, KvArgs c,
                                                                                  AttendPlan plan) {
  typedef Tile<T, kDim, kFast> L;
  typedef AttendWave<T, kDim, kFast, kRowTiles> Wave;
  constexpr int kPad = kDim + 4;
  constexpr int kTilesUnit = kUnit / L::kKeys;
  __shared__ float sh_o[kAttendWaves][16][kPad];
  __shared__ float sh_m[kAttendWaves][kRowTiles * 16], sh_l[kAttendWaves][kRowTiles * 16];
  __shared__ float sh_top[kAttendWaves][kRowTiles * 16], sh_sum[kAttendWaves][kRowTiles * 16];
  __shared__ u32x4 sh_q[Wave::kQueryLds ? kAttendWaves : 1][Wave::kQueryLds ? kRowTiles * L::kSteps : 1][64];
  __shared__ long long sh_scan[kAttendWaves], sh_before;
  __shared__ int sh_b;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int group = a.q_heads / c.heads;
  const int segs = c.heads * plan.chunks;  // segments of a sequence
  // Units before each sequence: every thread sums a run of sequences, then a scan over the threads.
  const int per = (a.B + kAttendThreads - 1) / kAttendThreads;
  const int run0 = min(a.B, tid * per), run1 = min(a.B, run0 + per);
  long long mine = 0;
  for (int b = run0; b < run1; ++b) mine += units_of(round_rows(c, a.num_draft, a.kv_len, b, a.K));
  long long upto = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const long long y = shfl64(upto, max(lane - off, 0));
    if (lane >= off) upto += y;
  }
  if (lane == 63) sh_scan[wave] = upto;
  __syncthreads();
  long long all = 0;
  for (int x = 0; x < kAttendWaves; ++x) {
    if (x < wave) upto += sh_scan[x];
    all += sh_scan[x];
  }
  long long before = upto - mine;
  const long long total_units = all * segs;
  const int groups = active_groups(total_units, plan.groups);
  // Neighbouring ranges go to workgroups of one XCD (workgroups are dealt to the 8 XCDs in turn), so
  // that row chunks of the same slots meet in its L2; too few units for that go round all XCDs.
  const int w = groups == plan.groups
                    ? static_cast<int>(blockIdx.x % 8 * (plan.groups / 8) + blockIdx.x / 8)
                    : static_cast<int>(blockIdx.x);
  // Sequences without units are invalid: their rows are NaN.
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const RoundRows r = round_rows(c, a.num_draft, a.kv_len, b, a.K);
    if (r.n > 0) continue;
    const long long row = static_cast<long long>(b) * (a.K + 1) * a.q_heads;
    const long long bad = static_cast<long long>(r.rows) * a.q_heads;
    const long long rows = (a.K + 1LL) * a.q_heads;
    T* out = static_cast<T*>(a.out) + row * c.dim;
    for (long long x = tid; x < rows * c.dim; x += kAttendThreads)
      out[x] = from_float<T>(x < bad * c.dim ? __builtin_nanf("") : 0.f);
    for (long long x = tid; a.lse && x < rows; x += kAttendThreads)
      a.lse[row + x] = x < bad ? __builtin_nanf("") : -INFINITY;
  }
  if (tid == 0) plan.cut[w].parts = 0;
  if (w >= groups) return;
  const long long begin = range_begin(w, total_units, groups);
  const long long end = range_begin(w + 1, total_units, groups);
  if (mine > 0 && before * segs <= begin && begin < (before + mine) * segs) {
    int b = run0;
    for (;; ++b) {
      const long long u = units_of(round_rows(c, a.num_draft, a.kv_len, b, a.K));
      if (begin < (before + u) * segs) break;
      before += u;
    }
    sh_b = b;
    sh_before = before;
  }
  __syncthreads();
  int b = uniform(sh_b);
  RoundRows r = round_rows(c, a.num_draft, a.kv_len, b, a.K);
  // From here on 32 bits do: a sequence has under 2^24 units, and a range that starts in one of its
  // segments is cut at the segment's end piece by piece.
  int units = static_cast<int>(units_of(r));
  const long long inside = begin - sh_before * segs;
  int seg = uniform(static_cast<int>(inside / units));
  int at = uniform(static_cast<int>(inside - static_cast<long long>(seg) * units));
  long long left = end - begin;
  int slot_of_part = 0;

  const int rw = wave % plan.row_waves, kw = wave / plan.row_waves;
  const int key_waves = kAttendWaves / plan.row_waves;
  Wave s(c);
  s.page_shift = plan.page_shift;
  s.lane = lane;
  s.col = col;
  s.g = g;
  s.scale = plan.scale_log2;
  s.sh_q = sh_q[Wave::kQueryLds ? wave : 0];

  while (left > 0) {
    // One piece: units [at, stop) of segment (b, h, chunk).
    const int len = uniform(r.len), n = uniform(r.n);
    const int stop = uniform(static_cast<int>(min(static_cast<long long>(units), at + left)));
    const int h = seg / plan.chunks, chunk = seg - h * plan.chunks;
    const int row0 = chunk * plan.rows + rw * 16 * kRowTiles;
    s.len = len;
    s.total = len + n;
    s.kpool = reinterpret_cast<const T*>(c.k) + h * c.head_stride;
    s.vpool = reinterpret_cast<const T*>(c.v) + h * c.head_stride;
    s.table = c.table + static_cast<long long>(b) * c.max_pages;
    s.bad = false;
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      const int qrow = row0 + 16 * t + col;
      const int i = qrow / group;
      s.m[t] = -INFINITY;
      s.l[t] = 0.f;
      s.limit[t] = i < n ? len + i : -1;
#pragma unroll
      for (int x = 0; x < L::kOut; ++x) s.o[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
      u32x4 qt[L::kSteps];
#pragma unroll
      for (int x = 0; x < L::kSteps; ++x) qt[x] = u32x4{0, 0, 0, 0};
      if (i < n)
        L::template load_row<false>(qt,
                    static_cast<const T*>(a.q) + (static_cast<long long>(b) * (a.K + 1) + i) * a.q_stride +
                        static_cast<long long>(h * group + qrow - i * group) * c.dim,
                    0u, g, c.dim);
#pragma unroll
      for (int x = 0; x < L::kSteps; ++x) {
        if constexpr (Wave::kQueryLds)
          sh_q[wave][t * L::kSteps + x][lane] = qt[x];  // (read back by this lane alone)
        else
          s.q[t][x] = qt[x];
      }
    }
    if (row0 < n * group)  // (a wave without rows has nothing to read)
      s.walk(at * kTilesUnit + kw, min(stop * kTilesUnit, (len + n + L::kKeys - 1) / L::kKeys),
             key_waves);

    // Join the waves that split the slots, 16 rows a round, and write the segment's rows or, if another
    // workgroup holds the rest of it, this piece's part.
    const bool whole = at == 0 && stop == units;
    const bool bad = __any(s.bad);
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      s.l[t] = row_sum(s.l[t]);
      if (bad) {  // a page id outside the pool: the rows' sums are NaN, whatever else they hold
        s.l[t] = __builtin_nanf("");
        if (s.m[t] == -INFINITY) s.m[t] = 0.f;
      }
      if (g == 0) {
        sh_m[wave][16 * t + col] = s.m[t];
        sh_l[wave][16 * t + col] = s.l[t];
      }
    }
    __syncthreads();
    const long long part = 2LL * w + slot_of_part;
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      float top = -INFINITY;
      for (int x = 0; x < key_waves; ++x) top = fmaxf(top, sh_m[x * plan.row_waves + rw][16 * t + col]);
      const float base = top == -INFINITY ? 0.f : top;
      if (kw == 0 && g == 0) {
        float sum = 0.f;
        for (int x = 0; x < key_waves; ++x)
          sum += sh_l[x * plan.row_waves + rw][16 * t + col] *
                 exp2_hw(sh_m[x * plan.row_waves + rw][16 * t + col] - base);
        sh_top[rw][16 * t + col] = top;
        sh_sum[rw][16 * t + col] = sum;
      }
      const float f = exp2_hw(s.m[t] - base);
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < L::kOut; y += 4)
          *reinterpret_cast<f32x4*>(&sh_o[wave][col][L::kChunk * (4 * g + x) + y]) =
              f32x4{s.o[t][y][x], s.o[t][y + 1][x], s.o[t][y + 2][x], s.o[t][y + 3][x]} * f;
      __syncthreads();
      constexpr int kVecs = 16 * kDim / 4;
      for (int idx = tid; idx < plan.row_waves * kVecs; idx += kAttendThreads) {
        const int rwi = idx / kVecs, rr = idx % kVecs / (kDim / 4), d = idx % (kDim / 4) * 4;
        f32x4 sum = *reinterpret_cast<f32x4*>(&sh_o[rwi][rr][d]);
        for (int x = 1; x < key_waves; ++x)
          sum += *reinterpret_cast<f32x4*>(&sh_o[x * plan.row_waves + rwi][rr][d]);
        const int local = rwi * 16 * kRowTiles + 16 * t + rr;
        const float rtop = sh_top[rwi][16 * t + rr], rsum = sh_sum[rwi][16 * t + rr];
        if (whole) {
          const int qrow = chunk * plan.rows + local, i = qrow / group;
          if (i <= a.K && d < c.dim)
            write_row<T>(a, c, (static_cast<long long>(b) * (a.K + 1) + i) * a.q_heads + h * group + qrow - i * group,
                         i < n, d, sum, rtop, rsum);
        } else if (chunk * plan.rows + local < n * group) {
          const long long at_row = part * plan.rows + local;
          *reinterpret_cast<f32x4*>(plan.part_o + at_row * kDim + d) = sum;
          if (d == 0) {
            plan.part_m[at_row] = rtop;
            plan.part_l[at_row] = rsum;
          }
        }
      }
      __syncthreads();
    }
    if (at == 0 && stop < units && tid == 0) {
      const int last = owner_of(begin + (end - begin - left) + units - 1, total_units, groups);
      plan.cut[w] = CutSegment{last - w + 1, b, seg, slot_of_part};
    }
    slot_of_part = 1;
    left -= stop - at;
    at = 0;
    if (left > 0 && ++seg == segs) {
      seg = 0;
      do {
        r = round_rows(c, a.num_draft, a.kv_len, ++b, a.K);
        units = uniform(static_cast<int>(units_of(r)));
      } while (units == 0);
    }
  }
}

template <typename T, int kDim>
void launch_join(const AttendArgs& a, const KvArgs& c, const AttendPlan& p) {
  constexpr int kRowsOnce = kAttendThreads / (kDim / 4);
  const int rows = p.rows < (a.K + 1) * (a.q_heads / c.heads) ? p.rows : (a.K + 1) * (a.q_heads / c.heads);
  const dim3 grid(p.groups, (rows + kRowsOnce - 1) / kRowsOnce);
  attend_join_kernel<T, kDim><<<grid, kAttendThreads, 0, a.stream>>>(a, c, p);
}

template <typename T, int kDim, bool kFast>
void launch_attend_dim(const AttendArgs& a, const KvArgs& c, const AttendPlan& p) {
  const dim3 grid(p.groups), block(kAttendThreads);
  if (p.tile_rows == 1)
    attend_split_kernel<T, kDim, kFast, 1, kDim == 256 ? 1 : 2><<<grid, block, 0, a.stream>>>(a, c, p);
  else if constexpr (kDim < 256) {
    if (p.tile_rows == 2)
      attend_split_kernel<T, kDim, kFast, 2, kDim == 128 && sizeof(T) == 4 ? 1 : 2><<<grid, block, 0, a.stream>>>(a, c, p);
    else if constexpr (kDim == 64 || sizeof(T) == 2)
      attend_split_kernel<T, kDim, kFast, 4, 1><<<grid, block, 0, a.stream>>>(a, c, p);
  }
  launch_join<T, kDim>(a, c, p);
}

template <typename T>
void launch_attend_type(const AttendArgs& a, const KvArgs& c, const AttendPlan& p) {
  const bool fast = c.dim == p.dim && c.page_size % 16 == 0 && c.slot_stride < (1LL << 25);
  if (p.dim == 64)
    fast ? launch_attend_dim<T, 64, true>(a, c, p) : launch_attend_dim<T, 64, false>(a, c, p);
  else if (p.dim == 128)
    fast ? launch_attend_dim<T, 128, true>(a, c, p) : launch_attend_dim<T, 128, false>(a, c, p);
  else
    fast ? launch_attend_dim<T, 256, true>(a, c, p) : launch_attend_dim<T, 256, false>(a, c, p);
}

void launch_attend_bf16(const AttendArgs& a, const KvArgs& c, const AttendPlan& p);
void launch_attend_f16(const AttendArgs& a, const KvArgs& c, const AttendPlan& p);
void launch_attend_f32(const AttendArgs& a, const KvArgs& c, const AttendPlan& p);

}  // namespace specdec
