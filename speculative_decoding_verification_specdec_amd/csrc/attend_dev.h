// The attention kernels over the paged cache (paged_attention.cpp makes the plan they follow),
// instantiated for one element type in each of attend_bf16.hip, attend_f16.hip and attend_f32.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "attend_plan.h"
#include "paged_tiles.h"
#include "wave_ops.h"

namespace specdec {

constexpr int kJoinThreads = 256;
// The kernel for many rows leaves segments of so many tiles whole, with the workgroup that has their first tile: a part
// of 64 or 128 rows costs as much as several tiles.  (64 x 100-300 slots, 64 rows on 8 heads: 35 us, 41 with all of
// them cut; 14 x 1-9 slots, 512 rows on 8 heads, f32: 58 and 88; 64 x 500-4000 slots, 48 rows: 144 and 143, but 152
// with segments of up to 32 tiles whole.)
constexpr int kWholeTiles = 16;

// Row chunks of a sequence with n new tokens; tiles of its slots; tiles of all its segments (none if it
// is invalid).
__device__ __forceinline__ int chunks_of(int n, int group, int rows) { return (n * group + rows - 1) / rows; }
template <int kKeys>
__device__ __forceinline__ int tiles_of(int len, int n) {
  return (len + n - 1) / kKeys + 1;
}
template <int kKeys>
__device__ __forceinline__ long long work_of(const RoundRows& r, int heads, int group, int rows) {
  return r.n > 0 ? static_cast<long long>(tiles_of<kKeys>(r.len, r.n)) * (heads * chunks_of(r.n, group, rows)) : 0;
}
// First tile of range w, and the range that holds a tile.  Fewer tiles than ranges: one tile each.
__device__ __forceinline__ long long range_begin(long long w, long long total, int log_ranges) {
  return total >> log_ranges == 0 ? min(w, total) : w * total >> log_ranges;
}
__device__ __forceinline__ int range_of(long long tile, long long total, int log_ranges) {
  if (total >> log_ranges == 0) return static_cast<int>(tile);
  // The w with w total <= (tile + 1) 2^log - 1 < (w + 1) total, by a quotient in f64 (both under 2^53)
  // and a correction by one.
  const long long n = ((tile + 1) << log_ranges) - 1;
  long long q = static_cast<long long>(static_cast<double>(n) / static_cast<double>(total));
  if (q * total > n) --q;
  if ((q + 1) * total <= n) ++q;
  return static_cast<int>(q);
}

// Maximum over the four lanes 16 apart that share a row (like row_sum).
__device__ __forceinline__ float row_max(float x) {
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const unsigned v = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
// Where a tile's rows lie.  kPaged16: pages are whole 16-slot groups, so each group has one page and a
// wave-uniform address, and lanes add 32-bit offsets that stay the same for the whole walk; otherwise a
// lane looks up one slot and the others get its row by shuffles.
template <bool kPaged16, int kSub>
struct TileRows {
  long long at[kPaged16 ? kSub : 1];
};

// One piece of a wave's range: tiles [first, end) of a segment (b, seg = kv head * chunks + chunk) of `tiles`;
// none: end 0.
template <typename T>
struct AttendPiece {
  int b, seg, len, n, chunks, tiles, first, end;
  const T *kpool, *vpool;     // of the kv head
  const int32_t* table;       // of the sequence
};

template <typename T, int kDim, bool kFast, int kRowTiles, bool kQueryLds, bool kShared = false>
struct AttendWave {
  typedef Tile<T, kDim, kFast> L;
  // kQueryLds: the query operands are read from LDS for each tile instead of staying in registers.
  static constexpr int kQueryTiles = kQueryLds ? 1 : kRowTiles;
  // kShared: the operands of K and V are read from the workgroup's tile in LDS step by step; of V two words of each
  // row at a time, which make kPair groups of the output.
  static constexpr int kPairs = L::kWords / 2, kPair = L::kOut / kPairs;

  const KvArgs& c;
  int page_shift, lane, col, g;
  float scale;
  u32x4 (*sh_q)[64];        // [row tile * steps][lane]
  u32x4 q[kQueryTiles][L::kSteps];
  u32x4 kf[kShared ? 1 : L::kSub][kShared ? 1 : L::kSteps];
  unsigned vf[kShared ? 1 : L::kRowsV][kShared ? 1 : L::kWords];
  const u32x4 (*sh_k)[64];  // [sub * steps][lane]
  const u32x2 (*sh_v)[64];  // [pair * rows][lane]
  u32x2 vp[kShared ? L::kRowsV : 1];
  f32x4 o[kRowTiles][L::kOut];
  float m[kRowTiles], l[kRowTiles];
  int limit[kRowTiles];     // last slot that the lane's row sees
  bool bad, bad_next;       // a page id outside the pool, in this piece and in the next one's first tile

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

  __device__ __forceinline__ Pages find(const AttendPiece<T>& piece, int tile) const {
    Pages p;
    const int last = piece.len + piece.n - 1;
    if constexpr (kFast) {
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub) {
        // (a group past the last slot takes the last slot's)
        const int slot = min(tile * L::kKeys + 16 * sub, last & ~15);
        const int idx = uniform(page_index(slot));
        p.off[sub] = slot - idx * c.page_size;
        p.page[sub] = table_at(piece.table, idx);
      }
    } else {
      const int slot = min(tile * L::kKeys + (lane & (L::kKeys - 1)), last);
      const int idx = page_index(slot);
      p.off[0] = slot - idx * c.page_size;
      p.page[0] = piece.table[idx];
    }
    return p;
  }

  __device__ __forceinline__ Rows resolve(const Pages& p, bool& wrong) {
    Rows r;
#pragma unroll
    for (int x = 0; x < (kFast ? L::kSub : 1); ++x) {
      const bool good = static_cast<unsigned>(p.page[x]) < static_cast<unsigned>(c.num_pages);
      wrong = wrong || !good;
      r.at[x] = (good ? p.page[x] : 0) * c.page_stride + p.off[x] * c.slot_stride;
    }
    return r;
  }

  __device__ __forceinline__ void load_k(const T* kpool, const Rows& r) {
#pragma unroll
    for (int sub = 0; sub < L::kSub; ++sub) {
      if constexpr (kFast)
        L::template load_row<true>(kf[sub], scalar_base(kpool + r.at[sub]),
                    static_cast<unsigned>(col) * static_cast<unsigned>(c.slot_stride), g, c.dim);
      else
        L::template load_row<true>(kf[sub], (GlobalBytes)(kpool + shfl64(r.at[0], 16 * sub + col)), 0u, g, c.dim);
    }
  }

  __device__ __forceinline__ void load_v(const T* vpool, const Rows& r) {
#pragma unroll
    for (int x = 0; x < L::kRowsV; ++x) {
      if constexpr (kFast)
        L::template load_v<true>(vf[x], scalar_base(vpool + r.at[x / 4]),
                  static_cast<unsigned>(4 * g + x % 4) * static_cast<unsigned>(c.slot_stride), col,
                  c.dim);
      else
        L::template load_v<true>(vf[x], (GlobalBytes)(vpool + shfl64(r.at[0], L::slot_of(x / 4, x % 4, g))), 0u, col,
                                 c.dim);
    }
  }

  // All row tiles' and slot groups' chains side by side: a product waits for the one before it in its chain.
  __device__ __forceinline__ void scores(f32x4 (&p)[kRowTiles][L::kSub]) const {
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub) p[t][sub] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < L::kSteps; ++e)
#pragma unroll
      for (int t = 0; t < kRowTiles; ++t) {
        const u32x4 qt = kQueryLds ? sh_q[t * L::kSteps + e][lane] : q[kQueryLds ? 0 : t][e];
#pragma unroll
        for (int sub = 0; sub < L::kSub; ++sub)
          p[t][sub] = mma16(kShared ? sh_k[sub * L::kSteps + e][lane] : kf[kShared ? 0 : sub][kShared ? 0 : e], qt,
                            p[t][sub], T{});
        // (few steps' operands at a time)
        if ((kQueryLds || (kShared && e % 2 == 1)) && t == kRowTiles - 1) __builtin_amdgcn_sched_barrier(0);
      }
  }

  // Scores to probabilities relative to a running base (in units of log2) that follows the row's maximum:
  // it moves up when a score passes it by more than kSlack, so that probabilities stay under 2^kSlack
  // (float16 holds 2^15) and the outputs are rescaled a few times a row, not with each new maximum.
  __device__ __forceinline__ void softmax(f32x4 (&p)[kRowTiles][L::kSub]) {
    constexpr float kSlack = 8.f;
    float top[kRowTiles];
    bool up = false;
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      top[t] = p[t][0][0];
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub)
#pragma unroll
        for (int x = 0; x < 4; ++x) top[t] = fmaxf(top[t], p[t][sub][x]);
      top[t] = row_max(top[t]) * scale;
      up = up || top[t] > m[t] + kSlack;
    }
    if (__any(up)) {
#pragma unroll
      for (int t = 0; t < kRowTiles; ++t) {
        const float now = fmaxf(m[t], top[t]);
        // (no slot yet: m = -inf, and everything that it would scale is 0)
        const float old = m[t] == -INFINITY ? 0.f : exp2_hw(m[t] - now);
        l[t] *= old;
#pragma unroll
        for (int x = 0; x < L::kOut; ++x) o[t][x] *= old;
        m[t] = now;
      }
    }
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      const float base = m[t] == -INFINITY ? 0.f : m[t];
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub)
#pragma unroll
        for (int x = 0; x < 4; ++x) p[t][sub][x] = exp2_hw(fmaf(p[t][sub][x], scale, -base));
      // (added in pairs: a shorter chain, and the order is fixed)
      f32x4 sum = p[t][0];
      if constexpr (L::kSub == 2) sum += p[t][1];
      l[t] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
  }

  // The words of V for output groups kPair * pair on; a word of a row.
  __device__ __forceinline__ void fetch_pair(int pair) {
    if constexpr (kShared)
#pragma unroll
      for (int row = 0; row < L::kRowsV; ++row) vp[row] = sh_v[pair * L::kRowsV + row][lane];
  }
  __device__ __forceinline__ unsigned word(int row, int w) const {
    if constexpr (kShared)
      return vp[row][w & 1];
    else
      return vf[row][w];
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
        v[i] = __builtin_amdgcn_perm(word(2 * i + 1, x / 2), word(2 * i, x / 2), select);
      return kMasked ? mma16(v & keep, packed & keep, acc, T{}) : mma16(v, packed, acc, T{});
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const unsigned pr = __float_as_uint(p[0][r]);
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(
            __uint_as_float(kMasked ? word(r, x) & keep[r] : word(r, x)),
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
    for (int x = 0; x < L::kOut; ++x) {
      if (x % kPair == 0) fetch_pair(x / kPair);
      if (kShared && x % kPair == 0) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < kRowTiles; ++t) o[t][x] = product<false>(p[t], pk[t], x, u32x4{}, o[t][x]);
    }
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
  __device__ __forceinline__ void products_edge(const f32x4 (&p)[kRowTiles][L::kSub], int first, int len, int total) {
    bool finite = true;
#pragma unroll
    for (int pair = 0; pair < kPairs; ++pair) {
      fetch_pair(pair);
      if (kShared) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int x = 0; x < L::kRowsV; ++x)
        finite = finite && word_finite(word(x, 2 * pair)) && word_finite(word(x, 2 * pair + 1));
    }
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
          if (x % kPair == 0) fetch_pair(x / kPair);
          if (kShared) __builtin_amdgcn_sched_barrier(0);
          const f32x4 add = product<true>(p[t], pk[t], x, keep, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int r = 0; r < 4; ++r) o[t][x][r] += sees ? add[r] : 0.f;
        }
      }
    }
  }

  // The next tile: of this piece, or past its end the next piece's first one (or none: the last again).
  static __device__ __forceinline__ bool stays(const AttendPiece<T>& now, const AttendPiece<T>& next, int t) {
    return t < now.end || next.end == 0;
  }
  __device__ __forceinline__ Pages ahead(const AttendPiece<T>& now, const AttendPiece<T>& next, int t) const {
    if (stays(now, next, t)) return find(now, min(t, now.end - 1));
    return find(next, next.first);
  }

  // Loads K of the tile after `tile`, looks up the pages of the one after that.
  __device__ __forceinline__ Rows next_k(const AttendPiece<T>& now, const AttendPiece<T>& next, int tile,
                                         Pages& pages) {
    const bool inside = stays(now, next, tile + 1);
    bool wrong = false;
    const Rows rows = resolve(pages, wrong);
    bad = bad || (wrong && inside);
    bad_next = bad_next || (wrong && !inside);
    const T* pool = now.kpool;
    if (!inside) pool = next.kpool;
    load_k(pool, rows);
    pages = ahead(now, next, tile + 2);
    return rows;
  }
  __device__ __forceinline__ void next_v(const AttendPiece<T>& now, const AttendPiece<T>& next, int tile,
                                         const Rows& rows) {
    const T* pool = now.vpool;
    if (!stays(now, next, tile + 1)) pool = next.vpool;
    load_v(pool, rows);
  }

  // The first tile of a piece before which there is no other one to load it ahead in.
  __device__ __forceinline__ void enter(const AttendPiece<T>& piece) {
    const Rows rows = resolve(find(piece, piece.first), bad);
    load_k(piece.kpool, rows);
    load_v(piece.vpool, rows);
  }

  // One row tile's rows of q of a piece.
  __device__ __forceinline__ void load_q(u32x4 (&qt)[L::kSteps], const AttendArgs& a, const AttendPlan& plan,
                                         int group, const AttendPiece<T>& p, int t) const {
    const int h = p.seg / p.chunks, chunk = p.seg - h * p.chunks;
    const int qrow = chunk * plan.rows + 16 * t + col, i = qrow / group;
#pragma unroll
    for (int x = 0; x < L::kSteps; ++x) qt[x] = u32x4{0, 0, 0, 0};
    if (i < p.n)
      L::template load_row<false>(
          qt,
          (GlobalBytes)(static_cast<const T*>(a.q) +
                        (static_cast<long long>(p.b) * (a.K + 1) + i) * a.q_stride +
                        static_cast<long long>(h * group + qrow - i * group) * c.dim),
          0u, g, c.dim);
  }

  // No slot of a row tile's rows seen yet; the lane's row sees those up to `upto`.
  __device__ __forceinline__ void clear(int t, int upto) {
    m[t] = -INFINITY;
    l[t] = 0.f;
    limit[t] = upto;
#pragma unroll
    for (int x = 0; x < L::kOut; ++x) o[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  __device__ __forceinline__ void mask(f32x4 (&p)[kRowTiles][L::kSub], int first) const {
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (first + L::slot_of(sub, x, g) > limit[t]) p[t][sub][x] = -INFINITY;
  }

  // The state before a piece's first tile.
  __device__ __forceinline__ void begin(const AttendArgs& a, const AttendPlan& plan, int group,
                                        const AttendPiece<T>& p) {
    const int chunk = p.seg % p.chunks;
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      const int i = (chunk * plan.rows + 16 * t + col) / group;
      clear(t, i < p.n ? p.len + i : -1);
      if constexpr (kQueryLds) {
        u32x4 qt[L::kSteps];
        load_q(qt, a, plan, group, p, t);
#pragma unroll
        for (int x = 0; x < L::kSteps; ++x) sh_q[t * L::kSteps + x][lane] = qt[x];  // (read by this lane alone)
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // Query operands in registers are on their way while the piece before is written.
  __device__ __forceinline__ void prefetch_q(const AttendArgs& a, const AttendPlan& plan, int group,
                                             const AttendPiece<T>& p) {
    if constexpr (!kQueryLds)
#pragma unroll
      for (int t = 0; t < kRowTiles; ++t) load_q(q[t], a, plan, group, p, t);
  }

  // A piece's tiles; K and V of the first are on their way already.  The next tile's K is loaded while
  // this one's scores become probabilities, its V after the products, and its pages are looked up one
  // tile earlier.  After the last tile comes the next piece's first one: its loads are in flight while
  // this piece is written.
  __device__ __forceinline__ void walk(const AttendPiece<T>& now, const AttendPiece<T>& next) {
    int tile = now.first;
    Pages pages = ahead(now, next, tile + 1);
    f32x4 p[kRowTiles][L::kSub];
    const int whole_end = min(now.end, (now.len + 1) / L::kKeys);  // every row sees every slot
    for (; tile < whole_end; ++tile) {
      scores(p);
      __builtin_amdgcn_sched_barrier(0);
      const Rows rows = next_k(now, next, tile, pages);
      __builtin_amdgcn_sched_barrier(0);
      softmax(p);
      products(p);
      __builtin_amdgcn_sched_barrier(0);
      next_v(now, next, tile, rows);
      __builtin_amdgcn_sched_barrier(0);
    }
    for (; tile < now.end; ++tile) {
      const int first = tile * L::kKeys;
      scores(p);
      __builtin_amdgcn_sched_barrier(0);
      const Rows rows = next_k(now, next, tile, pages);
      __builtin_amdgcn_sched_barrier(0);
      mask(p, first);
      softmax(p);
      products_edge(p, first, now.len, now.len + now.n);
      __builtin_amdgcn_sched_barrier(0);
      next_v(now, next, tile, rows);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// Four elements from d on of an output row, and with the first its lse.
template <typename T>
__device__ __forceinline__ void write_row(const AttendArgs& a, const KvArgs& c, long long row, int d, f32x4 sum,
                                          float top, float total) {
  sum *= 1.f / total;
  T* out = static_cast<T*>(a.out) + row * c.dim + d;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<u32x2*>(out) = u32x2{pack2<T>(sum[0], sum[1]), pack2<T>(sum[2], sum[3])};
  else
    *reinterpret_cast<f32x4*>(out) = sum;
  if (d == 0 && a.lse)
    a.lse[row] = top == -INFINITY ? __builtin_nanf("") : top * kLn2 + logf(total);
}

// Adds up the parts of a cut segment: workgroups (w, *) those of the one whose first part workgroup w of
// the split holds.  kDim / 4 lanes take a row's part; with few parts such groups take different rows, with
// many they take parts of one row and are added up in LDS.
template <typename T, int kDim>
__global__ __launch_bounds__(kJoinThreads) void attend_join_kernel(AttendArgs a, KvArgs c, AttendPlan plan) {
  constexpr int kLanes = kDim / 4;
  constexpr int kTeams = kJoinThreads / kLanes;
  constexpr int kAhead = 4;
  __shared__ f32x4 sh_o[kTeams][kLanes];
  __shared__ float sh_m[kTeams], sh_l[kTeams];
  const int w = blockIdx.x;
  const CutSegment cut = plan.cut[w];
  if (cut.parts == 0) return;
  const int group = a.q_heads / c.heads;
  const int chunks = chunks_of(cut.n, group, plan.rows);
  const int h = cut.seg / chunks, chunk = cut.seg - h * chunks;
  const int team = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
  const int end = min(plan.rows, cut.n * group - chunk * plan.rows);
  // Teams share out the parts of a row or the rows, whichever takes fewer turns.
  const int by = gridDim.y;
  const bool by_part = (end + by - 1) / by * ((cut.parts + kAhead * kTeams - 1) / (kAhead * kTeams)) <
                       (end + by * kTeams - 1) / (by * kTeams) * ((cut.parts + kAhead - 1) / kAhead);
  const int rows_once = by_part ? 1 : kTeams, part_step = by_part ? kTeams : 1;
  for (int row = blockIdx.y * rows_once; row < end; row += gridDim.y * rows_once) {
    const int local = by_part ? row : row + team;
    const int qrow = chunk * plan.rows + local, i = qrow / group;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float top = -INFINITY, sum = 0.f;
    if (local < end) {
      for (int p = by_part ? team : 0; p < cut.parts; p += kAhead * part_step) {
        f32x4 x[kAhead];
        float m[kAhead], l[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          const int part = min(p + e * part_step, cut.parts - 1);
          const long long at = (2LL * (w + part) + (part == 0 ? 1 : 0)) * plan.rows + local;
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
          if (p + e * part_step >= cut.parts) break;
          const float f = exp2_hw(m[e] - base);
          o += x[e] * f;
          sum += l[e] * f;
        }
        top = now;
      }
    }
    if (by_part) {
      sh_o[team][d / 4] = o;
      if (d == 0) {
        sh_m[team] = top;
        sh_l[team] = sum;
      }
      __syncthreads();
      top = -INFINITY;
      for (int t = 0; t < kTeams; ++t) top = fmaxf(top, sh_m[t]);
      const float base = top == -INFINITY ? 0.f : top;
      o = f32x4{0.f, 0.f, 0.f, 0.f};
      sum = 0.f;
      for (int t = 0; t < kTeams; ++t) {
        const float f = exp2_hw(sh_m[t] - base);
        o += sh_o[t][d / 4] * f;
        sum += sh_l[t] * f;
      }
      __syncthreads();
    }
    if (local < end && d < c.dim && (!by_part || team == 0))
      write_row<T>(a, c,
                   (static_cast<long long>(cut.b) * (a.K + 1) + i) * a.q_heads + h * group + qrow - i * group,
                   d, o, top, sum);
  }
}

// The piece of a range that begins with tile `first` of a segment and has `left` tiles at most.
template <typename T, int kKeys>
__device__ __forceinline__ AttendPiece<T> make_piece(const KvArgs& c, const AttendPlan& plan, int group, int b,
                                                     int seg, int len, int n, int first, long long left,
                                                     int whole = 0) {
  AttendPiece<T> p;
  p.b = b;
  p.seg = seg;
  p.len = len;
  p.n = n;
  p.chunks = chunks_of(n, group, plan.rows);
  p.tiles = tiles_of<kKeys>(len, n);
  p.first = first;
  p.end = p.tiles <= whole ? p.tiles : static_cast<int>(min(static_cast<long long>(p.tiles), first + left));
  const int h = seg / p.chunks;
  p.kpool = reinterpret_cast<const T*>(c.k) + h * c.head_stride;
  p.vpool = reinterpret_cast<const T*>(c.v) + h * c.head_stride;
  p.table = c.table + static_cast<long long>(b) * c.max_pages;
  return p;
}

// A wave's (or workgroup's) range, and the piece of a segment that it begins with.
struct RangeStart {
  long long total, begin, end;
  int wg, log_waves, log_ranges, b, len, n, seg, first;
};

// Every wave finds its own; its number in the workgroup is `wave` (0 where the workgroup shares one range).
template <int kKeys>
__device__ __forceinline__ RangeStart range_start(const AttendArgs& a, const KvArgs& c, const AttendPlan& plan,
                                                  int group, int lane, int wave) {
  // Tiles before each sequence: every lane sums a run of sequences, then a scan over the lanes.
  const int per = (a.B + 63) / 64;
  const int run0 = min(a.B, lane * per), run1 = min(a.B, run0 + per);
  long long mine = 0;
  RoundRows r{};
  for (int b = run0; b < run1; ++b) {
    r = round_rows(c, a.num_draft, a.kv_len, b, a.K);
    mine += work_of<kKeys>(r, c.heads, group, plan.rows);
  }
  const long long upto = scan_work(mine);
  RangeStart s{};
  s.total = read_lane64(upto, 63);
  // Few tiles: fewer waves of a workgroup have a range (the first ones), so that the tiles are spread over the
  // CUs: 200 tiles of one sequence take 13.6 us on 200 of them, each part straight to memory, and 16.1 on 50.
  const int log_groups = plan.log_ranges - plan.log_waves;
  int log_waves = plan.log_waves;
  while (log_waves > 0 && s.total <= 1LL << (log_groups + log_waves - 1)) --log_waves;
  s.log_waves = log_waves;
  s.log_ranges = log_groups + log_waves;
  // Neighbouring ranges go to one XCD (workgroups are dealt to the 8 XCDs in turn), so that row chunks of
  // the same slots meet in its L2; too few tiles for that go round all XCDs.
  s.wg = s.total >> s.log_ranges == 0 ? static_cast<int>(blockIdx.x)
                                      : static_cast<int>(blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8);
  if (wave >> log_waves) return s;
  const int w = (s.wg << log_waves) + wave;
  s.begin = range_begin(w, s.total, s.log_ranges);
  s.end = range_begin(w + 1, s.total, s.log_ranges);
  if (s.begin >= s.end) return s;
  // The sequence that holds tile `begin`: the lane whose run does, then along its run.
  const int owner = __builtin_ctzll(__ballot(mine > 0 && s.begin < upto));
  long long before = read_lane64(upto - mine, owner);
  s.b = uniform(owner * per);
  s.len = __builtin_amdgcn_readlane(r.len, owner);
  s.n = __builtin_amdgcn_readlane(r.n, owner);
  for (; per > 1; ++s.b) {
    const RoundRows x = round_rows(c, a.num_draft, a.kv_len, s.b, a.K);
    s.len = uniform(x.len);
    s.n = uniform(x.n);
    const long long work = work_of<kKeys>(x, c.heads, group, plan.rows);
    if (s.begin < before + work) break;
    before += work;
  }
  // (a sequence has under 2^28 tiles; `inside` is under 2^53, so the quotient's floor is exact)
  const int tiles = tiles_of<kKeys>(s.len, s.n);
  const long long inside = s.begin - before;
  s.seg = uniform(static_cast<int>(static_cast<double>(inside) / static_cast<double>(tiles)));
  s.first = uniform(static_cast<int>(inside - static_cast<long long>(s.seg) * tiles));
  return s;
}

// Rows past the last new token are 0, those of an invalid sequence NaN.
template <typename T>
__device__ __forceinline__ void fill_unused_rows(const AttendArgs& a, const KvArgs& c) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const RoundRows r = round_rows(c, a.num_draft, a.kv_len, b, a.K);
    const long long row = static_cast<long long>(b) * (a.K + 1) * a.q_heads;
    const long long rows = (a.K + 1LL) * a.q_heads, wrong = static_cast<long long>(r.rows) * a.q_heads;
    T* out = static_cast<T*>(a.out) + row * c.dim;
    const long long from = static_cast<long long>(r.n) * a.q_heads;
    for (long long x = from * c.dim + threadIdx.x; x < rows * c.dim; x += blockDim.x)
      out[x] = from_float<T>(x < wrong * c.dim ? __builtin_nanf("") : 0.f);
    for (long long x = from + threadIdx.x; a.lse && x < rows; x += blockDim.x)
      a.lse[row + x] = x < wrong ? __builtin_nanf("") : -INFINITY;
  }
}

// What a wave leaves of a segment that it has a part of.
struct PartNote {
  int b, seg, n, chunks;
  bool any, begins, ends;
  long long segment_end;  // of one that begins: the tile after its last
};

// Waves a SIMD that the registers of the split kernel are planned for.
template <typename T>
constexpr int split_occupancy(int dim, bool fast, int row_tiles) {
  return dim == 256 || (dim == 128 && row_tiles == 2 && (!fast || sizeof(T) == 4)) ? 1 : 2;
}

// A wave works through its range on its own: none waits for another until all are done.  Then a workgroup of
// several waves adds up in LDS the segments that its waves have cut between them.  kFast: head_dim is kDim,
// pages are whole groups of 16 slots and 16 slots lie within 2^32 bytes.
template <typename T, int kDim, bool kFast, int kRowTiles, int kWaves>
__global__ __launch_bounds__(64 * kWaves, split_occupancy<T>(kDim, kFast, kRowTiles)) void attend_split_kernel(
    AttendArgs a, KvArgs c, AttendPlan plan) {
  typedef Tile<T, kDim, kFast> L;
  // (where the LDS does not hold parts and they would take over 32 registers)
  constexpr bool kQueryLds = kWaves == 1 && kRowTiles * L::kSteps > 8;
  typedef AttendWave<T, kDim, kFast, kRowTiles, kQueryLds> Wave;
  constexpr int kRows = 16 * kRowTiles, kPad = kDim + 4;
  __shared__ u32x4 sh_q[kQueryLds ? kRowTiles * L::kSteps : 1][64];
  // (dynamic, so that the compiler plans registers for two waves a SIMD: with one it keeps the outputs in
  // accumulation registers and moves them back and forth for every tile)
  extern __shared__ float sh_parts[];
  auto sh_o = [&](int note, int row, int d) __attribute__((always_inline)) {
    return reinterpret_cast<f32x4*>(sh_parts + (note * kRows + row) * kPad + d);
  };
  __shared__ float sh_m[2 * kWaves][kRows], sh_l[2 * kWaves][kRows];
  __shared__ PartNote sh_note[2 * kWaves];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int group = a.q_heads / c.heads;
  const RangeStart at = range_start<L::kKeys>(a, c, plan, group, lane, wave);
  const int wg = at.wg;
  const long long begin = at.begin, end = at.end, total = at.total;
  fill_unused_rows<T>(a, c);
  if (threadIdx.x == 0) plan.cut[wg].parts = 0;
  const bool in_lds = kWaves > 1 && at.log_waves > 0;  // (else one wave's parts are the workgroup's)
  if (kWaves > 1 && lane < 2) sh_note[2 * wave + lane].any = false;
  if (begin < end) {
  Wave s(c);
  s.page_shift = plan.page_shift;
  s.lane = lane;
  s.col = col;
  s.g = g;
  s.scale = plan.scale_log2;
  s.sh_q = sh_q;
  s.bad = s.bad_next = false;

  long long left = end - begin;
  AttendPiece<T> now = make_piece<T, L::kKeys>(c, plan, group, at.b, at.seg, at.len, at.n, at.first, left), next;
  left -= now.end - now.first;
  s.enter(now);
  s.prefetch_q(a, plan, group, now);

  for (;;) {
    const bool more = left > 0;
    next = now;
    next.end = 0;
    if (more) {
      int nb = now.b, seg = now.seg + 1, nlen = now.len, nn = now.n;
      if (seg == c.heads * now.chunks) {
        seg = 0;
        do {
          const RoundRows x = round_rows(c, a.num_draft, a.kv_len, ++nb, a.K);
          nlen = uniform(x.len);
          nn = uniform(x.n);
        } while (nn == 0);
      }
      next = make_piece<T, L::kKeys>(c, plan, group, nb, seg, nlen, nn, 0, left);
      left -= next.end;
    }
    s.begin(a, plan, group, now);
    s.walk(now, next);
    if (more) s.prefetch_q(a, plan, group, next);

    // The rows, or if other ranges hold the rest of the segment this piece's part of them.
    const bool begins = now.first == 0, ends = now.end == now.tiles, whole = begins && ends;
    const int h = now.seg / now.chunks, chunk = now.seg - h * now.chunks;
    const int slot = begins ? 1 : 0;
    if (in_lds && !whole && lane == 0)
      sh_note[2 * wave + slot] = PartNote{now.b,  now.seg, now.n, now.chunks,
                                             true,   begins,  ends,  end - now.end + now.tiles};
    if (!in_lds && begins && !ends && lane == 0)
      plan.cut[wg] = CutSegment{range_of(end - now.end + now.tiles - 1, total, at.log_ranges) - wg + 1,
                                now.b, now.seg, now.n};
    const bool bad = __any(s.bad);
    int id = threadIdx.x & 63;  // (volatile: addresses are made here, not kept through the walk)
    asm volatile("" : "+v"(id));
    const int col = id & 15, g = id >> 4;
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      const int local = 16 * t + col, qrow = chunk * plan.rows + local, i = qrow / group;
      float sum = row_sum(s.l[t]), top = s.m[t];
      if (bad) {  // a page id outside the pool: the rows' sums are NaN, whatever else they hold
        sum = __builtin_nanf("");
        if (top == -INFINITY) top = 0.f;
      }
      if (i >= now.n) continue;
      const long long row =
          (static_cast<long long>(now.b) * (a.K + 1) + i) * a.q_heads + h * group + qrow - i * group;
      const long long part_row = (2LL * wg + slot) * plan.rows + local;
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < L::kOut; y += 4) {
          const int d = L::kChunk * (4 * g + x) + y;
          const f32x4 four = {s.o[t][y][x], s.o[t][y + 1][x], s.o[t][y + 2][x], s.o[t][y + 3][x]};
          if (whole) {
            if (d < c.dim) write_row<T>(a, c, row, d, four, top, sum);
          } else if (in_lds) {
            *sh_o(2 * wave + slot, local, d) = four;
          } else {
            *reinterpret_cast<f32x4*>(plan.part_o + part_row * kDim + d) = four;
          }
          __builtin_amdgcn_sched_barrier(0);  // (few copies of the outputs at a time)
        }
      if (!whole && g == 0) {
        if (in_lds) {
          sh_m[2 * wave + slot][local] = top;
          sh_l[2 * wave + slot][local] = sum;
        } else {
          plan.part_m[part_row] = top;
          plan.part_l[part_row] = sum;
        }
      }
    }
    if (!more) break;
    now = next;
    s.bad = s.bad_next;
    s.bad_next = false;
  }
  }
  if (in_lds) {
    __syncthreads();
    // Neighbouring parts of one segment, in order: a wave's part that begins nothing comes first.
    for (int x = 0; x < 2 * kWaves;) {
      const PartNote first = sh_note[x];
      if (!first.any) {
        ++x;
        continue;
      }
      int last = x;
      bool ends = first.ends;
      for (int y = x + 1; y < 2 * kWaves && !ends; ++y)
        if (sh_note[y].any) {
          last = y;
          ends = sh_note[y].ends;
        }
      const int h = first.seg / first.chunks, chunk = first.seg - h * first.chunks;
      const int used = min(kRows, first.n * group - chunk * plan.rows);
      for (int idx = threadIdx.x; idx < used * (kDim / 4); idx += 64 * kWaves) {
        const int local = idx / (kDim / 4), d = idx % (kDim / 4) * 4;
        float top = -INFINITY;
        for (int y = x; y <= last; ++y)
          if (sh_note[y].any) top = fmaxf(top, sh_m[y][local]);
        const float base = top == -INFINITY ? 0.f : top;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        float sum = 0.f;
        for (int y = x; y <= last; ++y)
          if (sh_note[y].any) {
            const float f = exp2_hw(sh_m[y][local] - base);
            o += *sh_o(y, local, d) * f;
            sum += sh_l[y][local] * f;
          }
        if (first.begins && ends) {
          const int qrow = chunk * plan.rows + local, i = qrow / group;
          if (d < c.dim)
            write_row<T>(a, c,
                         (static_cast<long long>(first.b) * (a.K + 1) + i) * a.q_heads + h * group + qrow - i * group,
                         d, o, top, sum);
        } else {
          const long long row = (2LL * wg + (first.begins ? 1 : 0)) * plan.rows + local;
          *reinterpret_cast<f32x4*>(plan.part_o + row * kDim + d) = o;
          if (d == 0) {
            plan.part_m[row] = top;
            plan.part_l[row] = sum;
          }
        }
      }
      if (first.begins && !ends && threadIdx.x == 0) {  // (it ends the workgroup's range)
        plan.cut[wg] = CutSegment{(range_of(first.segment_end - 1, total, at.log_ranges) >> at.log_waves) - wg + 1,
                                  first.b, first.seg, first.n};
      }
      x = last + 1;
    }
  }
}

// The same for many rows: four waves with 16 or 32 rows each share every tile of K and V through LDS; the next tile
// is on its way in registers while this one is computed on.  A tile lies in LDS operand by operand, 64 lanes x 16
// or 8 bytes as the matrix instructions take them, so that it is written and read in order, without bank conflicts,
// and is read as it is needed: whole operands in registers left no room for 32 rows a wave, which halve the bytes
// read from LDS for each product (64 tokens of 32 heads on 4 kv heads over 44 x 416-3329 slots of float16: head
// dim 128 277 -> 217 us, 256 859 -> 558 us, 310 TFLOP/s).
// (Two tiles a barrier took 650 us for 64 rows over 64 x 8-16k slots where one takes 596; two tiles ahead in
// registers 648; 16 rows a wave 648 where 64 rows in one wave took 588-670.)
template <typename T, int kDim, bool kFast, int kRowTiles, int kWaves>
__global__ __launch_bounds__(64 * kWaves, kDim == 256 && kRowTiles == 2 ? 1 : 2) void attend_wide_kernel(
    AttendArgs a, KvArgs c, AttendPlan plan) {
  typedef Tile<T, kDim, kFast> L;
  typedef AttendWave<T, kDim, kFast, kRowTiles, false, true> Wave;
  constexpr int kStepsK = L::kSub * L::kSteps;     // K operands a tile, a wave's share of them to load
  constexpr int kStepsV = L::kRowsV * L::kLoadsV;  // V loads a tile, likewise
  constexpr int kMineK = kStepsK / kWaves, kMineV = kStepsV / kWaves;
  typedef typename L::LoadV VecV;
  extern __shared__ float sh_parts[];
  constexpr int kPlanes = L::kRowsV * Wave::kPairs;
  u32x4(*sh_k)[64] = reinterpret_cast<u32x4(*)[64]>(sh_parts);              // [2][kStepsK]
  u32x2(*sh_v)[64] = reinterpret_cast<u32x2(*)[64]>(sh_k + 2 * kStepsK);    // [2][kPlanes]
  __shared__ int sh_bad[kWaves];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int group = a.q_heads / c.heads;
  const RangeStart at = range_start<L::kKeys>(a, c, plan, group, lane, 0);
  const int wg = at.wg;
  fill_unused_rows<T>(a, c);
  if (threadIdx.x == 0) plan.cut[wg].parts = 0;
  if (at.begin >= at.end) return;

  Wave s(c);
  s.page_shift = plan.page_shift;
  s.lane = lane;
  s.col = col;
  s.g = g;
  s.scale = plan.scale_log2;
  s.bad = false;
  long long left = at.end - at.begin;
  const int whole_tiles = at.total >> at.log_ranges == 0 ? 0 : kWholeTiles;  // (few tiles: one each)
  AttendPiece<T> now =
      make_piece<T, L::kKeys>(c, plan, group, at.b, at.seg, at.len, at.n, at.first, left, whole_tiles);
  auto advance = [&]() __attribute__((always_inline)) {
    int nb = now.b, seg = now.seg + 1, nlen = now.len, nn = now.n;
    if (seg == c.heads * now.chunks) {
      seg = 0;
      do {
        const RoundRows x = round_rows(c, a.num_draft, a.kv_len, ++nb, a.K);
        nlen = uniform(x.len);
        nn = uniform(x.n);
      } while (nn == 0);
    }
    now = make_piece<T, L::kKeys>(c, plan, group, nb, seg, nlen, nn, 0, left, whole_tiles);
  };
  if (now.first > 0 && now.tiles <= whole_tiles) {  // (done by the workgroup that has its first tile)
    left -= now.tiles - now.first;
    if (left <= 0) return;
    advance();
  }
  const int sub = L::kSub == 2 ? 2 * wave / kWaves : 0;  // the 16-slot group of all that this wave loads
  const int step_k = wave * kMineK % L::kSteps, step_v = wave * kMineV;

  for (;;) {
    left -= now.end - now.first;
    const int h = now.seg / now.chunks, chunk = now.seg - h * now.chunks;
    const int wave_row = chunk * plan.rows + 16 * kRowTiles * wave;
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      const int qrow = wave_row + 16 * t + col, i = qrow / group;
      s.clear(t, i < now.n ? now.len + i : -1);
#pragma unroll
      for (int x = 0; x < L::kSteps; ++x) s.q[t][x] = u32x4{0, 0, 0, 0};
      if (i < now.n)
        L::template load_row<false>(
            s.q[t],
            (GlobalBytes)(static_cast<const T*>(a.q) +
                          (static_cast<long long>(now.b) * (a.K + 1) + i) * a.q_stride +
                          static_cast<long long>(h * group + qrow - i * group) * c.dim),
            0u, g, c.dim);
    }

    // The wave's part of the tile on its way, in registers, and where the next one's rows lie.
    u32x4 mine_k[kMineK];
    VecV mine_v[kMineV];
    int page[kFast ? 1 : 1 + kMineV], off[kFast ? 1 : 1 + kMineV];
    const int last_slot = now.len + now.n - 1;
    auto find = [&](int tile) __attribute__((always_inline)) {
      const int base = min(tile, now.end - 1) * L::kKeys;  // (past the end: the last tile again)
      if constexpr (kFast) {
        const int slot = min(base + 16 * sub, last_slot & ~15);
        const int idx = uniform(s.page_index(slot));
        off[0] = slot - idx * c.page_size;
        page[0] = table_at(now.table, idx);
      } else {
#pragma unroll
        for (int y = 0; y < 1 + kMineV; ++y) {
          const int v = (step_v + y - 1) / L::kLoadsV;
          const int slot = min(base + (y == 0 ? 16 * sub + col : 16 * (v / 4) + 4 * g + v % 4), last_slot);
          const int idx = s.page_index(slot);
          off[y] = slot - idx * c.page_size;
          page[y] = now.table[idx];
        }
      }
    };
    auto row_of = [&](int y) __attribute__((always_inline)) {
      const bool good = static_cast<unsigned>(page[y]) < static_cast<unsigned>(c.num_pages);
      s.bad = s.bad || !good;
      return (good ? page[y] : 0) * c.page_stride + off[y] * c.slot_stride;
    };
    auto fetch = [&]() __attribute__((always_inline)) {
      const long long k_row = row_of(0);
#pragma unroll
      for (int y = 0; y < kMineK; ++y) {
        if constexpr (kFast)
          mine_k[y] = L::template load_step<true>(
              scalar_base(now.kpool + k_row), static_cast<unsigned>(col) * static_cast<unsigned>(c.slot_stride),
              step_k + y, g, c.dim);
        else
          mine_k[y] = L::template load_step<true>((GlobalBytes)(now.kpool + k_row), 0u, step_k + y, g, c.dim);
      }
#pragma unroll
      for (int y = 0; y < kMineV; ++y) {
        const int v = (step_v + y) / L::kLoadsV, z = (step_v + y) % L::kLoadsV;
        if constexpr (kFast)
          mine_v[y] = L::template load_v_step<true>(
              scalar_base(now.vpool + k_row),
              static_cast<unsigned>(4 * g + v % 4) * static_cast<unsigned>(c.slot_stride), z, col, c.dim);
        else
          mine_v[y] = L::template load_v_step<true>((GlobalBytes)(now.vpool + row_of(1 + y)), 0u, z, col, c.dim);
      }
    };
    auto put = [&](int buffer) __attribute__((always_inline)) {
#pragma unroll
      for (int y = 0; y < kMineK; ++y)
        sh_k[buffer * kStepsK + wave * kMineK + y][lane] = mine_k[y];
#pragma unroll
      for (int y = 0; y < kMineV; ++y)
#pragma unroll
        for (int e = 0; e < L::kLoadWords / 2; ++e) {
          const int row = (step_v + y) / L::kLoadsV, pair = (step_v + y) % L::kLoadsV * (L::kLoadWords / 2) + e;
          sh_v[buffer * kPlanes + pair * L::kRowsV + row][lane] = u32x2{mine_v[y][2 * e], mine_v[y][2 * e + 1]};
        }
    };

    find(now.first);
    fetch();
    find(now.first + 1);
    put(0);
    // (two loops, as in the split kernel: with both kinds of tile in one the compiler keeps two copies of the outputs)
    auto step = [&](int tile, int buffer, auto edge) __attribute__((always_inline)) {
      fetch();
      find(tile + 2);
      // All waves' parts of this buffer are written, and the other buffer's are read.  (LDS alone is waited
      // for: the loads above stay in flight.)
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (wave_row < now.n * group) {
        s.sh_k = sh_k + buffer * kStepsK;
        s.sh_v = sh_v + buffer * kPlanes;
        f32x4 p[kRowTiles][L::kSub];
        s.scores(p);
        if constexpr (decltype(edge)::value) {
          s.mask(p, tile * L::kKeys);
          s.softmax(p);
          s.products_edge(p, tile * L::kKeys, now.len, now.len + now.n);
        } else {
          s.softmax(p);
          s.products(p);
        }
      }
      put(buffer ^ 1);
    };
    const int whole_end = min(now.end, (now.len + 1) / L::kKeys);  // every row sees every slot
    int tile = now.first, buffer = 0;
    for (; tile < whole_end; ++tile, buffer ^= 1) step(tile, buffer, std::false_type{});
    for (; tile < now.end; ++tile, buffer ^= 1) step(tile, buffer, std::true_type{});

    const bool begins = now.first == 0, whole = begins && now.end == now.tiles;
    const int slot = begins ? 1 : 0;
    if (begins && !whole && threadIdx.x == 0)
      plan.cut[wg] = CutSegment{range_of(at.end - now.end + now.tiles - 1, at.total, at.log_ranges) - wg + 1,
                                now.b, now.seg, now.n};
    const bool mine_bad = __any(s.bad);
    if (lane == 0) sh_bad[wave] = mine_bad;
    __syncthreads();  // (also: all have read the buffers that the next piece writes)
    int bad = 0;
#pragma unroll
    for (int x = 0; x < kWaves; ++x) bad |= sh_bad[x];
    s.bad = false;
    int id = threadIdx.x & 63;  // (volatile: addresses are made here, not kept through the walk)
    asm volatile("" : "+v"(id));
    const int col = id & 15, g = id >> 4;
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      const int qrow = wave_row + 16 * t + col, i = qrow / group;
      float sum = row_sum(s.l[t]), top = s.m[t];
      if (bad) {
        sum = __builtin_nanf("");
        if (top == -INFINITY) top = 0.f;
      }
      if (i >= now.n) continue;
      const long long row =
          (static_cast<long long>(now.b) * (a.K + 1) + i) * a.q_heads + h * group + qrow - i * group;
      const long long part_row = (2LL * wg + slot) * plan.rows + qrow - chunk * plan.rows;
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < L::kOut; y += 4) {
          const int d = L::kChunk * (4 * g + x) + y;
          const f32x4 four = {s.o[t][y][x], s.o[t][y + 1][x], s.o[t][y + 2][x], s.o[t][y + 3][x]};
          if (!whole)
            *reinterpret_cast<f32x4*>(plan.part_o + part_row * kDim + d) = four;
          else if (d < c.dim)
            write_row<T>(a, c, row, d, four, top, sum);
          __builtin_amdgcn_sched_barrier(0);  // (few copies of the outputs at a time)
        }
      if (!whole && g == 0) {
        plan.part_m[part_row] = top;
        plan.part_l[part_row] = sum;
      }
    }
    if (left <= 0) return;
    advance();
  }
}

template <typename T, int kDim, bool kFast>
void launch_attend_dim(const AttendArgs& a, const KvArgs& c, const AttendPlan& p) {
  const unsigned groups = 1u << (p.log_ranges - p.log_waves);
  if (p.wide) {
    constexpr unsigned kLds = 2 * 2 * Tile<T, kDim, kFast>::kKeys * kDim * sizeof(T);  // two tiles of K and V
    if (p.rows == 64)
      attend_wide_kernel<T, kDim, kFast, 1, 4><<<groups, 256, kLds, a.stream>>>(a, c, p);
    else
      attend_wide_kernel<T, kDim, kFast, 2, 4><<<groups, 256, kLds, a.stream>>>(a, c, p);
  } else if constexpr (kDim == 256) {
    attend_split_kernel<T, kDim, kFast, 1, 1><<<groups, 64, 0, a.stream>>>(a, c, p);
  } else {
    const unsigned lds = 8 * p.rows * (kDim + 4) * sizeof(float);
    if (p.rows == 16)
      attend_split_kernel<T, kDim, kFast, 1, 4><<<groups, 256, lds, a.stream>>>(a, c, p);
    else
      attend_split_kernel<T, kDim, kFast, 2, 4><<<groups, 256, lds, a.stream>>>(a, c, p);
  }
  const int rows = p.rows < (a.K + 1) * (a.q_heads / c.heads) ? p.rows : (a.K + 1) * (a.q_heads / c.heads);
  // (the widest heads have half as many rows a workgroup; more for the others cost what they gained)
  const int by = kDim == 256 ? 16 : 8;
  attend_join_kernel<T, kDim><<<dim3(groups, rows < by ? rows : by), kJoinThreads, 0, a.stream>>>(a, c, p);
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

}  // namespace specdec
