// gfx950 kernels of the eviction by accumulated attention weight.
//
// Of a (sequence, kv head)'s L slots the `budget` ones with the largest keys stay; a key is the order of the weight
// as an unsigned number, with protected positions above all.  A radix search (11, 11 and 10 bits) finds the budget-th
// largest key; then the slots are walked over in order.  A slot's rank is what decides:  with G(s) and T(s) the slots
// before s that lie above the threshold key and at it, and `left` the number at it that stay,
//   kept before s = G(s) + min(T(s), left),
// which is the place among the holes of an evicted slot s < budget (s - kept before s) and, counted from the end, of
// a kept slot s >= budget among the movers.  There are as many of one as of the other, and mover i is copied over
// hole i.  Sources lie at or above `budget` and destinations below it, so the copies are independent of each other.
//
// Few slots: one workgroup per sequence and head reads the records once and does everything, keys and positions in
// registers.  Many: a workgroup has 4096 slots of a pair, and each pass is a launch, as the next needs all
// workgroups' counts; the keys lie in the workspace.
//
// Bound: for a full cache that gives up a round's slots the latency of one workgroup's passes (the records are 8
// bytes a slot): 64 x 4097-4105 slots of 8 heads down to 4096 take 22 us, 61 in passes over parts.  For a deep cut
// the rows that move: 4 x 50-65 k slots of 8 heads down to 8000 take 96 us, 54 of them copies at 4.2 TB/s (one
// workgroup a pair: 127, keys in registers as far as they fit).
#include <hip/hip_runtime.h>

#include "paged.h"
#include "paged_tiles.h"
#include "wave_ops.h"

namespace specdec {
namespace {

constexpr int kGroup = 256;        // slots a wave takes at once, four a lane
constexpr int kBins = 2048;
constexpr int kFewWaves = 8, kFewHold = 4;       // groups that a wave holds: up to 8192 slots
constexpr int kFewSlots = kFewWaves * kFewHold * kGroup;
constexpr int kPartWaves = 4, kPartHold = 4;     // of a part
constexpr int kPartSlots = kPartWaves * kPartHold * kGroup;
constexpr int kMoveWaves = 4;
constexpr int kMoveBatch = 16;     // rows that a wave moves at once
// The select kernel's workgroup moves the rows itself where there cannot be more than these: 64 x 8 full caches that
// give up some slots take 28.0 us so and 29.7 with a second launch, 229 x 8 that move up to 187 rows 114 and 123.
constexpr int kOwnMoves = 256;

// What the passes over many slots leave of a (sequence, head).
struct EvictState {
  unsigned threshold;
  int left;
};
struct PartRecord {
  int newest, bad;    // of a part's slots: the largest position, a page outside the pool
  int above, ties;    // and those above the threshold and at it
};

// Workspace: per (sequence, head) the number of moves, the movers and the holes; for caches of many slots also what
// the passes hand on.
struct EvictLists {
  int32_t* count;
  int32_t* from;       // the movers, at the end of `most` places
  int32_t* to;         // the holes, from the first place on
  long long most;      // entries per (sequence, head)
  unsigned* keys;      // [slots] per (sequence, head)
  unsigned* positions;
  unsigned* hist;      // [3][kBins]
  EvictState* state;   // [3], after each pass
  PartRecord* part;    // [parts]
  long long slots;     // capacity rounded up to whole parts
  int parts;
  int own_moves;       // the select kernel moves the rows and writes new_len
  unsigned magic;      // 2^32 / (16-byte vectors of a row of k and v) rounded up
};

long long most_moves(long long capacity, int budget) {
  return capacity <= budget ? 0 : capacity - budget < budget ? capacity - budget : budget;
}
long long part_count(long long capacity) { return (capacity + kPartSlots - 1) / kPartSlots; }

// Unsigned order of a weight: NaN 0, then ascending; -0 and +0 alike.
__device__ __forceinline__ unsigned weight_order(float w) {
  if (w != w) return 0u;
  const unsigned u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int wave_scan(int v) {  // inclusive
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

// Copies movers [first, first + count) of `total` over their holes; count <= kMoveBatch.  kFlight: 16-byte loads of a
// lane on their way at once.
template <int kFlight>
__device__ __forceinline__ void move_rows(const KvArgs& c, const EvictLists& lists, long long bh, int b, int h,
                                          int esize, int total, int first, int count, int lane) {
  typedef u32x4 __attribute__((address_space(1)))* Rows;
  long long src = 0, dst = 0;
  if (lane < count) {
    const int s = lists.from[bh * lists.most + lists.most - total + first + lane];
    const int d = lists.to[bh * lists.most + first + lane];
    const int sp = page_of(c, b, s), dp = page_of(c, b, d);
    const int so = s % c.page_size, dof = d % c.page_size;
    src = row_at(c, sp, so, h) * esize;
    dst = row_at(c, dp, dof, h) * esize;
    const long long from = record_at(c, sp, so, h), to = record_at(c, dp, dof, h);
    c.weight[to] = c.weight[from];
    c.position[to] = c.position[from];
  }
  const int vectors = c.dim * esize / 16, row = 2 * vectors;  // of k, and of k and v
  const int all = count * row;
  for (int x0 = 0; x0 < all; x0 += 64 * kFlight) {
    u32x4 data[kFlight];
    Rows to[kFlight];
#pragma unroll
    for (int y = 0; y < kFlight; ++y) {
      const int x = min(x0 + 64 * y + lane, all - 1);
      const int m = static_cast<int>(__umulhi(static_cast<unsigned>(x), lists.magic)), z = x - m * row;
      const char* part = z < vectors ? c.k : c.v;
      const uintptr_t pool = reinterpret_cast<uintptr_t>(part) + 16 * (z < vectors ? z : z - vectors);
      to[y] = (Rows)(pool + shfl64(dst, m));
      data[y] = *(Rows)(pool + shfl64(src, m));
    }
#pragma unroll
    for (int y = 0; y < kFlight; ++y)
      if (x0 + 64 * y + lane < all) *to[y] = data[y];
  }
}

// A group's part in a lane: the records of four slots from `slot` on, as they are.  kQuad: four slots from a multiple
// of four on lie in one page.
template <bool kQuad>
struct RecordAt {
  int page[kQuad ? 1 : 4], off[kQuad ? 1 : 4];

  __device__ __forceinline__ void find(const KvArgs& c, const int32_t* table, int slot, int L) {
    const int s0 = min(slot, (L - 1) & ~3);  // (past the last slot: the last ones again)
#pragma unroll
    for (int j = 0; j < (kQuad ? 1 : 4); ++j) {
      const int s = min(s0 + j, L - 1), idx = s / c.page_size;
      off[j] = s - idx * c.page_size;
      page[j] = table[idx];
    }
  }
  __device__ __forceinline__ void load(const KvArgs& c, int h, u32x4& weight, u32x4& pos, bool& bad) const {
    typedef unsigned Words __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int j = 0; j < (kQuad ? 1 : 4); ++j) {
      const bool good = static_cast<unsigned>(page[j]) < static_cast<unsigned>(c.num_pages);
      bad = bad || !good;
      const long long r = record_at(c, good ? page[j] : 0, off[j], h);
      if constexpr (kQuad) {
        pos = *reinterpret_cast<const Words*>(c.position + r);
        weight = *reinterpret_cast<const Words*>(c.weight + r);
      } else {
        pos[j] = static_cast<unsigned>(c.position[r]);
        weight[j] = __float_as_uint(c.weight[r]);
      }
    }
  }
};

// Weights to keys; the largest position of slots before L.
__device__ __forceinline__ u32x4 keys_of(u32x4 weight, const u32x4& pos, int slot, int L, int keep_first, int& newest) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int p = static_cast<int>(pos[j]);
    if (slot + j < L) newest = max(newest, p);
    weight[j] = p < keep_first ? 0xffffffffu : weight_order(__uint_as_float(weight[j]));
  }
  return weight;
}
__device__ __forceinline__ void protect(u32x4& key, const u32x4& pos, long long recent) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (static_cast<int>(pos[j]) > recent) key[j] = 0xffffffffu;
}

struct Digit {
  int shift;
  unsigned bits, above, prefix;  // (key & above) == prefix: the digits before are the threshold's
};
// Counts a group's digits.  Where all are the same (zero weights, protected slots) they are added at once: additions
// to one address go one at a time.
__device__ __forceinline__ void count_keys(unsigned* hist, const u32x4& key, int slot, int L, const Digit& d,
                                           int lane) {
  bool in[4], any = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    in[j] = slot + j < L && (key[j] & d.above) == d.prefix;
    any = any || in[j];
  }
  if (!__any(any)) return;
  const unsigned first = uniform(key[0]) >> d.shift & d.bits;
  bool same = true;
  unsigned digit[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    digit[j] = key[j] >> d.shift & d.bits;
    same = same && in[j] && digit[j] == first;
  }
  if (__all(same)) {
    if (lane == 0) atomicAdd(&hist[first], 256u);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (in[j]) atomicAdd(&hist[digit[j]], 1u);
}
__device__ __forceinline__ void count_order(const u32x4& key, int slot, int L, unsigned threshold, int& above,
                                            int& ties) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    above += slot + j < L && key[j] > threshold;
    ties += slot + j < L && key[j] == threshold;
  }
}

// Lists a group's movers and holes; `above` and `ties` are those before the group, then those before the next.
__device__ __forceinline__ void list_moves(const EvictLists& lists, long long bh, const u32x4& key, int slot, int L,
                                           unsigned threshold, int left, int budget, int& above, int& ties,
                                           int* stay) {
  int mine = 0;  // above the threshold and (from bit 16 on) at it
#pragma unroll
  for (int j = 0; j < 4; ++j)
    mine += slot + j >= L ? 0 : key[j] > threshold ? 1 : key[j] == threshold ? 0x10000 : 0;
  const int upto = wave_scan(mine);
  int g = above + ((upto - mine) & 0xffff), t = ties + ((upto - mine) >> 16);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool in = slot + j < L, tie = key[j] == threshold;
    const bool kept = key[j] > threshold || (tie && t < left);
    const int before = g + min(t, left);
    if (in && kept && slot + j >= budget) lists.from[bh * lists.most + lists.most - budget + before] = slot + j;
    if (in && !kept && slot + j < budget) lists.to[bh * lists.most + slot + j - before] = slot + j;
    if (slot + j == budget - 1) *stay = before + kept;
    g += key[j] > threshold;
    t += tie;
  }
  const int all = __builtin_amdgcn_readlane(upto, 63);
  above += all & 0xffff;
  ties += all >> 16;
}

// The digit at which the counts, from the highest digit down, reach `left`, which becomes what is left of it.  A thread
// has kMine of the kBins counts, the highest first; exactly one digit of all fits.  The workgroup's threads come
// together twice.
template <int kWaves, int kMine>
__device__ __forceinline__ unsigned find_digit(const int (&n)[kMine], int& left, int (&sh_sum)[kWaves],
                                               int (&sh_found)[2], int tid, int lane, int wave) {
  int mine = 0;
#pragma unroll
  for (int x = 0; x < kMine; ++x) mine += n[x];
  const int upto = wave_scan(mine);
  if (lane == 63) sh_sum[wave] = upto;
  __syncthreads();
  int before = upto - mine;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) before += w < wave ? sh_sum[w] : 0;
#pragma unroll
  for (int x = 0; x < kMine; ++x) {
    if (before < left && left <= before + n[x]) {
      sh_found[0] = kBins - 1 - kMine * tid - x;
      sh_found[1] = left - before;
    }
    before += n[x];
  }
  __syncthreads();
  left = sh_found[1];
  return static_cast<unsigned>(sh_found[0]);
}

__device__ __forceinline__ Digit digit_of(int pass, unsigned threshold) {
  return Digit{pass == 0 ? 21 : pass == 1 ? 10 : 0, pass == 2 ? 1023u : 2047u,
               pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10), threshold};
}

// The groups [g0, g0 + kHold) that exist (below g1) of a wave: records to registers, four groups on their way at once.
template <int kHold, bool kQuad>
__device__ __forceinline__ void load_records(const KvArgs& c, const int32_t* table, int h, int g0, int g1, int L,
                                             int keep_first, int lane, u32x4 (&key)[kHold], u32x4 (&pos)[kHold],
                                             int& newest, bool& bad) {
  RecordAt<kQuad> at[kHold];
  if (g0 >= g1) return;
#pragma unroll
  for (int x = 0; x < kHold; ++x) at[x].find(c, table, min(g0 + x, g1 - 1) * kGroup + 4 * lane, L);
#pragma unroll
  for (int x = 0; x < kHold; ++x) at[x].load(c, h, key[x], pos[x], bad);
#pragma unroll
  for (int x = 0; x < kHold; ++x)
    if (g0 + x < g1) key[x] = keys_of(key[x], pos[x], (g0 + x) * kGroup + 4 * lane, L, keep_first, newest);
}

__device__ __forceinline__ int wave_max_i(int x) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) x = max(x, __shfl_xor(x, off, 64));
  return x;
}

template <bool kQuad>
__global__ __launch_bounds__(64 * kFewWaves, 4) void evict_select_kernel(EvictArgs a, KvArgs c, EvictLists lists,
                                                                         int esize) {
  constexpr int kThreads = 64 * kFewWaves, kMine = kBins / kThreads;
  __shared__ unsigned sh_hist[kBins];
  __shared__ int sh_wave[2][kFewWaves];
  __shared__ int sh_found[2], sh_stay;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const long long cap = static_cast<long long>(c.max_pages) * c.page_size;
  const long long pairs = static_cast<long long>(a.B) * c.heads;
  for (long long bh = blockIdx.x; bh < pairs; bh += gridDim.x) {
    const int b = static_cast<int>(bh / c.heads), h = static_cast<int>(bh - static_cast<long long>(b) * c.heads);
    const int L = uniform(a.kv_len[b]);
    const bool wrong = L < 0 || L > cap;
    __syncthreads();  // (LDS of the pair before)
    if (wrong || L <= a.budget) {
      if (tid == 0) lists.count[bh] = wrong ? -1 : 0;
      if (tid == 0 && lists.own_moves && h == 0 && a.new_len) a.new_len[b] = wrong ? -1 : L;
      continue;
    }
    // Every wave has a run of groups; their keys stay in registers.
    const int groups = (L + kGroup - 1) / kGroup;
    const int g0 = groups * wave / kFewWaves, g1 = groups * (wave + 1) / kFewWaves;
    const int32_t* table = c.table + static_cast<long long>(b) * c.max_pages;
    u32x4 key[kFewHold] = {}, pos[kFewHold] = {};
    int newest = -0x7fffffff - 1;
    bool bad = false;
    load_records<kFewHold, kQuad>(c, table, h, g0, g1, L, a.keep_first, lane, key, pos, newest, bad);
    newest = wave_max_i(newest);
    bad = __any(bad);
    if (lane == 0) {
      sh_wave[0][wave] = newest;
      sh_wave[1][wave] = bad;
    }
    for (int x = tid; x < kBins; x += kThreads) sh_hist[x] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
      newest = max(newest, sh_wave[0][w]);
      bad = bad || sh_wave[1][w] != 0;
    }
    if (bad) {
      if (tid == 0) lists.count[bh] = -1;
      if (tid == 0 && lists.own_moves && h == 0 && a.new_len) a.new_len[b] = -1;
      continue;
    }
    const long long recent = static_cast<long long>(newest) - a.keep_last;
#pragma unroll
    for (int x = 0; x < kFewHold; ++x) protect(key[x], pos[x], recent);

    // The budget-th largest key, from its highest bits down; `left` of the slots with it are kept.
    unsigned threshold = 0;
    int left = a.budget;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const Digit d = digit_of(pass, threshold);
#pragma unroll
      for (int x = 0; x < kFewHold; ++x)
        if (g0 + x < g1) count_keys(sh_hist, key[x], (g0 + x) * kGroup + 4 * lane, L, d, lane);
      __syncthreads();
      int n[kMine];
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        n[x] = static_cast<int>(sh_hist[kBins - 1 - kMine * tid - x]);
        sh_hist[kBins - 1 - kMine * tid - x] = 0;
      }
      threshold |= find_digit<kFewWaves>(n, left, sh_wave[0], sh_found, tid, lane, wave) << d.shift;
    }

    // Slots above the threshold and at it before each wave's, then the lists.
    int above = 0, ties = 0;
#pragma unroll
    for (int x = 0; x < kFewHold; ++x)
      if (g0 + x < g1) count_order(key[x], (g0 + x) * kGroup + 4 * lane, L, threshold, above, ties);
    above = wave_scan(above);
    ties = wave_scan(ties);
    if (lane == 63) {
      sh_wave[0][wave] = above;
      sh_wave[1][wave] = ties;
    }
    __syncthreads();
    above = ties = 0;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
      above += w < wave ? sh_wave[0][w] : 0;
      ties += w < wave ? sh_wave[1][w] : 0;
    }
#pragma unroll
    for (int x = 0; x < kFewHold; ++x)
      if (g0 + x < g1)
        list_moves(lists, bh, key[x], (g0 + x) * kGroup + 4 * lane, L, threshold, left, a.budget, above, ties,
                   &sh_stay);
    __syncthreads();
    const int moves = a.budget - sh_stay;  // (the slots below the budget that stay are not moved to)
    if (tid == 0) lists.count[bh] = moves;
    if (lists.own_moves) {
      if (tid == 0 && h == 0 && a.new_len) a.new_len[b] = a.budget;
      for (int i = wave * kMoveBatch; i < moves; i += kFewWaves * kMoveBatch)
        move_rows<2>(c, lists, bh, b, h, esize, moves, i, min(kMoveBatch, moves - i), lane);
    }
  }
}

// One pass over many slots; a workgroup has one part of a pair's.
//   0 records to keys and positions   1, 2, 3 counts of a digit   4 slots above the threshold and at it   5 the lists
template <int kPass, bool kQuad>
__global__ __launch_bounds__(64 * kPartWaves) void evict_part_kernel(EvictArgs a, KvArgs c, EvictLists lists) {
  constexpr int kThreads = 64 * kPartWaves, kMine = kBins / kThreads;
  __shared__ unsigned sh_hist[kPass >= 1 && kPass <= 3 ? kBins : 1];
  __shared__ int sh_wave[2][kPartWaves];
  __shared__ int sh_found[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), part = blockIdx.x;
  const long long cap = static_cast<long long>(c.max_pages) * c.page_size;
  const long long pairs = static_cast<long long>(a.B) * c.heads;
  for (long long bh = blockIdx.y; bh < pairs; bh += gridDim.y) {
    const int b = static_cast<int>(bh / c.heads), h = static_cast<int>(bh - static_cast<long long>(b) * c.heads);
    const int L = uniform(a.kv_len[b]);
    const bool wrong = L < 0 || L > cap;
    if (wrong || L <= a.budget) {
      if (kPass == 5 && part == 0 && tid == 0) lists.count[bh] = wrong ? -1 : 0;
      continue;
    }
    // (the last part of L's: it need not be whole; the parts after it only clear counts)
    const int parts = static_cast<int>((L + kPartSlots - 1LL) / kPartSlots);
    const int groups = (L - 1) / kGroup + 1, g0 = (part * kPartWaves + wave) * kPartHold;
    const int g1 = min(groups, g0 + kPartHold);
    u32x4* far_keys = reinterpret_cast<u32x4*>(lists.keys + bh * lists.slots) + g0 * 64LL + lane;
    u32x4* far_pos = reinterpret_cast<u32x4*>(lists.positions + bh * lists.slots) + g0 * 64LL + lane;
    unsigned* hist = lists.hist + bh * 3 * kBins;
    EvictState* state = lists.state + bh * 3;
    PartRecord* records = lists.part + bh * lists.parts;
    if (kPass == 0)
      for (int x = part * kThreads + tid; x < 3 * kBins; x += lists.parts * kThreads) hist[x] = 0;
    if (part >= parts) continue;
    __syncthreads();  // (LDS of the pair before)

    u32x4 key[kPartHold] = {}, pos[kPartHold] = {};
    if constexpr (kPass == 0) {
      int newest = -0x7fffffff - 1;
      bool bad = false;
      load_records<kPartHold, kQuad>(c, c.table + static_cast<long long>(b) * c.max_pages, h, g0, g1, L, a.keep_first,
                                     lane, key, pos, newest, bad);
      newest = wave_max_i(newest);
      bad = __any(bad);
#pragma unroll
      for (int x = 0; x < kPartHold; ++x)
        if (g0 + x < g1) {
          far_keys[64 * x] = key[x];
          far_pos[64 * x] = pos[x];
        }
      if (lane == 0) {
        sh_wave[0][wave] = newest;
        sh_wave[1][wave] = bad;
      }
      __syncthreads();
      if (tid == 0) {
#pragma unroll
        for (int w = 0; w < kPartWaves; ++w) {
          newest = max(newest, sh_wave[0][w]);
          bad = bad || sh_wave[1][w] != 0;
        }
        records[part] = PartRecord{newest, bad, 0, 0};
      }
      continue;
    }

#pragma unroll
    for (int x = 0; x < kPartHold; ++x)
      if (g0 + x < g1) {
        key[x] = far_keys[64 * x];
        if (kPass == 1) pos[x] = far_pos[64 * x];
      }
    // All parts' records, each wave for itself.
    int newest = -0x7fffffff - 1, bad = 0, above = 0, ties = 0;
    for (int x = lane; x < parts; x += 64) {
      const PartRecord r = records[x];
      newest = max(newest, r.newest);
      bad |= r.bad;
      if (kPass == 5 && x < part) {
        above += r.above;
        ties += r.ties;
      }
    }
    if (__any(bad)) {
      if (kPass == 5 && part == 0 && tid == 0) lists.count[bh] = -1;
      continue;
    }
    unsigned threshold = 0;
    int left = a.budget;
    if constexpr (kPass == 1) {
      const long long recent = static_cast<long long>(wave_max_i(newest)) - a.keep_last;
#pragma unroll
      for (int x = 0; x < kPartHold; ++x)
        if (g0 + x < g1) {
          protect(key[x], pos[x], recent);
          far_keys[64 * x] = key[x];
        }
    } else if constexpr (kPass == 5) {
      threshold = state[2].threshold;
      left = state[2].left;
    } else {
      // The digit that the pass before counted, and the state after it for the next one.
      if (kPass > 2) {
        threshold = state[kPass - 3].threshold;
        left = state[kPass - 3].left;
      }
      int n[kMine];
#pragma unroll
      for (int x = 0; x < kMine; ++x)
        n[x] = static_cast<int>(hist[(kPass - 2) * kBins + kBins - 1 - kMine * tid - x]);
      threshold |= find_digit<kPartWaves>(n, left, sh_wave[0], sh_found, tid, lane, wave)
                   << digit_of(kPass - 2, 0).shift;
      if (part == 0 && tid == 0) state[kPass - 2] = EvictState{threshold, left};
    }
    if constexpr (kPass <= 3) {
      for (int x = tid; x < kBins; x += kThreads) sh_hist[x] = 0;
      __syncthreads();
      const Digit d = digit_of(kPass - 1, threshold);
#pragma unroll
      for (int x = 0; x < kPartHold; ++x)
        if (g0 + x < g1) count_keys(sh_hist, key[x], (g0 + x) * kGroup + 4 * lane, L, d, lane);
      __syncthreads();
      for (int x = tid; x < kBins; x += kThreads)
        if (sh_hist[x]) atomicAdd(&hist[(kPass - 1) * kBins + x], sh_hist[x]);  // (whole numbers: any order)
    } else {
      int mine_above = 0, mine_ties = 0;
#pragma unroll
      for (int x = 0; x < kPartHold; ++x)
        if (g0 + x < g1) count_order(key[x], (g0 + x) * kGroup + 4 * lane, L, threshold, mine_above, mine_ties);
      mine_above = wave_scan(mine_above);
      mine_ties = wave_scan(mine_ties);
      if (lane == 63) {
        sh_wave[0][wave] = mine_above;
        sh_wave[1][wave] = mine_ties;
      }
      __syncthreads();
      if constexpr (kPass == 4) {
        if (tid == 0) {
#pragma unroll
          for (int w = 0; w < kPartWaves; ++w) {
            above += sh_wave[0][w];
            ties += sh_wave[1][w];
          }
          records[part].above = above;
          records[part].ties = ties;
        }
      } else {
        above = __builtin_amdgcn_readlane(wave_scan(above), 63);
        ties = __builtin_amdgcn_readlane(wave_scan(ties), 63);
#pragma unroll
        for (int w = 0; w < kPartWaves; ++w) {
          above += w < wave ? sh_wave[0][w] : 0;
          ties += w < wave ? sh_wave[1][w] : 0;
        }
        int stay = -1;
#pragma unroll
        for (int x = 0; x < kPartHold; ++x)
          if (g0 + x < g1)
            list_moves(lists, bh, key[x], (g0 + x) * kGroup + 4 * lane, L, threshold, left, a.budget, above, ties,
                       &stay);
        if (stay >= 0) lists.count[bh] = a.budget - stay;  // (the lane of slot budget - 1)
      }
    }
  }
}

__global__ __launch_bounds__(64 * kMoveWaves) void evict_move_kernel(EvictArgs a, KvArgs c, EvictLists lists,
                                                                     int esize) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const long long pairs = static_cast<long long>(a.B) * c.heads;
  for (long long bh = blockIdx.y; bh < pairs; bh += gridDim.y) {
    const int b = static_cast<int>(bh / c.heads), h = static_cast<int>(bh - (bh / c.heads) * c.heads);
    const int n = lists.count[bh];
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0 && a.new_len)
      a.new_len[b] = n < 0 ? -1 : min(a.kv_len[b], a.budget);
    const int step = gridDim.x * kMoveWaves * kMoveBatch;
    for (long long i = (blockIdx.x * kMoveWaves + wave) * kMoveBatch; i < n; i += step)
      move_rows<8>(c, lists, bh, b, h, esize, n, static_cast<int>(i), min(kMoveBatch, n - static_cast<int>(i)), lane);
  }
}

// The passes, each when the one before has ended.
template <bool kQuad, int kPass = 0>
void launch_parts(const EvictArgs& a, const KvArgs& c, const EvictLists& lists, dim3 grid) {
  evict_part_kernel<kPass, kPass == 0 && kQuad><<<grid, 64 * kPartWaves, 0, a.stream>>>(a, c, lists);
  if constexpr (kPass < 5) launch_parts<kQuad, kPass + 1>(a, c, lists, grid);
}

// The workspace's parts in order, and its size.
size_t lay_out(EvictLists& lists, char* ws, long long pairs, long long capacity, int budget) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = ws + at;
    at += (bytes + 15) & ~size_t{15};
    return p;
  };
  lists.most = most_moves(capacity, budget);
  lists.parts = static_cast<int>(part_count(capacity));
  lists.slots = static_cast<long long>(lists.parts) * kPartSlots;
  lists.count = reinterpret_cast<int32_t*>(take(pairs * 4));
  lists.from = reinterpret_cast<int32_t*>(take(pairs * lists.most * 4));
  lists.to = reinterpret_cast<int32_t*>(take(pairs * lists.most * 4));
  if (capacity > kFewSlots) {
    lists.keys = reinterpret_cast<unsigned*>(take(pairs * lists.slots * 4));
    lists.positions = reinterpret_cast<unsigned*>(take(pairs * lists.slots * 4));
    lists.hist = reinterpret_cast<unsigned*>(take(pairs * 3 * kBins * 4));
    lists.state = reinterpret_cast<EvictState*>(take(pairs * 3 * sizeof(EvictState)));
    lists.part = reinterpret_cast<PartRecord*>(take(pairs * lists.parts * sizeof(PartRecord)));
  }
  return at + 16;
}

}  // namespace

size_t evict_workspace_bytes(int B, int heads, long long capacity, int budget) {
  EvictLists lists{};
  return lay_out(lists, nullptr, static_cast<long long>(B) * heads, capacity, budget);
}

hipError_t launch_kv_evict(const EvictArgs& a, const KvArgs& c, int dtype) {
  const long long pairs = static_cast<long long>(a.B) * c.heads;
  const long long cap = static_cast<long long>(c.max_pages) * c.page_size;
  const int esize = dtype == 0 ? 4 : 2;
  EvictLists lists{};
  lay_out(lists, static_cast<char*>(a.workspace), pairs, cap, a.budget);
  lists.magic = static_cast<unsigned>((1ull << 32) / static_cast<unsigned>(c.dim * esize / 8) + 1);
  // (new_len in kv_len's place is written when all workgroups have read kv_len)
  lists.own_moves = cap <= kFewSlots && lists.most <= kOwnMoves && a.new_len != a.kv_len;
  const unsigned rows = static_cast<unsigned>(pairs < 65535 ? pairs : 65535);
  if (cap <= kFewSlots) {
    if (c.page_size % 4 == 0)
      evict_select_kernel<true><<<rows, 64 * kFewWaves, 0, a.stream>>>(a, c, lists, esize);
    else
      evict_select_kernel<false><<<rows, 64 * kFewWaves, 0, a.stream>>>(a, c, lists, esize);
  } else {
    const dim3 grid(lists.parts, rows);
    c.page_size % 4 == 0 ? launch_parts<true>(a, c, lists, grid) : launch_parts<false>(a, c, lists, grid);
  }
  if (!lists.own_moves) {
    // About 16384 waves, or as many as there can be batches.
    const long long need = (lists.most + kMoveWaves * kMoveBatch - 1) / (kMoveWaves * kMoveBatch);
    long long chunks = 4096 / pairs;
    if (chunks > need) chunks = need;
    if (chunks < 1) chunks = 1;
    const dim3 grid(static_cast<unsigned>(chunks), rows);
    evict_move_kernel<<<grid, 64 * kMoveWaves, 0, a.stream>>>(a, c, lists, esize);
  }
  return hipGetLastError();
}

}  // namespace specdec
