// gfx950 kernels of the eviction by accumulated attention weight.
//
// Of a (sequence, kv head)'s L slots the `budget` ones with the largest keys stay; a key is the order of the weight
// as an unsigned number, with protected positions above all.  One workgroup per sequence and head reads the records
// once, finds the budget-th largest key by a radix search (11, 11 and 10 bits) over keys that it keeps in LDS, or in
// the workspace where the cache can hold more slots than fit, and then walks over them in order.  A slot's rank is
// what decides:  with G(s) and T(s) the slots before s that lie above the threshold key and at it, and `left` the
// number at it that stay,
//   kept before s = G(s) + min(T(s), left),
// which is the place among the holes of an evicted slot s < budget (s - kept before s) and, counted from the end, of
// a kept slot s >= budget among the movers.  There are as many of one as of the other, and mover i is copied over
// hole i.  Sources lie at or above `budget` and destinations below it, so the copies are independent of each other.
//
// Bound: for a full cache that gives up a round's slots the latency of one workgroup's passes (the records are 8
// bytes a slot); for a deep cut the rows that move.
#include <hip/hip_runtime.h>

#include "paged.h"
#include "paged_tiles.h"
#include "wave_ops.h"

namespace specdec {
namespace {

constexpr int kGroup = 256;        // slots a wave takes at once, four a lane
constexpr int kLdsSlots = 8192;    // keys and positions in LDS up to so many: 64 KiB, two workgroups a CU
constexpr int kBins = 2048;
constexpr int kMoveWaves = 4;
constexpr int kMoveBatch = 16;     // rows that a wave moves at once
// The select kernel's workgroup moves the rows itself where there cannot be more than these: a second launch would
// take longer.
constexpr int kOwnMoves = 256;

// Workspace: per (sequence, head) the number of moves, the movers and the holes; where LDS is too small also keys and
// positions.
struct EvictLists {
  int32_t* count;
  int32_t* from;     // the movers, at the end of `most` places
  int32_t* to;       // the holes, from the first place on
  long long most;    // entries per (sequence, head)
  unsigned* keys;    // [2][slots] per (sequence, head)
  long long slots;   // capacity rounded up to whole groups
  int own_moves;     // the select kernel moves the rows and writes new_len
  unsigned magic;    // 2^32 / (16-byte vectors of a row of k and v) rounded up
};

long long most_moves(long long capacity, int budget) {
  return capacity <= budget ? 0 : capacity - budget < budget ? capacity - budget : budget;
}
long long whole_groups(long long capacity) { return (capacity + kGroup - 1) / kGroup * kGroup; }

size_t align16(size_t x) { return (x + 15) & ~size_t{15}; }

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

// Counts a digit; a wave whose lanes all have the same one (zero weights, protected slots) adds them at once.
__device__ __forceinline__ void count_digit(unsigned* hist, unsigned digit, bool active, int lane) {
  const unsigned long long who = __ballot(active);
  if (who == 0) return;
  const int leader = __builtin_ctzll(who);
  const unsigned first = __builtin_amdgcn_readlane(digit, leader);
  if (__ballot(active && digit == first) == who) {
    if (lane == leader) atomicAdd(&hist[first], static_cast<unsigned>(__popcll(who)));
  } else if (active) {
    atomicAdd(&hist[digit], 1u);
  }
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
      const uintptr_t pool = reinterpret_cast<uintptr_t>(z < vectors ? c.k : c.v) + 16 * (z < vectors ? z : z - vectors);
      to[y] = (Rows)(pool + shfl64(dst, m));
      data[y] = *(Rows)(pool + shfl64(src, m));
    }
#pragma unroll
    for (int y = 0; y < kFlight; ++y)
      if (x0 + 64 * y + lane < all) *to[y] = data[y];
  }
}

// Threads of a workgroup.  Few slots: a pair has little work and there are many of them, two or three a CU.
constexpr int select_threads(bool lds) { return lds ? 512 : 1024; }

// kLds: keys and positions of all slots lie in LDS.  kQuad: four slots from a multiple of four on lie in one page.
template <bool kLds, bool kQuad>
__global__ __launch_bounds__(select_threads(kLds), 4) void evict_select_kernel(EvictArgs a, KvArgs c,
                                                                               EvictLists lists, int esize) {
  constexpr int kThreads = select_threads(kLds), kWaves = kThreads / 64, kMine = kBins / kThreads;
  extern __shared__ u32x4 sh_slots[];  // [2][lists.slots / 4]
  __shared__ unsigned sh_hist[kBins];
  __shared__ int sh_wave[2][kWaves];
  __shared__ int sh_digit, sh_left;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const long long cap = static_cast<long long>(c.max_pages) * c.page_size;
  const long long pairs = static_cast<long long>(a.B) * c.heads;
  typedef int Int4 __attribute__((ext_vector_type(4), aligned(4)));
  typedef float Float4 __attribute__((ext_vector_type(4), aligned(4)));
  for (long long bh = blockIdx.x; bh < pairs; bh += gridDim.x) {
    const int b = static_cast<int>(bh / c.heads), h = static_cast<int>(bh - (bh / c.heads) * c.heads);
    const int L = a.kv_len[b];
    const bool wrong = L < 0 || L > cap;
    __syncthreads();  // (LDS of the pair before)
    if (wrong || L <= a.budget) {
      if (tid == 0) lists.count[bh] = wrong ? -1 : 0;
      if (tid == 0 && lists.own_moves && h == 0 && a.new_len) a.new_len[b] = wrong ? -1 : L;
      continue;
    }
    u32x4* keys;
    if constexpr (kLds)
      keys = sh_slots;
    else
      keys = reinterpret_cast<u32x4*>(lists.keys + 2 * bh * lists.slots);
    u32x4* positions = keys + lists.slots / 4;
    // Every wave has a run of groups; all passes take the same slots in the same lanes.
    const int groups = (L + kGroup - 1) / kGroup;
    const int g0 = static_cast<int>(static_cast<long long>(groups) * wave / kWaves);
    const int g1 = static_cast<int>(static_cast<long long>(groups) * (wave + 1) / kWaves);
    const int32_t* table = c.table + static_cast<long long>(b) * c.max_pages;

    // Records to keys and positions, four groups on their way at once.
    int newest = -0x7fffffff - 1;
    bool bad = false;
    for (int gi = g0; gi < g1; gi += 4) {
      int page[4][kQuad ? 1 : 4];
      long long at[4][kQuad ? 1 : 4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int j = 0; j < (kQuad ? 1 : 4); ++j) {
          const int s = min(min(gi + u, g1 - 1) * kGroup + 4 * lane, (L - 1) & ~3) + j;
          const int idx = s / c.page_size;
          at[u][j] = s - idx * c.page_size;
          page[u][j] = table[min(s, L - 1) / c.page_size];
        }
      u32x4 order[4], pos[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if constexpr (kQuad) {
          const bool good = static_cast<unsigned>(page[u][0]) < static_cast<unsigned>(c.num_pages);
          bad = bad || !good;
          const long long r = record_at(c, good ? page[u][0] : 0, static_cast<int>(at[u][0]), h);
          pos[u] = __builtin_bit_cast(u32x4, *reinterpret_cast<const Int4*>(c.position + r));
          order[u] = __builtin_bit_cast(u32x4, *reinterpret_cast<const Float4*>(c.weight + r));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool good = static_cast<unsigned>(page[u][j]) < static_cast<unsigned>(c.num_pages);
            bad = bad || !good;
            const int s = min(min(gi + u, g1 - 1) * kGroup + 4 * lane, (L - 1) & ~3) + j;
            const long long r = record_at(c, good ? page[u][j] : 0, s < L ? static_cast<int>(at[u][j]) : 0, h);
            pos[u][j] = static_cast<unsigned>(c.position[r]);
            order[u][j] = __float_as_uint(c.weight[r]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (gi + u >= g1) break;
        const int s = (gi + u) * kGroup + 4 * lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int p = static_cast<int>(pos[u][j]);
          if (s + j < L) newest = max(newest, p);
          order[u][j] = p < a.keep_first ? 0xffffffffu : weight_order(__uint_as_float(order[u][j]));
        }
        keys[(gi + u) * 64 + lane] = order[u];
        positions[(gi + u) * 64 + lane] = pos[u];
      }
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) newest = max(newest, __shfl_xor(newest, off, 64));
    bad = __any(bad);
    if (lane == 0) {
      sh_wave[0][wave] = newest;
      sh_wave[1][wave] = bad;
    }
    for (int x = tid; x < kBins; x += kThreads) sh_hist[x] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      newest = max(newest, sh_wave[0][w]);
      bad = bad || sh_wave[1][w] != 0;
    }
    if (bad) {
      if (tid == 0) lists.count[bh] = -1;
      if (tid == 0 && lists.own_moves && h == 0 && a.new_len) a.new_len[b] = -1;
      continue;
    }
    const long long recent = static_cast<long long>(newest) - a.keep_last;

    // The budget-th largest key, from its highest bits down; `left` of the slots with it are kept.
    unsigned prefix = 0;
    int left = a.budget;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const unsigned above = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
      const unsigned bits = pass == 2 ? 1023u : 2047u;
      for (int gi = g0; gi < g1; gi += 2) {
        u32x4 key[2], pos[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int x = min(gi + u, g1 - 1) * 64 + lane;
          key[u] = keys[x];
          if (pass == 0) pos[u] = positions[x];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (gi + u >= g1) break;
          const int s = (gi + u) * kGroup + 4 * lane;
          if (pass == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (static_cast<int>(pos[u][j]) > recent) key[u][j] = 0xffffffffu;
            keys[(gi + u) * 64 + lane] = key[u];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            count_digit(sh_hist, key[u][j] >> shift & bits, s + j < L && (key[u][j] & above) == prefix, lane);
        }
      }
      __syncthreads();
      // Counts from the highest digit down: a thread has a few digits, and exactly one of all reaches `left`.
      const int top = kBins - 1 - kMine * tid;
      int n[kMine], mine = 0;
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        n[x] = static_cast<int>(sh_hist[top - x]);
        sh_hist[top - x] = 0;
        mine += n[x];
      }
      const int upto = wave_scan(mine);
      if (lane == 63) sh_wave[0][wave] = upto;
      __syncthreads();
      int before = upto - mine;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) before += w < wave ? sh_wave[0][w] : 0;
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        if (before < left && left <= before + n[x]) {
          sh_digit = top - x;
          sh_left = left - before;
        }
        before += n[x];
      }
      __syncthreads();
      prefix |= static_cast<unsigned>(sh_digit) << shift;
      left = sh_left;
    }

    // Slots above the threshold and at it before each wave's.
    int above = 0, ties = 0;
    for (int gi = g0; gi < g1; ++gi) {
      const u32x4 key = keys[gi * 64 + lane];
      const int s = gi * kGroup + 4 * lane;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        above += __popcll(__ballot(s + j < L && key[j] > prefix));
        ties += __popcll(__ballot(s + j < L && key[j] == prefix));
      }
    }
    if (lane == 0) {
      sh_wave[0][wave] = above;
      sh_wave[1][wave] = ties;
    }
    __syncthreads();
    above = ties = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      above += w < wave ? sh_wave[0][w] : 0;
      ties += w < wave ? sh_wave[1][w] : 0;
    }
    __syncthreads();
    for (int gi = g0; gi < g1; ++gi) {
      const u32x4 key = keys[gi * 64 + lane];
      const int s = gi * kGroup + 4 * lane;
      int mine = 0;  // above and (from bit 16 on) at the threshold
#pragma unroll
      for (int j = 0; j < 4; ++j)
        mine += s + j >= L ? 0 : key[j] > prefix ? 1 : key[j] == prefix ? 0x10000 : 0;
      const int upto = wave_scan(mine);
      int g = above + ((upto - mine) & 0xffff), t = ties + ((upto - mine) >> 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = s + j < L, tie = key[j] == prefix;
        const bool kept = key[j] > prefix || (tie && t < left);
        const int before = g + min(t, left);
        if (in && kept && s + j >= a.budget)
          lists.from[bh * lists.most + lists.most - a.budget + before] = s + j;
        if (in && !kept && s + j < a.budget) lists.to[bh * lists.most + s + j - before] = s + j;
        // (the slots below the budget that stay: as many as are not moved to)
        if (s + j == a.budget - 1) sh_left = before + kept;
        g += key[j] > prefix;
        t += tie;
      }
      const int all = __builtin_amdgcn_readlane(upto, 63);
      above += all & 0xffff;
      ties += all >> 16;
    }
    __syncthreads();
    const int moves = a.budget - sh_left;
    if (tid == 0) lists.count[bh] = moves;
    if (lists.own_moves) {
      if (tid == 0 && h == 0 && a.new_len) a.new_len[b] = a.budget;
      for (int i = wave * kMoveBatch; i < moves; i += kWaves * kMoveBatch)
        move_rows<2>(c, lists, bh, b, h, esize, moves, i, min(kMoveBatch, moves - i), lane);
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

template <bool kLds>
void launch_select(const EvictArgs& a, const KvArgs& c, const EvictLists& lists, unsigned groups, int esize) {
  const size_t lds = kLds ? 8 * lists.slots : 0;
  if (c.page_size % 4 == 0)
    evict_select_kernel<kLds, true><<<groups, select_threads(kLds), lds, a.stream>>>(a, c, lists, esize);
  else
    evict_select_kernel<kLds, false><<<groups, select_threads(kLds), lds, a.stream>>>(a, c, lists, esize);
}

}  // namespace

size_t evict_workspace_bytes(int B, int heads, long long capacity, int budget) {
  const long long pairs = static_cast<long long>(B) * heads, slots = whole_groups(capacity);
  return align16(pairs * 4) + align16(static_cast<size_t>(pairs) * most_moves(capacity, budget) * 8) +
         (slots > kLdsSlots ? static_cast<size_t>(pairs) * slots * 8 : 0) + 16;
}

hipError_t launch_kv_evict(const EvictArgs& a, const KvArgs& c, int dtype) {
  const long long pairs = static_cast<long long>(a.B) * c.heads;
  const long long cap = static_cast<long long>(c.max_pages) * c.page_size;
  const int esize = dtype == 0 ? 4 : 2;
  EvictLists lists;
  lists.most = most_moves(cap, a.budget);
  lists.slots = whole_groups(cap);
  char* ws = static_cast<char*>(a.workspace);
  lists.count = reinterpret_cast<int32_t*>(ws);
  ws += align16(pairs * 4);
  lists.from = reinterpret_cast<int32_t*>(ws);
  lists.to = lists.from + pairs * lists.most;
  lists.keys = reinterpret_cast<unsigned*>(ws + align16(static_cast<size_t>(pairs) * lists.most * 8));
  lists.magic = static_cast<unsigned>((1ull << 32) / static_cast<unsigned>(c.dim * esize / 8) + 1);
  // (new_len in kv_len's place is written when all workgroups have read kv_len)
  const uintptr_t len = reinterpret_cast<uintptr_t>(a.kv_len), out = reinterpret_cast<uintptr_t>(a.new_len);
  const uintptr_t size = static_cast<uintptr_t>(a.B) * 4;
  lists.own_moves = lists.most <= kOwnMoves && (!a.new_len || out + size <= len || len + size <= out);
  const unsigned groups = static_cast<unsigned>(pairs < (1 << 20) ? pairs : 1 << 20);
  if (lists.slots <= kLdsSlots)
    launch_select<true>(a, c, lists, groups, esize);
  else
    launch_select<false>(a, c, lists, groups, esize);
  if (!lists.own_moves) {
    // About 16384 waves, or as many as there can be batches.
    const long long need = (lists.most + kMoveWaves * kMoveBatch - 1) / (kMoveWaves * kMoveBatch);
    long long chunks = 4096 / pairs;
    if (chunks > need) chunks = need;
    if (chunks < 1) chunks = 1;
    const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(pairs < 65535 ? pairs : 65535));
    evict_move_kernel<<<grid, 64 * kMoveWaves, 0, a.stream>>>(a, c, lists, esize);
  }
  return hipGetLastError();
}

}  // namespace specdec
