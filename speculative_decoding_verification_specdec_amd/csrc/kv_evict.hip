// gfx950 kernels of the eviction by accumulated attention weight.
//
// Of a (sequence, kv head)'s L slots the `budget` ones with the largest keys stay; a key is the order
// of the weight as an unsigned number, with protected positions above all.  The select kernel (one
// workgroup per sequence and head) finds the budget-th largest key by a radix search, 8 bits a pass,
// then walks over the slots in order and lists the kept slots from `budget` on (movers) and the
// evicted ones below it (holes).  There are as many of one as of the other; the move kernel copies
// mover i over hole i.  Sources lie at or above `budget` and destinations below it, so the copies are
// independent of each other.
#include <hip/hip_runtime.h>

#include "paged.h"

namespace specdec {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kMoveWaves = 4;

// Workspace: per (sequence, head) the number of moves, then the movers and the holes.
struct EvictLists {
  int32_t* count;
  int32_t* from;
  int32_t* to;
  long long most;  // entries per (sequence, head)
};

long long most_moves(long long capacity, int budget) {
  return capacity <= budget ? 0 : capacity - budget < budget ? capacity - budget : budget;
}

size_t count_bytes(long long pairs) { return (static_cast<size_t>(pairs) * 4 + 15) & ~size_t{15}; }

// Unsigned order of a weight: NaN 0, then ascending; -0 and +0 alike.
__device__ __forceinline__ unsigned weight_order(float w) {
  if (w != w) return 0u;
  const unsigned u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ unsigned slot_key(const EvictArgs& a, const KvArgs& c, int b, int h,
                                             int slot, int newest) {
  const long long at = record_at(c, page_of(c, b, slot), slot % c.page_size, h);
  const int p = c.position[at];
  if (p < a.keep_first || p > static_cast<long long>(newest) - a.keep_last) return 0xffffffffu;
  return weight_order(c.weight[at]);
}

__global__ __launch_bounds__(kSelThreads) void evict_select_kernel(EvictArgs a, KvArgs c,
                                                                   EvictLists lists) {
  __shared__ unsigned sh_hist[256];
  __shared__ int sh_scan[3][kSelWaves];
  __shared__ int sh_newest, sh_bad, sh_digit, sh_left;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const long long cap = static_cast<long long>(c.max_pages) * c.page_size;
  const long long pairs = static_cast<long long>(a.B) * c.heads;
  for (long long bh = blockIdx.x; bh < pairs; bh += gridDim.x) {
    const int b = static_cast<int>(bh / c.heads), h = static_cast<int>(bh - (bh / c.heads) * c.heads);
    const int L = a.kv_len[b];
    __syncthreads();
    if (L < 0 || L > cap || L <= a.budget) {
      if (tid == 0) lists.count[bh] = L < 0 || L > cap ? -1 : 0;
      continue;
    }
    if (tid == 0) {
      sh_newest = -0x7fffffff - 1;
      sh_bad = 0;
    }
    __syncthreads();
    int newest = -0x7fffffff - 1;
    for (int s = tid; s < L; s += kSelThreads) {
      const int page = page_of(c, b, s);
      if (page < 0)
        sh_bad = 1;
      else
        newest = max(newest, c.position[record_at(c, page, s % c.page_size, h)]);
    }
    atomicMax(&sh_newest, newest);
    __syncthreads();
    if (sh_bad) {
      if (tid == 0) lists.count[bh] = -1;
      continue;
    }
    newest = sh_newest;
    // The budget-th largest key, from its highest byte down; `left` of the slots with it are kept.
    unsigned prefix = 0;
    int left = a.budget;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) sh_hist[tid] = 0;
      __syncthreads();
      for (int s = tid; s < L; s += kSelThreads) {
        const unsigned key = slot_key(a, c, b, h, s, newest);
        if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&sh_hist[(key >> shift) & 255], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255, n = left;
        while (d > 0 && n > static_cast<int>(sh_hist[d])) n -= sh_hist[d--];
        sh_digit = d;
        sh_left = n;
      }
      __syncthreads();
      prefix |= static_cast<unsigned>(sh_digit) << shift;
      left = sh_left;
    }
    // Movers and holes in ascending order.
    int ties = 0, movers = 0, holes = 0;  // before this tile
    for (int s0 = 0; s0 < L; s0 += kSelThreads) {
      const int s = s0 + tid;
      const unsigned key = s < L ? slot_key(a, c, b, h, s, newest) : 0u;
      const bool tie = s < L && key == prefix;
      const unsigned long long tie_mask = __ballot(tie);
      if (lane == 0) sh_scan[0][wave] = __popcll(tie_mask);
      __syncthreads();
      int rank = ties + __popcll(tie_mask & ((1ull << lane) - 1));
      for (int w = 0; w < kSelWaves; ++w) {
        if (w < wave) rank += sh_scan[0][w];
        ties += sh_scan[0][w];
      }
      const bool kept = s < L && (key > prefix || (tie && rank < left));
      const bool mover = kept && s >= a.budget, hole = s < L && !kept && s < a.budget;
      const unsigned long long mover_mask = __ballot(mover), hole_mask = __ballot(hole);
      if (lane == 0) {
        sh_scan[1][wave] = __popcll(mover_mask);
        sh_scan[2][wave] = __popcll(hole_mask);
      }
      __syncthreads();
      int mover_rank = movers + __popcll(mover_mask & ((1ull << lane) - 1));
      int hole_rank = holes + __popcll(hole_mask & ((1ull << lane) - 1));
      for (int w = 0; w < kSelWaves; ++w) {
        if (w < wave) {
          mover_rank += sh_scan[1][w];
          hole_rank += sh_scan[2][w];
        }
        movers += sh_scan[1][w];
        holes += sh_scan[2][w];
      }
      if (mover) lists.from[bh * lists.most + mover_rank] = s;
      if (hole) lists.to[bh * lists.most + hole_rank] = s;
    }
    if (tid == 0) lists.count[bh] = movers;
  }
}

template <int kEsize>
__global__ __launch_bounds__(64 * kMoveWaves) void evict_move_kernel(EvictArgs a, KvArgs c,
                                                                     EvictLists lists) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long pairs = static_cast<long long>(a.B) * c.heads;
  const int vectors = c.dim * kEsize / 16;  // 16-byte vectors a row
  for (long long bh = blockIdx.y; bh < pairs; bh += gridDim.y) {
    const int b = static_cast<int>(bh / c.heads), h = static_cast<int>(bh - (bh / c.heads) * c.heads);
    const int n = lists.count[bh];
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0 && a.new_len)
      a.new_len[b] = n < 0 ? -1 : min(a.kv_len[b], a.budget);
    for (int i = blockIdx.x * kMoveWaves + wave; i < n; i += gridDim.x * kMoveWaves) {
      const int s = lists.from[bh * lists.most + i], d = lists.to[bh * lists.most + i];
      const int sp = page_of(c, b, s), dp = page_of(c, b, d);
      const int so = s % c.page_size, dof = d % c.page_size;
      const long long src = row_at(c, sp, so, h) * kEsize, dst = row_at(c, dp, dof, h) * kEsize;
      for (int x = lane; x < 2 * vectors; x += 64) {
        char* pool = x < vectors ? c.k : c.v;
        const int at = 16 * (x < vectors ? x : x - vectors);
        *reinterpret_cast<int4*>(pool + dst + at) = *reinterpret_cast<const int4*>(pool + src + at);
      }
      if (lane == 0) {
        const long long from = record_at(c, sp, so, h), to = record_at(c, dp, dof, h);
        c.weight[to] = c.weight[from];
        c.position[to] = c.position[from];
      }
    }
  }
}

}  // namespace

size_t evict_workspace_bytes(int B, int heads, long long capacity, int budget) {
  const long long pairs = static_cast<long long>(B) * heads;
  return count_bytes(pairs) + static_cast<size_t>(pairs) * most_moves(capacity, budget) * 8 + 16;
}

hipError_t launch_kv_evict(const EvictArgs& a, const KvArgs& c, int dtype) {
  const long long pairs = static_cast<long long>(a.B) * c.heads;
  EvictLists lists;
  lists.most = most_moves(static_cast<long long>(c.max_pages) * c.page_size, a.budget);
  lists.count = static_cast<int32_t*>(a.workspace);
  lists.from = reinterpret_cast<int32_t*>(static_cast<char*>(a.workspace) + count_bytes(pairs));
  lists.to = lists.from + pairs * lists.most;
  evict_select_kernel<<<static_cast<unsigned>(pairs < (1 << 20) ? pairs : 1 << 20), kSelThreads, 0,
                        a.stream>>>(a, c, lists);
  long long chunks = (lists.most + kMoveWaves - 1) / kMoveWaves;
  if (chunks > 64) chunks = 64;
  if (chunks < 1) chunks = 1;
  const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(pairs < 65535 ? pairs : 65535));
  if (dtype == 0)
    evict_move_kernel<4><<<grid, 64 * kMoveWaves, 0, a.stream>>>(a, c, lists);
  else
    evict_move_kernel<2><<<grid, 64 * kMoveWaves, 0, a.stream>>>(a, c, lists);
  return hipGetLastError();
}

}  // namespace specdec
