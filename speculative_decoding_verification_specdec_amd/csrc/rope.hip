// gfx950 kernel of the rotary positions and the append to the paged cache.
//
// Pair i of a head turns by t = position * inv_freq[i]:
//   a' = s (a cos t - b sin t),   b' = s (b cos t + a sin t).
// Positions of long contexts reach 2^20 and more, where an f32 angle is off by whole hundredths of a
// turn, so the angle is formed in f64 in turns, its whole turns are taken off there, and only the rest
// (at most half a turn) goes to f32.
//
// One wave takes one token.  A lane owns a "unit" of a head, 16 bytes or the two 16-byte halves that
// turn together, and walks over heads with it, 64 / units heads at a time: its cosines and sines stay
// in registers for all of them.  With few tokens the heads are spread over more waves instead.
// The work is bound by bytes: each element is read once and written once.  8 x 4096 tokens of 32 + 2 x 8 heads of 128,
// float16: 152 us, 5.3 TB/s, where a copy of 2 GiB reaches 4.9.
#include <hip/hip_runtime.h>

#include "paged.h"

namespace specdec {
namespace {

constexpr int kRopeWaves = 4;  // waves per workgroup

template <typename T>
struct alignas(16) Chunk {
  static constexpr int kCount = 16 / sizeof(T);
  T x[kCount];
};

// cos and sin of 2 pi (position * turns_per_position), times scale.
__device__ __forceinline__ void turn_of(double position, double freq, float scale, float& c,
                                        float& s) {
  constexpr double kPerTurn = 0.15915494309189533577;  // 1 / (2 pi)
  double t = position * (freq * kPerTurn);
  t -= rint(t);
  sincospif(2.f * static_cast<float>(t), &s, &c);
  c *= scale;
  s *= scale;
}

template <typename T>
__device__ __forceinline__ void turn_pair(T& a, T& b, float c, float s) {
  const float x = to_float(a), y = to_float(b);
  a = from_float<T>(x * c - y * s);
  b = from_float<T>(y * c + x * s);
}

// One head's row of the token: where it is read and where it goes.
template <typename T>
struct HeadRow {
  const T* src;
  T* dst;
  bool turned;
};

template <typename T>
__device__ __forceinline__ HeadRow<T> head_row(const RopeArgs& a, const KvArgs& c, long long token,
                                               int head, int page, int off) {
  HeadRow<T> r;
  if (head < a.q_heads) {
    r.src = static_cast<const T*>(a.q) + token * a.q_stride + head * static_cast<long long>(c.dim);
    r.dst = static_cast<T*>(a.q_out) + (token * a.q_heads + head) * c.dim;
    r.turned = true;
    return r;
  }
  head -= a.q_heads;
  if (head < c.heads) {
    r.src = static_cast<const T*>(a.k) + token * a.k_stride + head * static_cast<long long>(c.dim);
    r.dst = reinterpret_cast<T*>(c.k) + row_at(c, page, off, head);
    r.turned = true;
    return r;
  }
  head -= c.heads;
  r.src = static_cast<const T*>(a.v) + token * a.v_stride + head * static_cast<long long>(c.dim);
  r.dst = reinterpret_cast<T*>(c.v) + row_at(c, page, off, head);
  r.turned = false;
  return r;
}

enum RopeLayout { kHalves = 0, kAdjacent = 1, kScalar = 2 };

// `units` lanes hold one head's row and `per_pass` heads go through a wave at once; a wave does
// `per_wave` such passes of one token.  kScalar: one pair or one element a lane, one head at a time.
template <typename T, int kLayout>
__global__ __launch_bounds__(64 * kRopeWaves) void rope_append_kernel(RopeArgs a, KvArgs c,
                                                                      int units, int per_pass,
                                                                      int passes, int per_wave) {
  constexpr int E = Chunk<T>::kCount;
  const int lane = threadIdx.x & 63;
  const int splits = (passes + per_wave - 1) / per_wave;
  const long long tokens = static_cast<long long>(a.B) * (a.K + 1);
  const int half = a.rotary / 2;
  const int all_heads = a.q_heads + 2 * c.heads;
  for (long long w = static_cast<long long>(blockIdx.x) * kRopeWaves + (threadIdx.x >> 6);
       w < tokens * splits; w += static_cast<long long>(gridDim.x) * kRopeWaves) {
    // (tokens < 2^31, and there are splits only of a few thousand: 32 bits)
    const unsigned t = static_cast<unsigned>(w) / static_cast<unsigned>(splits);
    const int split = static_cast<int>(static_cast<unsigned>(w) - t * splits);
    const long long token = t;
    const int b = static_cast<int>(t / static_cast<unsigned>(a.K + 1));
    const int i = static_cast<int>(t - static_cast<unsigned>(b) * (a.K + 1));
    const RoundRows r = round_rows(c, a.num_draft, a.kv_len, b, a.K);
    const long long pos = static_cast<long long>(a.first_pos[b]) + i;
    const int first_head = split * per_wave * per_pass;
    const int end_head = min(all_heads, first_head + per_wave * per_pass);
    bool good = r.n > 0 && pos - i >= 0 && pos - i + r.n - 1 <= 0x7fffffffLL;
    const bool used = i < r.rows;
    int page = 0, off = 0;
    if (good && used) {
      const int slot = r.len + i;
      page = page_of(c, b, slot);
      off = slot % c.page_size;
      good = page >= 0;
    }
    if (!used || !good) {  // rows past the last new token are 0, an invalid sequence's rows NaN
      const T fill = from_float<T>(used ? __builtin_nanf("") : 0.f);
      for (int h = first_head; h < min(end_head, a.q_heads); ++h) {
        T* dst = static_cast<T*>(a.q_out) + (token * a.q_heads + h) * c.dim;
        for (int d = lane; d < c.dim; d += 64) dst[d] = fill;
      }
      continue;
    }
    if (kLayout == kScalar) {
      for (int u = lane; u < units; u += 64) {
        float cs = 1.f, sn = 0.f;
        if (u < half) turn_of(static_cast<double>(pos), a.inv_freq[u], a.scale, cs, sn);
        for (int h = first_head; h < end_head; ++h) {
          const HeadRow<T> row = head_row<T>(a, c, token, h, page, off);
          if (u >= half) {
            row.dst[u + half] = row.src[u + half];
          } else {
            T x = row.src[u], y = row.src[u + half];
            if (row.turned) turn_pair(x, y, cs, sn);
            row.dst[u] = x;
            row.dst[u + half] = y;
          }
        }
      }
    } else {
      const int hs = lane / units, u = lane - hs * units;
      const bool active = hs < per_pass;
      // Pairs of this lane, the first element of its one or two chunks, and whether it has two.
      constexpr int P = kLayout == kHalves ? E : E / 2;
      const bool two = kLayout == kHalves && u * E < half;
      const int at = kLayout == kAdjacent || two ? u * E : a.rotary + u * E - half;
      const int pair0 = u * P;
      float cs[P], sn[P];
#pragma unroll
      for (int e = 0; e < P; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
        if (active && pair0 + e < half)
          turn_of(static_cast<double>(pos), a.inv_freq[pair0 + e], a.scale, cs[e], sn[e]);
      }
      for (int h = first_head + hs; active && h < end_head; h += per_pass) {
        const HeadRow<T> row = head_row<T>(a, c, token, h, page, off);
        Chunk<T> x = *reinterpret_cast<const Chunk<T>*>(row.src + at), y;
        if (two) y = *reinterpret_cast<const Chunk<T>*>(row.src + at + half);
        if (row.turned) {
#pragma unroll
          for (int e = 0; e < P; ++e) {
            if (kLayout == kHalves) {
              if (two) turn_pair(x.x[e], y.x[e], cs[e], sn[e]);
            } else if (pair0 + e < half) {
              turn_pair(x.x[2 * e], x.x[2 * e + 1], cs[e], sn[e]);
            }
          }
        }
        *reinterpret_cast<Chunk<T>*>(row.dst + at) = x;
        if (two) *reinterpret_cast<Chunk<T>*>(row.dst + at + half) = y;
      }
    }
    // The slot's record, by the wave that holds the first head of all.
    if (split == 0) {
      for (int h = lane; h < c.heads; h += 64) {
        const long long at = record_at(c, page, off, h);
        if (c.weight) c.weight[at] = 0.f;
        if (c.position) c.position[at] = static_cast<int32_t>(pos);
      }
    }
  }
}

template <typename T>
hipError_t launch_rope_type(const RopeArgs& a, const KvArgs& c) {
  constexpr int E = Chunk<T>::kCount;
  const int half = a.rotary / 2;
  // 16-byte chunks hold whole pairs when the pairs are adjacent, and meet whole partner chunks when
  // half the rotated width is a multiple of a chunk; other widths go element by element.
  const int layout = a.interleaved ? kAdjacent : half % E == 0 ? kHalves : kScalar;
  const int units = layout == kScalar   ? a.rotary / 2 + c.dim - a.rotary
                    : layout == kHalves ? half / E + (c.dim - a.rotary) / E
                                        : c.dim / E;
  const int per_pass = layout == kScalar ? 1 : 64 / units;
  const int all_heads = a.q_heads + 2 * c.heads;
  const int passes = (all_heads + per_pass - 1) / per_pass;
  const long long tokens = static_cast<long long>(a.B) * (a.K + 1);
  // Few tokens: as many waves a token as it takes to have 4096 of them (16 a CU) in flight (one token of 48 heads
  // 6.5 us, 8.4 in one wave; 384 tokens 7.6 and 8.8).
  long long splits = (4096 + tokens - 1) / tokens;
  if (splits > passes) splits = passes;
  const int per_wave = static_cast<int>((passes + splits - 1) / splits);
  splits = (passes + per_wave - 1) / per_wave;
  const long long groups = (tokens * splits + kRopeWaves - 1) / kRopeWaves;
  const dim3 grid(static_cast<unsigned>(groups < (1 << 22) ? groups : 1 << 22));
  const dim3 block(64 * kRopeWaves);
  if (layout == kHalves)
    rope_append_kernel<T, kHalves><<<grid, block, 0, a.stream>>>(a, c, units, per_pass, passes, per_wave);
  else if (layout == kAdjacent)
    rope_append_kernel<T, kAdjacent><<<grid, block, 0, a.stream>>>(a, c, units, per_pass, passes, per_wave);
  else
    rope_append_kernel<T, kScalar><<<grid, block, 0, a.stream>>>(a, c, units, per_pass, passes, per_wave);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, const KvArgs& c, int dtype) {
  if (dtype == 0) return launch_rope_type<float>(a, c);
  if (dtype == 1) return launch_rope_type<__bf16>(a, c);
  return launch_rope_type<_Float16>(a, c);
}

}  // namespace specdec
