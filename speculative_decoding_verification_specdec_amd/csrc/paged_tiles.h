// Matrix tiles over the paged cache, shared by the attention and the weights kernels.
//
// A wave takes kKeys slots of one kv head and 16-row groups of query rows.  Scores come transposed,
//   S^T [slots x rows] = K [slots x dim] . Q^T [dim x rows],
// so that a lane's four results belong to one row (its column lane % 16) and to the slots
// 4 (lane / 16) + r: statistics of a row stay in a lane and its three partners 16 lanes apart, and the
// results are already where the second product wants them,
//   O^T [dim x rows] = V^T [dim x slots] . P^T [slots x rows],
// whose operand takes the slots of a lane's group in any order that both sides share.
//
// Operands go straight from memory into registers, each byte of the cache once: an instruction's 64
// lanes read 16 keys x 64 bytes (K) or 4 whole rows of V.  V's operand needs one dim of eight slots in a
// lane while a lane has loaded eight dims of each of its eight slots: the 8 x 8 block is turned within
// the lane by byte permutes, 32 of them a tile, so neither LDS nor a shuffle lies on the way.
#pragma once

#include <hip/hip_runtime.h>

#include "paged.h"
#include "wave_ops.h"

namespace specdec {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

template <typename T>
struct Half8;
template <>
struct Half8<__bf16> {
  typedef __bf16 type __attribute__((ext_vector_type(8)));
  typedef __bf16 pair __attribute__((ext_vector_type(2)));
};
template <>
struct Half8<_Float16> {
  typedef _Float16 type __attribute__((ext_vector_type(8)));
  typedef _Float16 pair __attribute__((ext_vector_type(2)));
};

__device__ __forceinline__ f32x4 mma16(const u32x4& a, const u32x4& b, const f32x4& c, __bf16) {
  typedef Half8<__bf16>::type H;
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(H, a), __builtin_bit_cast(H, b),
                                                 c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma16(const u32x4& a, const u32x4& b, const f32x4& c, _Float16) {
  typedef Half8<_Float16>::type H;
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(H, a), __builtin_bit_cast(H, b),
                                                c, 0, 0, 0);
}
// Four products of depth 4: element e of the lanes' vectors together.
__device__ __forceinline__ f32x4 mma16(const u32x4& a, const u32x4& b, f32x4 c, float) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
  return c;
}

template <typename T>
__device__ __forceinline__ unsigned pack2(float lo, float hi) {
  typedef typename Half8<T>::pair P;
  P p = {static_cast<T>(lo), static_cast<T>(hi)};
  return __builtin_bit_cast(unsigned, p);
}

// Global memory by its own pointer type, so that a base known to be wave-uniform stays scalar.
typedef const __attribute__((address_space(1))) char* GlobalBytes;

// A lane's 32-bit offset as it is where it is used: hoisted out of a loop it would be widened to 64 bits
// there, and the load could not take it beside a scalar base.
__device__ __forceinline__ unsigned lane_offset(unsigned x) {
  asm("" : "+v"(x));
  return x;
}

// A load; kStream: of bytes that nothing reads again (a stream of such loads reaches 7.1-7.3 TB/s on
// MI355X, one of plain loads 6.0-6.4: 4 GiB, any grid from 256 to 16384 workgroups).
template <typename V, bool kStream>
__device__ __forceinline__ V load(GlobalBytes p) {
  typedef const __attribute__((address_space(1))) V* Pointer;
  if constexpr (kStream)
    return __builtin_nontemporal_load((Pointer)p);
  else
    return *(Pointer)p;
}

// Sum over the four lanes 16 apart that share a row (or a slot): each step swaps halves of two copies.
__device__ __forceinline__ float row_sum(float x) {
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const unsigned v = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ long long shfl64(long long x, int src) {
  const int lo = __shfl(static_cast<int>(x), src, 64);
  const int hi = __shfl(static_cast<int>(x >> 32), src, 64);
  return static_cast<long long>(hi) << 32 | static_cast<unsigned>(lo);
}

__device__ __forceinline__ long long read_lane64(long long x, int src) {
  const int lo = __builtin_amdgcn_readlane(static_cast<int>(x), src);
  const int hi = __builtin_amdgcn_readlane(static_cast<int>(x >> 32), src);
  return static_cast<long long>(hi) << 32 | static_cast<unsigned>(lo);
}

// Inclusive sum over the lanes of whole numbers whose sums stay under 2^53: in f64 by moves between neighbouring
// lanes, without a trip to LDS for each step.
__device__ __forceinline__ long long scan_work(long long mine) {
  return static_cast<long long>(wave_inclusive_scan(static_cast<double>(mine)));
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// A wave-uniform pointer as it is, in scalar registers: without this the compiler adds the lanes' offsets
// to its loop-invariant part and keeps a 64-bit vector address for each row.
__device__ __forceinline__ GlobalBytes scalar_base(const void* p) {
  unsigned long long bits = reinterpret_cast<uintptr_t>(p);
  asm("" : "+s"(bits));
  return (GlobalBytes)bits;
}

// A page-table entry at a wave-uniform place, by a scalar load.
__device__ __forceinline__ int table_at(const int32_t* table, long long i) {
  typedef const __attribute__((address_space(4))) int32_t* Scalar;
  return *(Scalar)(reinterpret_cast<uintptr_t>(table + i));
}

// kDim: head_dim rounded up to 64, 128 or 256; kFull: equal to it; else the rest of a
// row is taken as 0.
template <typename T, int kDim, bool kFull>
struct Tile {
  static constexpr int kHalf = sizeof(T) == 2;         // a 16-bit type
  static constexpr int kKeys = kHalf ? 32 : 16;        // slots a tile
  static constexpr int kSub = kKeys / 16;              // 16-slot groups of the scores
  static constexpr int kVec = 16 / sizeof(T);          // elements of 16 bytes
  static constexpr int kSteps = kDim / (4 * kVec);     // 16-byte loads of a lane for one row of K or Q
  static constexpr int kChunk = kDim / 16;             // elements a lane takes of a row of V
  static constexpr int kOut = kDim / 16;               // 16-dim groups of the output
  static constexpr int kRowsV = kKeys / 4;             // rows of V a lane takes
  static constexpr int kWords = kChunk * sizeof(T) / 4;

  // A lane's part of a row of K or Q: kVec elements from 4 kVec s + kVec g on, for every step s.  The row
  // lies `off` elements from `base`; a wave-uniform base keeps the 64-bit part of the address scalar.
  template <bool kStream>
  static __device__ __forceinline__ void load_row(u32x4 (&f)[kSteps], GlobalBytes base, unsigned off, int g,
                                                  int dim) {
    const unsigned at = lane_offset((off + kVec * g) * static_cast<unsigned>(sizeof(T)));
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      f[s] = u32x4{0, 0, 0, 0};
      if (kFull || 4 * kVec * s + kVec * g < dim)
        f[s] = load<u32x4, kStream>(base + at + 64 * s);
    }
  }

  // One of those loads.
  template <bool kStream>
  static __device__ __forceinline__ u32x4 load_step(GlobalBytes base, unsigned off, int s, int g, int dim) {
    const unsigned at = lane_offset((off + 4 * kVec * s + kVec * g) * static_cast<unsigned>(sizeof(T)));
    u32x4 x = {0, 0, 0, 0};
    if (kFull || 4 * kVec * s + kVec * g < dim) x = load<u32x4, kStream>(base + at);
    return x;
  }

  // A lane's kChunk elements of a row of V, from kChunk * (lane % 16) on: load z of kLoadsV.
  static constexpr int kLoadsV = kWords < 4 ? 1 : kWords / 4;
  static constexpr int kLoadWords = kWords / kLoadsV;
  typedef unsigned LoadV __attribute__((ext_vector_type(kLoadWords)));
  template <bool kStream>
  static __device__ __forceinline__ LoadV load_v_step(GlobalBytes base, unsigned off, int z, int col, int dim) {
    const unsigned at = lane_offset((off + kChunk * col) * static_cast<unsigned>(sizeof(T)) + 16 * z);
    LoadV x = {};
    if (kFull || kChunk * col + z * kVec < dim) x = load<LoadV, kStream>(base + at);
    return x;
  }
  template <bool kStream>
  static __device__ __forceinline__ void load_v(unsigned (&f)[kWords], GlobalBytes base, unsigned off, int col,
                                                int dim) {
#pragma unroll
    for (int z = 0; z < kLoadsV; ++z) {
      const LoadV x = load_v_step<kStream>(base, off, z, col, dim);
#pragma unroll
      for (int e = 0; e < kLoadWords; ++e) f[z * kLoadWords + e] = x[e];
    }
  }

  // Slot within the tile of a lane's score r of group sub, and of its V row 4 sub + r.
  static __device__ __forceinline__ int slot_of(int sub, int r, int g) { return 16 * sub + 4 * g + r; }
};

}  // namespace specdec
