// Internal interface of the paged-cache entry points: host code in paged_api.cpp, kernels in
// rope.hip, attend_*.hip (their plan in paged_attention.cpp), kv_weights.hip and kv_evict.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace specdec {

constexpr int kMaxHeadDim = 256;

// The cache of include/specdec.h as the kernels take it.  Sizes were checked on the host:
// num_pages * page_size is below 2^31, max_pages * page_size (slots a sequence can have) at most 2^30.
struct KvArgs {
  char* k;
  char* v;
  const int32_t* table;
  float* weight;
  int32_t* position;
  long long page_stride, slot_stride, head_stride;  // elements
  int num_pages, page_size, max_pages, heads, dim;
};

// Rows of one sequence in a round.
struct RoundRows {
  int len;  // slots before the round
  int n;    // new tokens; 0 = the sequence is invalid
  int rows; // rows that an invalid sequence poisons
};

__device__ __forceinline__ RoundRows round_rows(const KvArgs& c, const int32_t* num_draft,
                                                const int32_t* kv_len, int b, int K) {
  RoundRows r;
  r.len = kv_len[b];
  const int k = num_draft ? num_draft[b] : K;
  const bool k_ok = k >= 0 && k <= K;
  r.rows = k_ok ? k + 1 : K + 1;
  const long long cap = static_cast<long long>(c.max_pages) * c.page_size;
  r.n = k_ok && r.len >= 0 && static_cast<long long>(r.len) + k + 1 <= cap ? k + 1 : 0;
  return r;
}

// Page id of a slot inside the table, or -1 if the id is outside the pool.
__device__ __forceinline__ int page_of(const KvArgs& c, int b, int slot) {
  const int p = c.table[static_cast<long long>(b) * c.max_pages + slot / c.page_size];
  return static_cast<unsigned>(p) < static_cast<unsigned>(c.num_pages) ? p : -1;
}

// First element of a slot's row of head h, and its entry of weight / position.
__device__ __forceinline__ long long row_at(const KvArgs& c, int page, int off, int h) {
  return page * c.page_stride + off * c.slot_stride + h * c.head_stride;
}
__device__ __forceinline__ long long record_at(const KvArgs& c, int page, int off, int h) {
  return (static_cast<long long>(page) * c.heads + h) * c.page_size + off;
}

// Elements: float, __bf16 and _Float16.
template <typename T>
__device__ __forceinline__ float to_float(T x) {
  return static_cast<float>(x);
}
template <typename T>
__device__ __forceinline__ T from_float(float x) {
  return static_cast<T>(x);  // nearest, ties to even
}

struct RopeArgs {
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  int B, K, q_heads;
  const int32_t *num_draft, *kv_len, *first_pos;
  const double* inv_freq;
  int rotary, interleaved;
  float scale;
  void* q_out;
  hipStream_t stream;
};

struct AttendArgs {
  const void* q;
  long long q_stride;
  int B, K, q_heads;
  const int32_t *num_draft, *kv_len;
  float scale;
  void* out;
  float* lse;
  void* workspace;
  hipStream_t stream;
};

struct WeightArgs {
  const void* q;
  long long q_stride;
  const float* lse;
  int B, K, q_heads;
  const int32_t *num_draft, *accept_len, *kv_len;
  float scale;
  hipStream_t stream;
};

struct EvictArgs {
  const int32_t* kv_len;
  int B, budget, keep_first, keep_last;
  int32_t* new_len;
  void* workspace;
  hipStream_t stream;
};

// dtype: a specdec_dtype.
hipError_t launch_rope(const RopeArgs& a, const KvArgs& c, int dtype);
hipError_t launch_attend(const AttendArgs& a, const KvArgs& c, int dtype);
hipError_t launch_kv_weights(const WeightArgs& a, const KvArgs& c, int dtype);
hipError_t launch_kv_evict(const EvictArgs& a, const KvArgs& c, int dtype);
size_t attend_workspace_bytes(int K, int q_heads, int kv_heads, int dim);
size_t evict_workspace_bytes(int B, int heads, long long capacity, int budget);

}  // namespace specdec
