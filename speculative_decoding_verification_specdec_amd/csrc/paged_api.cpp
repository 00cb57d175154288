// C ABI of the paged-cache entry points (declared in include/specdec.h): host-side argument checks,
// the host arithmetic of the rotary frequencies, and stream-ordered launches.  Allocates nothing,
// keeps no state, never synchronises.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "paged.h"
#include "specdec.h"

static_assert(SPECDEC_MAX_HEAD_DIM == specdec::kMaxHeadDim, "largest head");

namespace {

bool misaligned(const void* p, size_t a) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) != 0;
}

size_t element_size(int32_t dtype) { return dtype == SPECDEC_F32 ? 4 : 2; }

bool heads_valid(int32_t q_heads, int32_t kv_heads) {
  return kv_heads >= 1 && q_heads >= 1 && q_heads % kv_heads == 0;
}

bool dim_valid(int32_t dim) {
  return dim >= 8 && dim <= SPECDEC_MAX_HEAD_DIM && dim % 8 == 0;
}

bool rows_valid(int32_t B, int32_t K, int32_t heads) {
  return B >= 0 && K >= 0 &&
         static_cast<long long>(B) * (static_cast<long long>(K) + 1) < (1LL << 31) &&
         static_cast<long long>(heads) * (static_cast<long long>(K) + 1) < (1LL << 31);
}

specdec_status check_cache(const specdec_kv_cache* c) {
  if (!c) return SPECDEC_ERR_NULL;
  // (slots of a sequence: the kernels round them up to whole tiles and groups, in 32 bits)
  if (c->num_pages < 1 || c->page_size < 1 || c->num_kv_heads < 1 || c->num_kv_heads > 65536 ||
      c->max_pages < 1 || !dim_valid(c->head_dim) ||
      static_cast<long long>(c->num_pages) * c->page_size >= (1LL << 31) ||
      static_cast<long long>(c->max_pages) * c->page_size > (1LL << 30))
    return SPECDEC_ERR_SHAPE;
  if (c->dtype != SPECDEC_F32 && c->dtype != SPECDEC_BF16 && c->dtype != SPECDEC_F16)
    return SPECDEC_ERR_DTYPE;
  // The furthest element has to be addressable in bytes with 64 bits: each term below 2^60.
  const long long most = (1LL << 58) / c->num_pages;
  if ((c->num_pages > 1 && (c->page_stride < c->head_dim || c->page_stride > most)) ||
      (c->page_size > 1 &&
       (c->slot_stride < c->head_dim || c->slot_stride > (1LL << 58) / c->page_size)) ||
      (c->num_kv_heads > 1 &&
       (c->head_stride < c->head_dim || c->head_stride > (1LL << 58) / c->num_kv_heads)))
    return SPECDEC_ERR_SHAPE;
  return SPECDEC_OK;
}

// After check_cache and the early return of an empty batch.
specdec_status check_cache_pointers(const specdec_kv_cache* c) {
  if (!c->k || !c->v || !c->page_table) return SPECDEC_ERR_NULL;
  const long long unit = 16 / static_cast<long long>(element_size(c->dtype));
  if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->page_table, 4) ||
      misaligned(c->weight, 4) || misaligned(c->position, 4) ||
      (c->num_pages > 1 && c->page_stride % unit) || (c->page_size > 1 && c->slot_stride % unit) ||
      (c->num_kv_heads > 1 && c->head_stride % unit))
    return SPECDEC_ERR_ALIGN;
  return SPECDEC_OK;
}

specdec::KvArgs kv_args(const specdec_kv_cache* c) {
  specdec::KvArgs a{};
  a.k = static_cast<char*>(c->k);
  a.v = static_cast<char*>(c->v);
  a.table = c->page_table;
  a.weight = c->weight;
  a.position = c->position;
  // Strides of a dimension of one entry are never used: any value may stand there.
  a.page_stride = c->num_pages > 1 ? c->page_stride : 0;
  a.slot_stride = c->page_size > 1 ? c->slot_stride : 0;
  a.head_stride = c->num_kv_heads > 1 ? c->head_stride : 0;
  a.num_pages = c->num_pages;
  a.page_size = c->page_size;
  a.max_pages = c->max_pages;
  a.heads = c->num_kv_heads;
  a.dim = c->head_dim;
  return a;
}

// A [B, K+1, heads, dim] tensor whose tokens lie `stride` elements apart.
bool stride_valid(long long stride, int32_t B, int32_t K, int32_t heads, int32_t dim) {
  const long long tokens = static_cast<long long>(B) * (K + 1LL);
  return tokens <= 1 ||
         (stride >= static_cast<long long>(heads) * dim && stride <= (1LL << 58) / tokens);
}

bool stride_misaligned(long long stride, int32_t B, int32_t K, int32_t dtype) {
  return static_cast<long long>(B) * (K + 1LL) > 1 &&
         stride % (16 / static_cast<long long>(element_size(dtype))) != 0;
}

// A finite value over 0.
bool positive(float x) { return x > 0.f && x <= 3.402823466e38f; }

specdec_status status_of(hipError_t e) { return e == hipSuccess ? SPECDEC_OK : SPECDEC_ERR_LAUNCH; }

}  // namespace

extern "C" {

specdec_status specdec_rope_frequencies(int32_t rotary_dim, double base, int32_t scaling,
                                        double factor, double original_len, double turns_low,
                                        double turns_high, double* inv_freq) {
  const bool base_scaling = scaling == SPECDEC_ROPE_BASE;
  if (rotary_dim < (base_scaling ? 4 : 2) || rotary_dim > SPECDEC_MAX_HEAD_DIM || rotary_dim % 2 ||
      !(base > 1) || !isfinite(base) || scaling < SPECDEC_ROPE_PLAIN ||
      scaling > SPECDEC_ROPE_TURNS)
    return SPECDEC_ERR_SHAPE;
  if (scaling != SPECDEC_ROPE_PLAIN && (!(factor >= 1) || !isfinite(factor)))
    return SPECDEC_ERR_SHAPE;
  if (scaling == SPECDEC_ROPE_TURNS &&
      (!(original_len > 0) || !isfinite(original_len) || !(turns_low >= 0) ||
       !(turns_high > turns_low) || !isfinite(turns_high)))
    return SPECDEC_ERR_SHAPE;
  if (!inv_freq) return SPECDEC_ERR_NULL;
  if (misaligned(inv_freq, 8)) return SPECDEC_ERR_ALIGN;
  if (base_scaling) base *= pow(factor, static_cast<double>(rotary_dim) / (rotary_dim - 2));
  for (int32_t i = 0; i < rotary_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rotary_dim);
    if (scaling == SPECDEC_ROPE_LINEAR) f /= factor;
    if (scaling == SPECDEC_ROPE_TURNS) {
      const double turns = original_len * f / (2.0 * M_PI);
      const double keep = fmin(1.0, fmax(0.0, (turns - turns_low) / (turns_high - turns_low)));
      f = keep * f + (1.0 - keep) * (f / factor);
    }
    inv_freq[i] = f;
  }
  return SPECDEC_OK;
}

specdec_status specdec_rope_append(const void* q, const void* k, const void* v, int64_t q_stride,
                                   int64_t k_stride, int64_t v_stride, int32_t B, int32_t K,
                                   int32_t num_q_heads, const int32_t* num_draft,
                                   const int32_t* kv_len, const int32_t* first_pos,
                                   const specdec_rope* rope, const specdec_kv_cache* cache,
                                   void* q_out, void* stream) {
  specdec_status st = check_cache(cache);
  if (st != SPECDEC_OK) return st;
  if (!rope) return SPECDEC_ERR_NULL;
  const int32_t dim = cache->head_dim, kv_heads = cache->num_kv_heads;
  if (num_q_heads < 1 || !rows_valid(B, K, num_q_heads) ||
      num_q_heads + 2LL * kv_heads >= (1LL << 31) || rope->rotary_dim < 0 ||
      rope->rotary_dim % 2 || rope->rotary_dim > dim || !isfinite(rope->scale) ||
      !stride_valid(q_stride, B, K, num_q_heads, dim) ||
      !stride_valid(k_stride, B, K, kv_heads, dim) || !stride_valid(v_stride, B, K, kv_heads, dim))
    return SPECDEC_ERR_SHAPE;
  if (B == 0) return SPECDEC_OK;
  st = check_cache_pointers(cache);
  if (st == SPECDEC_ERR_NULL) return st;
  if (!q || !k || !v || !kv_len || !q_out || (rope->rotary_dim > 0 && !rope->inv_freq))
    return SPECDEC_ERR_NULL;
  if (st != SPECDEC_OK) return st;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(q_out, 16) ||
      misaligned(num_draft, 4) || misaligned(kv_len, 4) || misaligned(first_pos, 4) ||
      misaligned(rope->inv_freq, 8) || stride_misaligned(q_stride, B, K, cache->dtype) ||
      stride_misaligned(k_stride, B, K, cache->dtype) ||
      stride_misaligned(v_stride, B, K, cache->dtype))
    return SPECDEC_ERR_ALIGN;
  // (in place only where every row of q_out is its own row of q)
  if (q_out == q && static_cast<long long>(B) * (K + 1LL) > 1 &&
      q_stride != static_cast<long long>(num_q_heads) * dim)
    return SPECDEC_ERR_SHAPE;
  specdec::RopeArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.B = B;
  a.K = K;
  a.q_heads = num_q_heads;
  a.num_draft = num_draft;
  a.kv_len = kv_len;
  a.first_pos = first_pos ? first_pos : kv_len;
  a.inv_freq = rope->inv_freq;
  a.rotary = rope->rotary_dim;
  a.interleaved = rope->interleaved != 0;
  a.scale = rope->scale;
  a.q_out = q_out;
  a.stream = static_cast<hipStream_t>(stream);
  return status_of(specdec::launch_rope(a, kv_args(cache), cache->dtype));
}

size_t specdec_paged_attention_workspace_size(int32_t B, int32_t K, int32_t num_q_heads,
                                              int32_t num_kv_heads, int32_t head_dim) {
  if (B <= 0 || K < 0 || K > SPECDEC_MAX_K || !heads_valid(num_q_heads, num_kv_heads) ||
      !rows_valid(B, K, num_q_heads) || !dim_valid(head_dim))
    return 0;
  return specdec::attend_workspace_bytes(K, num_q_heads, num_kv_heads, head_dim);
}

specdec_status specdec_paged_attention(const void* q, int64_t q_stride, int32_t B, int32_t K,
                                       int32_t num_q_heads, const int32_t* num_draft,
                                       const int32_t* kv_len, float scale,
                                       const specdec_kv_cache* cache, void* out, float* lse,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  specdec_status st = check_cache(cache);
  if (st != SPECDEC_OK) return st;
  const int32_t dim = cache->head_dim, kv_heads = cache->num_kv_heads;
  if (K > SPECDEC_MAX_K || !heads_valid(num_q_heads, kv_heads) || !rows_valid(B, K, num_q_heads) ||
      !positive(scale) || !stride_valid(q_stride, B, K, num_q_heads, dim))
    return SPECDEC_ERR_SHAPE;
  if (B == 0) return SPECDEC_OK;
  st = check_cache_pointers(cache);
  if (st == SPECDEC_ERR_NULL) return st;
  if (!q || !kv_len || !out || !workspace) return SPECDEC_ERR_NULL;
  if (st != SPECDEC_OK) return st;
  if (misaligned(q, 16) || misaligned(out, 16) || misaligned(lse, 4) || misaligned(num_draft, 4) ||
      misaligned(kv_len, 4) || misaligned(workspace, 16) ||
      stride_misaligned(q_stride, B, K, cache->dtype))
    return SPECDEC_ERR_ALIGN;
  if (workspace_bytes < specdec::attend_workspace_bytes(K, num_q_heads, kv_heads, dim))
    return SPECDEC_ERR_WORKSPACE;
  specdec::AttendArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.B = B;
  a.K = K;
  a.q_heads = num_q_heads;
  a.num_draft = num_draft;
  a.kv_len = kv_len;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  a.stream = static_cast<hipStream_t>(stream);
  return status_of(specdec::launch_attend(a, kv_args(cache), cache->dtype));
}

specdec_status specdec_kv_weights(const void* q, int64_t q_stride, const float* lse, int32_t B,
                                  int32_t K, int32_t num_q_heads, const int32_t* num_draft,
                                  const int32_t* accept_len, const int32_t* kv_len, float scale,
                                  const specdec_kv_cache* cache, void* stream) {
  specdec_status st = check_cache(cache);
  if (st != SPECDEC_OK) return st;
  const int32_t dim = cache->head_dim, kv_heads = cache->num_kv_heads;
  if (K > SPECDEC_MAX_K || !heads_valid(num_q_heads, kv_heads) || !rows_valid(B, K, num_q_heads) ||
      !positive(scale) || !stride_valid(q_stride, B, K, num_q_heads, dim))
    return SPECDEC_ERR_SHAPE;
  if (B == 0) return SPECDEC_OK;
  st = check_cache_pointers(cache);
  if (st == SPECDEC_ERR_NULL) return st;
  if (!q || !lse || !kv_len || !cache->weight) return SPECDEC_ERR_NULL;
  if (st != SPECDEC_OK) return st;
  if (misaligned(q, 16) || misaligned(lse, 4) || misaligned(num_draft, 4) ||
      misaligned(accept_len, 4) || misaligned(kv_len, 4) ||
      stride_misaligned(q_stride, B, K, cache->dtype))
    return SPECDEC_ERR_ALIGN;
  specdec::WeightArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.lse = lse;
  a.B = B;
  a.K = K;
  a.q_heads = num_q_heads;
  a.num_draft = num_draft;
  a.accept_len = accept_len;
  a.kv_len = kv_len;
  a.scale = scale;
  a.stream = static_cast<hipStream_t>(stream);
  return status_of(specdec::launch_kv_weights(a, kv_args(cache), cache->dtype));
}

size_t specdec_kv_evict_workspace_size(int32_t B, const specdec_kv_cache* cache, int32_t budget) {
  if (B <= 0 || budget < 1 || check_cache(cache) != SPECDEC_OK) return 0;
  return specdec::evict_workspace_bytes(
      B, cache->num_kv_heads, static_cast<long long>(cache->max_pages) * cache->page_size, budget);
}

specdec_status specdec_kv_evict(const specdec_kv_cache* cache, const int32_t* kv_len, int32_t B,
                                int32_t budget, int32_t keep_first, int32_t keep_last,
                                int32_t* new_len, void* workspace, size_t workspace_bytes,
                                void* stream) {
  specdec_status st = check_cache(cache);
  if (st != SPECDEC_OK) return st;
  if (B < 0 || budget < 1 || keep_first < 0 || keep_last < 0 ||
      static_cast<long long>(keep_first) + keep_last > budget ||
      static_cast<long long>(B) * cache->num_kv_heads >= (1LL << 31))
    return SPECDEC_ERR_SHAPE;
  if (B == 0) return SPECDEC_OK;
  st = check_cache_pointers(cache);
  if (st == SPECDEC_ERR_NULL) return st;
  if (!kv_len || !workspace || !cache->weight || !cache->position) return SPECDEC_ERR_NULL;
  if (st != SPECDEC_OK) return st;
  if (misaligned(kv_len, 4) || misaligned(new_len, 4) || misaligned(workspace, 16))
    return SPECDEC_ERR_ALIGN;
  // new_len is kv_len or lies apart from it: a sequence's length is read while others' are written.
  const uintptr_t len = reinterpret_cast<uintptr_t>(kv_len), out = reinterpret_cast<uintptr_t>(new_len);
  const uintptr_t bytes = static_cast<uintptr_t>(B) * 4;
  if (new_len && out != len && out < len + bytes && len < out + bytes) return SPECDEC_ERR_SHAPE;
  if (workspace_bytes < specdec_kv_evict_workspace_size(B, cache, budget))
    return SPECDEC_ERR_WORKSPACE;
  specdec::EvictArgs a{};
  a.kv_len = kv_len;
  a.B = B;
  a.budget = budget;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  a.new_len = new_len;
  a.workspace = workspace;
  a.stream = static_cast<hipStream_t>(stream);
  return status_of(specdec::launch_kv_evict(a, kv_args(cache), cache->dtype));
}

}  // extern "C"
