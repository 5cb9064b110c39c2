// qz_cache.h -- the paged 8-bit key-value cache and the sequences of a call, as the kernels see them,
// and the argument checks that its calls share.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda_runtime.h>

#include "qz.h"
#include "qz_device.cuh"

namespace qz {

struct CacheView {
  uint8_t *k, *v;          // [pages, heads, page, dim]
  float *ks, *vs;          // [pages, heads, page / block]
  int64_t pages;
  int heads, page, block, dim;
  int log2_block;
};
struct BatchView {
  const int32_t *table, *lengths, *starts;
  int64_t ld_table;
  int32_t seqs, table_pages;
  int32_t tokens;          // rows of the call's tensors
};

// One sequence's new tokens: rows row .. row + n - 1, the first at position p0 (below 0 where the length
// says so), `len` tokens in all, no more than its pages hold.
struct Span {
  int32_t row, n, len;
  int64_t p0;
};

__device__ __forceinline__ int32_t start_of(const BatchView& b, int32_t s) {
  if (!b.starts) return s;
  return min(max(__ldg(b.starts + s), 0), b.tokens);
}
__device__ __forceinline__ Span span_of(const BatchView& b, int32_t s, int page) {
  Span r;
  r.row = start_of(b, s);
  r.n = max(start_of(b, s + 1) - r.row, 0);
  const int32_t len = max(__ldg(b.lengths + s), 0);
  r.p0 = static_cast<int64_t>(len) - r.n;
  r.len = static_cast<int32_t>(min(static_cast<int64_t>(len), static_cast<int64_t>(b.table_pages) * page));
  return r;
}
// The page of position `pos` (which lies below the span's len) of sequence s, or -1.
__device__ __forceinline__ int64_t page_of(const BatchView& b, const CacheView& c, int32_t s, int32_t pos) {
  const int32_t p = __ldg(b.table + s * b.ld_table + pos / c.page);
  return p >= 0 && p < c.pages ? p : -1;
}

// How many of the sequences' keys (not decreasing in s) are at most u; every thread of the block calls it.
template <class Key>
__device__ __forceinline__ int32_t count_upto(int32_t seqs, Key key, int64_t u) {
  int32_t n = 0;
  for (int32_t s0 = 0; s0 < seqs; s0 += static_cast<int32_t>(blockDim.x)) {
    const int32_t s = s0 + static_cast<int32_t>(threadIdx.x);
    const int32_t got = __syncthreads_count(s < seqs && key(s) <= u);
    n += got;
    if (got < static_cast<int32_t>(blockDim.x)) break;
  }
  return n;
}

// ---- checks on the host ------------------------------------------------------------------------
inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// [tokens, heads, dim] with strides ld and hd: vectors that do not overlap, offsets that fit
inline qz_status check_vectors(int64_t tokens, int64_t heads, int64_t dim, int64_t ld, int64_t hd) {
  if (tokens < 0 || heads < 0 || dim < 0) return QZ_ERR_SHAPE;
  if (tokens > INT32_MAX || heads > INT32_MAX || dim > INT32_MAX || heads * dim > INT32_MAX) return QZ_ERR_UNSUPPORTED;
  if (tokens == 0 || heads == 0) return QZ_OK;
  if ((heads > 1 && hd < dim) || (tokens > 1 && ld < dim) || hd < 0 || ld < 0) return QZ_ERR_SHAPE;
  constexpr int64_t kMost = INT64_MAX / 16;
  if ((heads > 1 && hd > kMost / heads) || (tokens > 1 && ld > kMost / tokens)) return QZ_ERR_SHAPE;
  // tokens outside heads, or heads outside tokens
  if (heads > 1 && tokens > 1 && ld < (heads - 1) * hd + dim && hd < (tokens - 1) * ld + dim) return QZ_ERR_SHAPE;
  return QZ_OK;
}
// rotated in place: each vector to where it came from
inline bool moves_in_place(const void* x, int64_t ld_x, int64_t hd_x, const void* y, int64_t ld_y, int64_t hd_y, int64_t tokens, int64_t heads) {
  return x == y && ((tokens > 1 && ld_x != ld_y) || (heads > 1 && hd_x != hd_y));
}
qz_status check_cache(const qz_cache* c);
qz_status check_batch(const qz_batch* b, int64_t tokens);
qz_status check_rotary_table(const qz_rotary_table* t, int64_t dim);
CacheView view_of(const qz_cache& c);
BatchView view_of(const qz_batch& b, int64_t tokens);

}  // namespace qz
