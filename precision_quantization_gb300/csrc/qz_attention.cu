// qz_attention.cu -- attention of new tokens to a paged 8-bit key-value cache (include/qz.h,
// qz_cache_attention): argument checks and the kernel.
#include <climits>
#include <cstdint>

#include "qz_cache.h"
#include "qz_internal.h"
#include "qz_weight.cuh"

namespace qz {
namespace {

struct AttentionArgs {
  CacheView c;
  BatchView b;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t ld_q, hd_q, ld_out, hd_out, ld_lse;
  int32_t heads, group;
  int64_t window;  // 0: none
  float scale;     // times log2(e)
};

template <int FMT>
__device__ __forceinline__ float code_value(uint32_t c) {
  if constexpr (FMT == QZ_INT8) return dec_int8(c);
  float lo, hi;
  dec8x2<FMT>(c, lo, hi);
  return lo;
}

// One warp per token and head, lane l of it elements l, l + 32, ...
template <int FMT>
__global__ void __launch_bounds__(128) attention_kernel(const AttentionArgs a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, h = static_cast<int>(i % a.heads);
  const int64_t t = i / a.heads;
  if (t >= a.b.tokens) return;
  int32_t s = static_cast<int32_t>(t);
  if (a.b.starts) {
    int32_t lo = 0, hi = a.b.seqs;
    while (lo < hi) {
      const int32_t m = lo + (hi - lo) / 2;
      if (start_of(a.b, m) <= t) lo = m + 1;
      else hi = m;
    }
    s = lo - 1;
  }
  if (s < 0) return;
  const Span sp = span_of(a.b, s, a.c.page);
  if (t < sp.row || t >= sp.row + sp.n) return;
  const int64_t pos = sp.p0 + (t - sp.row);
  const int64_t end = pos + 1 < sp.len ? pos + 1 : sp.len;
  int64_t j = a.window && pos + 1 > a.window ? pos + 1 - a.window : 0;
  const int dim = a.c.dim, kvh = h / a.group;
  float q[8], o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int d = lane + 32 * k;
    q[k] = d < dim ? bf16_float(a.q[t * a.ld_q + h * a.hd_q + d]) : 0.0f;
    o[k] = 0.0f;
  }
  const float none = -__int_as_float(0x7f800000);
  float top = none, sum = 0.0f;
  for (; j < end; ++j) {
    const int64_t page = page_of(a.b, a.c, s, static_cast<int32_t>(j));
    if (page < 0) continue;
    const int in_page = static_cast<int>(j % a.c.page);
    const int64_t head = page * a.c.heads + kvh, at = (head * a.c.page + in_page) * dim;
    const int64_t block = head * (a.c.page >> a.c.log2_block) + (in_page >> a.c.log2_block);
    float x = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int d = lane + 32 * k;
      if (d < dim) x = __fmaf_rn(q[k], code_value<FMT>(a.c.k[at + d]), x);
    }
#pragma unroll
    for (int w = 16; w; w >>= 1) x += __shfl_xor_sync(kFull, x, w);
    x *= a.c.ks[block] * a.scale;
    const float was = top;
    if (x > top || x != x) top = x;
    const float f = was == none ? 0.0f : exp2f(was - top), p = exp2f(x - top), pv = p * a.c.vs[block];
    sum = __fmaf_rn(sum, f, p);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int d = lane + 32 * k;
      if (d < dim) o[k] = __fmaf_rn(o[k], f, pv * code_value<FMT>(a.c.v[at + d]));
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int d = lane + 32 * k;
    if (d < dim) a.out[t * a.ld_out + h * a.hd_out + d] = bf16_bits(sum == 0.0f ? 0.0f : __fdiv_rn(o[k], sum));
  }
  if (a.lse && lane == 0) a.lse[t * a.ld_lse + h] = sum == 0.0f ? none : (top + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace
}  // namespace qz

using namespace qz;

extern "C" size_t qz_cache_attention_workspace(const qz_cache* cache, int64_t sequences, int64_t tokens, int64_t heads) {
  if (check_cache(cache) != QZ_OK || sequences <= 0 || tokens <= 0 || heads <= 0) return 0;
  return 0;
}

extern "C" qz_status qz_cache_attention(const qz_cache* cache, const qz_batch* batch, const void* q, int64_t ld_q, int64_t hd_q,
                                        int64_t tokens, int64_t heads, float scale, int64_t window, void* out, int64_t ld_out,
                                        int64_t hd_out, float* lse, int64_t ld_lse, void* ws, size_t ws_bytes, qz_stream_t stream) {
  qz_status st;
  if ((st = check_cache(cache)) != QZ_OK) return st;
  const int64_t dim = cache->dim;
  if ((st = check_vectors(tokens, heads, dim, ld_q, hd_q)) != QZ_OK || (st = check_vectors(tokens, heads, dim, ld_out, hd_out)) != QZ_OK ||
      (st = check_batch(batch, tokens)) != QZ_OK)
    return st;
  if (heads % cache->kv_heads || window < 0 || !(scale > 0.0f && scale <= 3.402823466e38f) || (lse && ld_lse < heads)) return QZ_ERR_SHAPE;
  if (lse && tokens > 0 && ld_lse > INT64_MAX / 16 / tokens) return QZ_ERR_SHAPE;
  if (tokens == 0 || heads == 0 || batch->sequences == 0) return QZ_OK;
  if (!q || !out) return QZ_ERR_NULL;
  if (!is_aligned(q, 2) || !is_aligned(out, 2) || !is_aligned(lse, 4)) return QZ_ERR_ALIGN;
  const size_t need = qz_cache_attention_workspace(cache, batch->sequences, tokens, heads);
  if (need) {
    if (!ws || ws_bytes < need) return QZ_ERR_WORKSPACE;
    if (!is_aligned(ws, 16)) return QZ_ERR_ALIGN;
  }
  AttentionArgs a{};
  a.c = view_of(*cache);
  a.b = view_of(*batch, tokens);
  a.q = static_cast<const uint16_t*>(q), a.out = static_cast<uint16_t*>(out), a.lse = lse;
  a.ld_q = ld_q, a.hd_q = hd_q, a.ld_out = ld_out, a.hd_out = hd_out, a.ld_lse = ld_lse;
  a.heads = static_cast<int32_t>(heads), a.group = static_cast<int32_t>(heads / cache->kv_heads);
  a.window = window;
  a.scale = scale * 1.4426950408889634f;
  const int64_t blocks = (tokens * heads + 3) / 4;
  if (blocks > INT32_MAX) return QZ_ERR_UNSUPPORTED;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(blocks);
  if (cache->format == QZ_INT8) attention_kernel<QZ_INT8><<<grid, 128, 0, s>>>(a);
  else if (cache->format == QZ_FP8_E4M3) attention_kernel<QZ_FP8_E4M3><<<grid, 128, 0, s>>>(a);
  else attention_kernel<QZ_FP8_E5M2><<<grid, 128, 0, s>>>(a);
  return launch_status();
}
