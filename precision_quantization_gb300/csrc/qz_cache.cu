// qz_cache.cu -- appending keys and values to a paged 8-bit cache, the keys (and the queries) rotated on
// the way (include/qz.h, qz_cache_append).
//
//   s = max(s_held, fl32(A / qmax)) per block of tokens and head, A = max |x| over its new values;
//   new codes RNE(fl32(x / s)), held codes RNE(fl32(decode(q) fl32(s_held / s))) where s has grown.
//
// A CTA takes one block of one kv head of one sequence, keys or values: its new values are read once and
// held in registers, 16 a thread and piece, from the amax to the codes.  Which blocks get tokens is known
// on the GPU only (lengths and starts lie there), so the grid covers the most that there can be: n tokens
// touch at most (n - 1) / block + 2 blocks, and with floor(start / block) + 2 s as sequence s's first slot
// no two sequences' slots meet.  Further CTAs rotate the queries.
#include "qz_cache.h"

#include <climits>
#include <cstdint>

#include "qz_internal.h"
#include "qz_rotary.cuh"

namespace qz {
namespace {

constexpr int kAppThreads = 256;
constexpr int kAppWarps = kAppThreads / 32;

struct AppendArgs {
  CacheView c;
  BatchView b;
  RotaryView r;
  const void *k, *v, *q;
  void* q_out;
  int64_t ld_k, hd_k, ld_v, hd_v, ld_q, hd_q, ld_qo, hd_qo;
  int32_t q_heads, q_units;  // threads of a query vector
  uint32_t kv_ctas;          // slots * kv heads * 2 (keys and values); the CTAs behind them rotate queries
};

template <int FMT>
__device__ __forceinline__ void encode16(const float (&x)[16], float s, uint32_t (&w)[4]) {
  const bool fast = fast_div_ok(s);
  const float r = __frcp_rn(s);
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = fast ? div_by(x[i], s, r) : __fdiv_rn(x[i], s);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = cvt8x2<FMT>(v[4 * i], v[4 * i + 1]) | (cvt8x2<FMT>(v[4 * i + 2], v[4 * i + 3]) << 16);
}
template <int FMT>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
  float v[4];
  dec8x2<FMT>(w & 0xffffu, v[0], v[1]);
  dec8x2<FMT>(w >> 16, v[2], v[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(v[i], r);
  return cvt8x2<FMT>(v[0], v[1]) | (cvt8x2<FMT>(v[2], v[3]) << 16);
}

// The queries of the call's tokens, rotated: VEC: 16 elements a thread, else a pair, or one past the pairs.
template <int DT, bool VEC>
__device__ __forceinline__ void rotate_queries(const AppendArgs& a, int64_t i) {
  const int64_t per_token = static_cast<int64_t>(a.q_heads) * a.q_units;
  const int64_t t = i / per_token;
  if (t >= a.b.tokens) return;
  const int rest = static_cast<int>(i - t * per_token), u = rest % a.q_units, h = rest / a.q_units;
  int32_t s = static_cast<int32_t>(t);
  if (a.b.starts) {  // the last sequence that starts at or before the row
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
  if (t < sp.row || t >= sp.row + sp.n) return;  // no sequence's row
  const int64_t pos = sp.p0 + (t - sp.row);
  const int64_t from = t * a.ld_q + h * a.hd_q, to = t * a.ld_qo + h * a.hd_qo;
  if constexpr (VEC) {
    int o0, o1;
    unit_offsets<true>(a.r, u, o0, o1);
    float v[16];
    load8<DT>(a.q, from + o0, v);
    load8<DT>(a.q, from + o1, v + 8);
    if (16 * u < 2 * a.r.pairs) {
      Turns turns;
      load_turns(a.r, u, pos, 1.0f, turns);
      turn_unit(a.r, turns, v);
    }
    store8v<DT>(a.q_out, to + o0, v);
    store8v<DT>(a.q_out, to + o1, v + 8);
  } else {
    if (u >= a.r.pairs) {
      store_elem<DT>(a.q_out, to + u + a.r.pairs, load_elem<DT>(a.q, from + u + a.r.pairs));
      return;
    }
    const int d0 = a.r.interleaved ? 2 * u : u, d1 = a.r.interleaved ? d0 + 1 : u + a.r.pairs;
    float v0 = load_elem<DT>(a.q, from + d0), v1 = load_elem<DT>(a.q, from + d1);
    if (pos < 0 || pos >= a.r.positions) v0 = v1 = __uint_as_float(0x7fc00000u);
    else turn(v0, v1, __ldg(a.r.cos + pos * a.r.pairs + u), __ldg(a.r.sin + pos * a.r.pairs + u));
    store_elem<DT>(a.q_out, to + d0, v0);
    store_elem<DT>(a.q_out, to + d1, v1);
  }
}

// R: pieces of 16 values a thread (block * dim / 16 / kAppThreads, rounded up).
template <int FMT, int DT, int R, bool VEC>
__global__ void __launch_bounds__(kAppThreads) append_kernel(const AppendArgs a) {
  __shared__ float warp_amax[kAppWarps];
  if (blockIdx.x >= a.kv_ctas) {
    rotate_queries<DT, VEC>(a, static_cast<int64_t>(blockIdx.x - a.kv_ctas) * kAppThreads + threadIdx.x);
    return;
  }
  const bool is_k = !(blockIdx.x & 1u);
  const uint32_t at = blockIdx.x >> 1;
  const int h = static_cast<int>(at % static_cast<uint32_t>(a.c.heads));
  const int64_t slot = at / static_cast<uint32_t>(a.c.heads);
  const int block = a.c.block, lb = a.c.log2_block;
  const auto first_slot = [&](int32_t s) { return static_cast<int64_t>(start_of(a.b, s) >> lb) + 2 * static_cast<int64_t>(s); };
  const int32_t s = a.b.starts ? count_upto(a.b.seqs, first_slot, slot) - 1 : static_cast<int32_t>(slot);
  if (s < 0) return;
  const Span sp = span_of(a.b, s, a.c.page);
  const int64_t first_new = sp.p0 > 0 ? sp.p0 : 0;
  const int64_t b0 = ((first_new >> lb) + (a.b.starts ? slot - first_slot(s) : 0)) << lb;  // the block's first position
  const int64_t new0 = first_new > b0 ? first_new : b0;
  int64_t end = b0 + block < sp.len ? b0 + block : sp.len;
  if (a.r.cos && end > a.r.positions) end = a.r.positions;
  if (new0 >= end) return;
  const int64_t page = page_of(a.b, a.c, s, static_cast<int32_t>(b0));
  if (page < 0) return;
  const int in_page = static_cast<int>(b0 % a.c.page);
  const int64_t head = page * a.c.heads + h;
  uint8_t* codes = (is_k ? a.c.k : a.c.v) + (head * a.c.page + in_page) * a.c.dim;
  float* scale = (is_k ? a.c.ks : a.c.vs) + head * (a.c.page >> lb) + (in_page >> lb);
  const float old = new0 > b0 ? *scale : 0.0f;

  // unit i: token i / units of the block, elements of unit i % units
  const int units = a.c.dim / 16, total = block * units;
  const void* src = is_k ? a.k : a.v;
  const int64_t ld = is_k ? a.ld_k : a.ld_v, hd = is_k ? a.hd_k : a.hd_v;
  RotaryView r = a.r;
  if (!is_k) r.cos = nullptr;
  float x[R][16];
  float amax = 0.0f;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int i = static_cast<int>(threadIdx.x) + k * kAppThreads, u = i % units;
    const int64_t pos = b0 + i / units;
    if (i < total && pos >= new0 && pos < end) {
      const int64_t base = (sp.row + (pos - sp.p0)) * ld + h * hd;
      if constexpr (VEC) {
        int o0, o1;
        unit_offsets<true>(r, u, o0, o1);
        load8<DT>(src, base + o0, x[k]);
        load8<DT>(src, base + o1, x[k] + 8);
        if (r.cos && 16 * u < 2 * r.pairs) {
          Turns turns;
          load_turns(r, u, pos, 1.0f, turns);
          turn_unit(r, turns, x[k]);
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < 16; ++j) {
          const float v = turned<DT>(r, src, base, 16 * u + j, pos, 1.0f);
#pragma unroll
          for (int q = 0; q < 16; ++q) x[k][q] = q == j ? v : x[k][q];
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) amax = absmax_nan(amax, x[k][j]);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = absmax_nan(amax, __shfl_xor_sync(kFull, amax, o));
  if ((threadIdx.x & 31u) == 0) warp_amax[threadIdx.x >> 5] = amax;
  __syncthreads();  // (every thread has read the old scale by now, too)
#pragma unroll
  for (int w = 0; w < kAppWarps; ++w) amax = absmax_nan(amax, warp_amax[w]);
  const float now = absmax_nan(__fdiv_rn(amax, Fmt8<FMT>::kMax), old);
  if (threadIdx.x == 0) *scale = now;
  const bool bad = !is_finite_f(now), zero = now == 0.0f;
  const bool grown = new0 > b0 && (bad || now > old);
  const float ratio = bad || zero ? 0.0f : __fdiv_rn(old, now);
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int i = static_cast<int>(threadIdx.x) + k * kAppThreads, u = i % units, t = i / units;
    const int64_t pos = b0 + t;
    if (i >= total) break;
    uint8_t* row = codes + static_cast<int64_t>(t) * a.c.dim;
    if (pos >= new0 && pos < end) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      if (!bad && !zero) encode16<FMT>(x[k], now, w);
      int o0, o1;
      unit_offsets<VEC>(r, u, o0, o1);
      *reinterpret_cast<uint2*>(row + o0) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + o1) = make_uint2(w[2], w[3]);
    } else if (pos < new0 && grown) {
      uint4* p = reinterpret_cast<uint4*>(row + 16 * u);
      uint4 w = *p;
      w.x = rescale4<FMT>(w.x, ratio);
      w.y = rescale4<FMT>(w.y, ratio);
      w.z = rescale4<FMT>(w.z, ratio);
      w.w = rescale4<FMT>(w.w, ratio);
      *p = bad ? make_uint4(0u, 0u, 0u, 0u) : w;
    }
  }
}

template <int FMT, int DT, bool VEC>
void run_append(const AppendArgs& a, unsigned grid, cudaStream_t s) {
  const int pieces = a.c.block * (a.c.dim / 16);
  if (pieces <= kAppThreads) append_kernel<FMT, DT, 1, VEC><<<grid, kAppThreads, 0, s>>>(a);
  else if (pieces <= 2 * kAppThreads) append_kernel<FMT, DT, 2, VEC><<<grid, kAppThreads, 0, s>>>(a);
  else if (pieces <= 4 * kAppThreads) append_kernel<FMT, DT, 4, VEC><<<grid, kAppThreads, 0, s>>>(a);
  else append_kernel<FMT, DT, 8, VEC><<<grid, kAppThreads, 0, s>>>(a);
}
template <int FMT>
void run_append(const AppendArgs& a, int dtype, bool vec, unsigned grid, cudaStream_t s) {
  if (dtype == QZ_BF16) vec ? run_append<FMT, QZ_BF16, true>(a, grid, s) : run_append<FMT, QZ_BF16, false>(a, grid, s);
  else vec ? run_append<FMT, QZ_F32, true>(a, grid, s) : run_append<FMT, QZ_F32, false>(a, grid, s);
}

}  // namespace

qz_status check_cache(const qz_cache* c) {
  if (!c) return QZ_ERR_NULL;
  if (c->format != QZ_INT8 && c->format != QZ_FP8_E4M3 && c->format != QZ_FP8_E5M2) return QZ_ERR_ENUM;
  if (c->pages < 0 || c->kv_heads <= 0 || c->page <= 0 || c->dim <= 0) return QZ_ERR_SHAPE;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return QZ_ERR_UNSUPPORTED;
  if (c->page > 1024 || c->dim > 256 || c->dim % 16) return QZ_ERR_UNSUPPORTED;
  if (c->page % c->block) return QZ_ERR_SHAPE;
  if (c->kv_heads > 65535 || c->pages > INT32_MAX / c->kv_heads) return QZ_ERR_UNSUPPORTED;
  if (c->pages > 0 && (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales)) return QZ_ERR_NULL;
  if (!is_aligned(c->k_codes, 16) || !is_aligned(c->v_codes, 16) || !is_aligned(c->k_scales, 4) || !is_aligned(c->v_scales, 4))
    return QZ_ERR_ALIGN;
  return QZ_OK;
}

qz_status check_batch(const qz_batch* b, int64_t tokens) {
  if (!b) return QZ_ERR_NULL;
  if (b->sequences < 0 || b->table_pages < 0 || b->ld_table < b->table_pages) return QZ_ERR_SHAPE;
  if (b->sequences > (1 << 24) || b->table_pages > (1 << 24) || tokens > (1 << 30)) return QZ_ERR_UNSUPPORTED;
  if (b->sequences > 0 && b->ld_table > INT64_MAX / 8 / b->sequences) return QZ_ERR_SHAPE;
  if (!b->starts && tokens != b->sequences) return QZ_ERR_SHAPE;
  if (b->sequences > 0 && tokens > 0 && (!b->lengths || (!b->table && b->table_pages > 0))) return QZ_ERR_NULL;
  if (!is_aligned(b->table, 4) || !is_aligned(b->lengths, 4) || !is_aligned(b->starts, 4)) return QZ_ERR_ALIGN;
  return QZ_OK;
}

CacheView view_of(const qz_cache& c) {
  CacheView v{};
  v.k = static_cast<uint8_t*>(c.k_codes), v.v = static_cast<uint8_t*>(c.v_codes);
  v.ks = c.k_scales, v.vs = c.v_scales;
  v.pages = c.pages;
  v.heads = c.kv_heads, v.page = c.page, v.block = c.block, v.dim = c.dim;
  v.log2_block = c.block == 16 ? 4 : c.block == 32 ? 5 : c.block == 64 ? 6 : 7;
  return v;
}
BatchView view_of(const qz_batch& b, int64_t tokens) {
  BatchView v{};
  v.table = b.table, v.lengths = b.lengths, v.starts = b.starts;
  v.ld_table = b.ld_table;
  v.seqs = static_cast<int32_t>(b.sequences), v.table_pages = static_cast<int32_t>(b.table_pages);
  v.tokens = static_cast<int32_t>(tokens);
  return v;
}

}  // namespace qz

using namespace qz;

extern "C" qz_status qz_cache_append(const qz_cache* cache, const qz_batch* batch, int32_t dtype, const void* k, int64_t ld_k,
                                     int64_t hd_k, const void* v, int64_t ld_v, int64_t hd_v, int64_t tokens,
                                     const qz_rotary_table* table, const void* q, int64_t ld_q, int64_t hd_q, int64_t heads,
                                     void* q_out, int64_t ld_qo, int64_t hd_qo, qz_stream_t stream) {
  qz_status st;
  if ((st = check_cache(cache)) != QZ_OK) return st;
  if (dtype != QZ_BF16 && dtype != QZ_F32) return QZ_ERR_ENUM;
  const int64_t kv = cache->kv_heads, dim = cache->dim;
  if ((st = check_vectors(tokens, kv, dim, ld_k, hd_k)) != QZ_OK || (st = check_vectors(tokens, kv, dim, ld_v, hd_v)) != QZ_OK ||
      (st = check_batch(batch, tokens)) != QZ_OK)
    return st;
  if (table && (st = check_rotary_table(table, dim)) != QZ_OK) return st;
  if ((q == nullptr) != (q_out == nullptr) || (q && !table)) return QZ_ERR_NULL;
  if (q && ((st = check_vectors(tokens, heads, dim, ld_q, hd_q)) != QZ_OK || (st = check_vectors(tokens, heads, dim, ld_qo, hd_qo)) != QZ_OK))
    return st;
  if (q && heads % kv) return QZ_ERR_SHAPE;
  if (tokens == 0 || batch->sequences == 0) return QZ_OK;
  if (!k || !v) return QZ_ERR_NULL;
  const int64_t e = dtype == QZ_BF16 ? 2 : 4;
  if (!is_aligned(k, e) || !is_aligned(v, e) || !is_aligned(q, e) || !is_aligned(q_out, e)) return QZ_ERR_ALIGN;
  AppendArgs a{};
  a.c = view_of(*cache);
  a.b = view_of(*batch, tokens);
  a.r = view_of(table);
  a.k = k, a.v = v, a.q = q, a.q_out = q_out;
  a.ld_k = ld_k, a.hd_k = hd_k, a.ld_v = ld_v, a.hd_v = hd_v;
  a.ld_q = ld_q, a.hd_q = hd_q, a.ld_qo = ld_qo, a.hd_qo = hd_qo;
  const bool vec = (!a.r.cos || rotary_vec(a.r, dim)) && rows_vec(k, e, tokens, ld_k, kv, hd_k) && rows_vec(v, e, tokens, ld_v, kv, hd_v) &&
                   (!q || (rows_vec(q, e, tokens, ld_q, heads, hd_q) && rows_vec(q_out, e, tokens, ld_qo, heads, hd_qo)));
  const int64_t slots = cache->pages == 0 ? 0 : batch->starts ? tokens / cache->block + 2 * batch->sequences : batch->sequences;
  a.q_heads = static_cast<int32_t>(heads);
  a.q_units = static_cast<int32_t>(vec ? dim / 16 : dim - a.r.pairs);
  const int64_t q_ctas = q ? (tokens * heads * a.q_units + kAppThreads - 1) / kAppThreads : 0;
  const int64_t ctas = 2 * slots * kv + q_ctas;
  if (slots > INT32_MAX / kv / 2 || ctas > INT32_MAX) return QZ_ERR_UNSUPPORTED;
  if (ctas == 0) return QZ_OK;
  a.kv_ctas = static_cast<uint32_t>(2 * slots * kv);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(ctas);
  if (cache->format == QZ_INT8) run_append<QZ_INT8>(a, dtype, vec, grid, s);
  else if (cache->format == QZ_FP8_E4M3) run_append<QZ_FP8_E4M3>(a, dtype, vec, grid, s);
  else run_append<QZ_FP8_E5M2>(a, dtype, vec, grid, s);
  return launch_status();
}
