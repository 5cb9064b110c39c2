// qz_attention.cu -- attention of new tokens to a paged 8-bit key-value cache (include/qz.h,
// qz_cache_attention): argument checks, the choice of kernel and its launch plan.
#include "qz_attention.h"

#include <algorithm>
#include <climits>
#include <cstdint>

#include "qz_internal.h"

namespace qz {

// A CTA takes whole items where no sequence can be long enough to be worth cutting: its pages hold at most kWhole
// tokens, or twice that where the items fill half the GPU (8 sequences of 1000 tokens, 8 kv heads: 11.5 us whole,
// 16.2 cut; 32 of 2000: 36.3 and 40.7; one of 2000: 17.9 and 16.7).  Else the steps are shared out evenly, kMinChunk
// tokens at least to a CTA (one sequence of 2000 tokens: 16.7 us, 18.9 with twice as many).
constexpr int64_t kWhole = 1024, kMinChunk = 256;

FewPlan few_att_plan(const qz_cache& c, int64_t seqs, int64_t tokens, int64_t heads, int64_t table_pages, int sms) {
  FewPlan p{};
  const int64_t group = heads / c.kv_heads, rows = (tokens * group + seqs - 1) / seqs;
  p.row_tiles = few_att_tiles(c.dim, rows);
  const int64_t items = c.kv_heads * ((tokens * group) / (8 * p.row_tiles) + seqs);
  p.whole = table_pages * c.page <= (2 * items >= sms ? 2 * kWhole : kWhole) && items < INT32_MAX;
  p.grid = p.whole ? static_cast<int>(items) : sms;
  p.min_chunk = static_cast<int>(kMinChunk / few_att_step(c.dim));
  return p;
}
size_t few_att_workspace(const FewPlan& p, int dim) {
  const size_t slot = static_cast<size_t>(8 * p.row_tiles) * (few_att_dim(dim) + 2) * sizeof(float);
  return p.whole ? 0 : static_cast<size_t>(p.grid) * (16 + 2 * slot);
}

// More than kTcRows rows a sequence and kv head go to the tensor-core tiles (16 sequences of 4096 tokens, 8 kv heads,
// E4M3: 32 rows 85 us by the few-row kernel and 91 by the tiles, 48 rows 143 and 90; INT8, 64 elements, 64 x 2048:
// 32 rows 117 and 170, 64 rows 205 and 174).  Tiles that do not fill the GPU are cut along the keys, a part no shorter
// than kTcPart tokens (64 queries of 8192: 39.7 us; 41.4 with twice as many).  Cutting tiles that fill it, to even out the
// last round, costs more in partial sums than it gives: prompt of 4096 tokens, with q staged more slowly, 485 us whole, 581 in two parts.
constexpr int64_t kTcRows = 32, kTcPart = 512;

TcAttPlan tc_att_plan(const qz_cache& c, int64_t seqs, int64_t tokens, int64_t heads, int64_t table_pages, int sms) {
  TcAttPlan p{};
  const int64_t group = heads / c.kv_heads, rows = (tokens * group + seqs - 1) / seqs;
  if (c.dim > 128 || rows <= kTcRows) return p;
  p.nq = rows > 128 ? 2 : 1;
  const int64_t slots = tokens * group / (128 * p.nq) + seqs, tiles = c.kv_heads * seqs * ((rows + 128 * p.nq - 1) / (128 * p.nq));
  const int64_t most = std::max<int64_t>(table_pages * c.page / kTcPart, 1);
  const int64_t splits = std::max<int64_t>(std::min<int64_t>(sms / std::max<int64_t>(tiles, 1), most), 1);
  const int64_t grid = slots * c.kv_heads * splits;
  if (grid > INT32_MAX || tokens * heads > INT32_MAX) return p;
  p.splits = static_cast<int>(splits), p.slots = static_cast<int>(slots), p.grid = static_cast<int>(grid);
  return p;
}

}  // namespace qz

using namespace qz;

extern "C" size_t qz_cache_attention_workspace(const qz_cache* cache, int64_t sequences, int64_t tokens, int64_t heads,
                                               int64_t table_pages) {
  if (check_cache(cache) != QZ_OK || sequences <= 0 || tokens <= 0 || heads <= 0 || table_pages < 0) return 0;
  if (heads % cache->kv_heads || tokens > (1 << 30) || heads > INT32_MAX / cache->dim || sequences > (1 << 24) || table_pages > (1 << 24)) return 0;
  const int sms = sm_count();
  const TcAttPlan tc = tc_att_plan(*cache, sequences, tokens, heads, table_pages, sms);
  if (tc.grid) return tc_att_workspace(tc, tokens, heads, cache->dim);
  return few_att_workspace(few_att_plan(*cache, sequences, tokens, heads, table_pages, sms), cache->dim);
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
  if (heads % cache->kv_heads || window < 0 || !(scale > 0.0f && scale <= 0x1p127f) || (lse && ld_lse < heads)) return QZ_ERR_SHAPE;
  if (lse && tokens > 0 && ld_lse > INT64_MAX / 16 / tokens) return QZ_ERR_SHAPE;
  if (tokens == 0 || heads == 0 || batch->sequences == 0) return QZ_OK;
  if (!q || !out) return QZ_ERR_NULL;
  if (!is_aligned(q, 2) || !is_aligned(out, 2) || !is_aligned(lse, 4)) return QZ_ERR_ALIGN;
  if (tokens > INT32_MAX / heads) return QZ_ERR_UNSUPPORTED;
  const int sms = sm_count();
  const TcAttPlan tc = tc_att_plan(*cache, batch->sequences, tokens, heads, batch->table_pages, sms);
  const FewPlan few = few_att_plan(*cache, batch->sequences, tokens, heads, batch->table_pages, sms);
  const size_t need = tc.grid ? tc_att_workspace(tc, tokens, heads, cache->dim) : few_att_workspace(few, cache->dim);
  if (need && (!ws || ws_bytes < need)) return QZ_ERR_WORKSPACE;
  if (!is_aligned(ws, 16)) return QZ_ERR_ALIGN;
  AttentionArgs a{};
  a.c = view_of(*cache);
  a.b = view_of(*batch, tokens);
  a.q = static_cast<const uint16_t*>(q), a.out = static_cast<uint16_t*>(out), a.lse = lse;
  a.ld_q = ld_q, a.hd_q = hd_q, a.ld_out = ld_out, a.hd_out = hd_out, a.ld_lse = ld_lse;
  a.heads = static_cast<int32_t>(heads), a.group = static_cast<int32_t>(heads / cache->kv_heads);
  a.window = window ? std::min<int64_t>(window, kNoWindow) : kNoWindow;
  a.scale = scale * 1.4426950408889634f;
  const auto pieces = [&](const void* p, int64_t ld, int64_t hd) {
    return is_aligned(p, 8) && (tokens <= 1 || ld % 4 == 0) && (heads <= 1 || hd % 4 == 0);
  };
  a.q_vec = pieces(q, ld_q, hd_q), a.out_vec = pieces(out, ld_out, hd_out);
  a.ws = ws;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (tc.grid) {
    if (cache->format == QZ_INT8) return launch_attention_tc_int8(a, tc, s);
    if (cache->format == QZ_FP8_E4M3) return launch_attention_tc_e4m3(a, tc, s);
    return launch_attention_tc_e5m2(a, tc, s);
  }
  if (cache->format == QZ_INT8) return launch_attention_few_int8(a, few, s);
  if (cache->format == QZ_FP8_E4M3) return launch_attention_few_e4m3(a, few, s);
  return launch_attention_few_e5m2(a, few, s);
}
