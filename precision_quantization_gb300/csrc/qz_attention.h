// qz_attention.h -- the arguments that the attention kernels share, and the choice among them.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "qz.h"
#include "qz_cache.h"

namespace qz {

constexpr int64_t kNoWindow = int64_t{1} << 32;  // more than there are positions

struct AttentionArgs {
  CacheView c;
  BatchView b;
  const uint16_t* q;
  uint16_t* out;
  float* lse;               // null: not written
  int64_t ld_q, hd_q, ld_out, hd_out, ld_lse;
  int32_t heads, group;     // query heads, and those of a kv head
  int64_t window;           // up to kNoWindow
  float scale;              // times log2(e)
  bool q_vec, out_vec;      // 8-byte pieces of q and out are aligned
  void* ws;
};

// The rows of an item are the (token, head of the group) pairs of one sequence and kv head, heads fastest:
// row r is new token r / group.

// ---- a few rows (qz_attention_few.cuh) ---------------------------------------------------------
constexpr int few_att_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
// tiles of 8 rows that a CTA holds, as many as the rows to be expected fill and registers allow
inline int few_att_tiles(int dim, int64_t rows) { return rows <= 8 ? 1 : rows <= 16 || dim > 128 ? 2 : 4; }
// tokens of a step of one warp: 4 or 8 KiB of keys and values
constexpr int few_att_step(int dim) { return dim > 128 ? 16 : 32; }

struct FewPlan {
  int row_tiles;      // of 8 rows
  bool whole;         // a CTA takes whole items, no partial results
  int grid;
  int min_chunk;      // steps of a CTA at least
};
FewPlan few_att_plan(const qz_cache& c, int64_t seqs, int64_t tokens, int64_t heads, int64_t table_pages, int sms);
size_t few_att_workspace(const FewPlan& p, int dim);

qz_status launch_attention_few_int8(const AttentionArgs& a, const FewPlan& p, cudaStream_t s);
qz_status launch_attention_few_e4m3(const AttentionArgs& a, const FewPlan& p, cudaStream_t s);
qz_status launch_attention_few_e5m2(const AttentionArgs& a, const FewPlan& p, cudaStream_t s);

// ---- many rows (qz_attention_tc.cuh) -------------------------------------------------------------
struct TcAttPlan {
  int nq;       // row tiles of 128 of a CTA
  int splits;   // parts of the keys
  int slots;    // places for a kv head's CTAs
  int grid;     // 0: not applicable
};
TcAttPlan tc_att_plan(const qz_cache& c, int64_t seqs, int64_t tokens, int64_t heads, int64_t table_pages, int sms);
// Places: sequence s's row tiles begin at slot floor(start group / tile_rows) + s, so that they end before the next one's
// begin.  Where starts decrease (which no caller may let them) a slot can be counted to a sequence that begins behind it.
__host__ __device__ inline int64_t tc_first_slot(int32_t start, int32_t s, int group, int tile_rows) {
  return static_cast<int64_t>(start) * group / tile_rows + s;
}
// The first row of the tile at `slot` of a sequence of `rows` rows; -1: no tile of it lies there.
__host__ __device__ inline int64_t tc_tile_row(int64_t slot, int64_t first_slot, int64_t rows, int tile_rows) {
  const int64_t row0 = (slot - first_slot) * tile_rows;
  return row0 >= 0 && row0 < rows ? row0 : -1;
}
inline size_t tc_att_workspace(const TcAttPlan& p, int64_t tokens, int64_t heads, int dim) {
  return p.splits > 1 ? static_cast<size_t>(p.splits) * tokens * heads * (dim + 2) * sizeof(float) : 0;
}

qz_status launch_attention_tc_int8(const AttentionArgs& a, const TcAttPlan& p, cudaStream_t s);
qz_status launch_attention_tc_e4m3(const AttentionArgs& a, const TcAttPlan& p, cudaStream_t s);
qz_status launch_attention_tc_e5m2(const AttentionArgs& a, const TcAttPlan& p, cudaStream_t s);

}  // namespace qz
