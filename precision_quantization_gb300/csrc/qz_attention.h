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
// row r is new token r / group.  The few-row kernel takes 16 or 32 of them at a time.
constexpr int kTile = 16;   // tokens of a step: every scale block and page is whole steps

// ---- a few rows (qz_attention_few.cuh) ---------------------------------------------------------
constexpr int kFewAttWarps = 8;
constexpr int kFewAttThreads = 32 * kFewAttWarps;
constexpr int few_att_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
// row tiles of 16 that a CTA holds: two where more than 16 rows are to be expected and registers allow it
inline int few_att_tiles(int dim, int64_t rows) { return rows > 16 && dim <= 128 ? 2 : 1; }

struct FewPlan {
  int row_tiles;      // MT
  bool whole;         // a CTA takes whole items, no partial results
  int grid;
  int min_chunk;      // steps of a CTA at least
};
FewPlan few_att_plan(const qz_cache& c, int64_t seqs, int64_t tokens, int64_t heads, int64_t table_pages, int sms);
size_t few_att_workspace(const FewPlan& p, int dim);

qz_status launch_attention_few_int8(const AttentionArgs& a, const FewPlan& p, cudaStream_t s);
qz_status launch_attention_few_e4m3(const AttentionArgs& a, const FewPlan& p, cudaStream_t s);
qz_status launch_attention_few_e5m2(const AttentionArgs& a, const FewPlan& p, cudaStream_t s);

}  // namespace qz
