// qz_product.h -- the arguments that the product kernels share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "qz.h"
#include "qz_weight.cuh"

namespace qz {

constexpr int kModeLinear = 0;    // y = x W^T
constexpr int kModeGated = 1;     // h = act(x W0^T) * (x W1^T)
constexpr int kModeBackward = 2;  // dx = x0 W0 (+ x1 W1)

struct ProductArgs {
  int mode, format, log2_block, n_weights, act;
  bool out_f32;
  WeightView w0, w1;
  int64_t rows, cols, tokens;
  const uint16_t *x0, *x1;  // bf16 [tokens, ld_x]: the activations, or the gradients dy / (dg, du)
  int64_t ld_x;
  void* y;                  // bf16 or fp32 [tokens, ld_y]
  int64_t ld_y;
  uint16_t *g_out, *u_out;  // bf16 [tokens, ld_gu] or null
  int64_t ld_gu;
};

// The streaming kernels for a few tokens (qz_product_few.cuh): their shared memory is a ring
// of code boxes and a buffer of partial sums per warp, and the activations.
// Tokens they are built for: E2M1 weights 16, INT4, whose tiles take two products a weight, 32.  Up to there
// the estimates of qz_product_plan.h decide.
constexpr int few_tokens(int format) { return format == QZ_INT4 ? 32 : 16; }
constexpr int kFewWarps = 16;
constexpr int kTokenStride = 20;                  // floats of a token's 16 sums (banks 8 t + g)
constexpr uint32_t kSlot = 2048;                  // a step: 16 rows x 128 bytes of codes
constexpr uint32_t kJoin = 8 * kTokenStride;      // floats of a warp's sums for 8 tokens
constexpr int kMaxDepth = 6;
constexpr uint32_t kFewSmem = 225 * 1024;         // dynamic; the barriers are static
constexpr uint32_t few_fixed(int depth) { return kFewWarps * (depth * kSlot + kJoin * 4) + 1024; }
inline int64_t few_steps(const ProductArgs& p) { return (p.cols + 255) / 256; }
// whole steps, whose scales are aligned vectors; else the steps' tails and scales take narrow loads
// (4 tokens, 32768 outputs, MXFP4: 8192 columns 38 us; 8160 columns 39 us, on the tensor-core tiles 70;
// INT4 groups of 32: 51, 56 and 134)
bool few_whole(const ProductArgs& p);
// the deepest ring that leaves room for the activations, 0: none does
inline int few_depth(const ProductArgs& p) {
  for (int d = kMaxDepth; d >= 2; --d)
    if (few_fixed(d) + p.tokens * few_steps(p) * 512 <= kFewSmem) return d;
  return 0;
}
bool product_few_applicable(const ProductArgs& p);
qz_status launch_product_few_mxfp4(const ProductArgs& p, cudaStream_t s);
qz_status launch_product_few_nvfp4(const ProductArgs& p, cudaStream_t s);
qz_status launch_product_few_int4(const ProductArgs& p, cudaStream_t s);
qz_status launch_product_few_mxfp4_ragged(const ProductArgs& p, cudaStream_t s);
qz_status launch_product_few_nvfp4_ragged(const ProductArgs& p, cudaStream_t s);
qz_status launch_product_few_int4_ragged(const ProductArgs& p, cudaStream_t s);

// The tcgen05 kernels (qz_product_tc.cuh): applicable when cols % 32 == 0 and codes, activations
// and their rows are 16-byte aligned.
bool product_tc_applicable(const ProductArgs& p);
qz_status launch_product_tc_mxfp4(const ProductArgs& p, cudaStream_t s);
qz_status launch_product_tc_nvfp4(const ProductArgs& p, cudaStream_t s);
qz_status launch_product_tc_int4(const ProductArgs& p, cudaStream_t s);

}  // namespace qz
