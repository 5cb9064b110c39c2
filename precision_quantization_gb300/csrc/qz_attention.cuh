// qz_attention.cuh -- what the attention kernels share on the device: 8-bit codes to f16 pairs, a row of q
// made f16, and the store of a finished row.
#pragma once

#include <cuda.h>  // CUtensorMap and its enumerators (types only; the encoder is looked up)
#include <cudaTypedefs.h>

#include "qz_attention.h"
#include "qz_device.cuh"
#include "qz_internal.h"
#include "qz_pipe.cuh"
#include "qz_weight.cuh"

namespace qz {
namespace {

constexpr float kNone = -__builtin_inff();

struct CacheMaps {
  CUtensorMap k, v;   // codes as [pages * kv heads][page][dim], boxes of 16 rows or more
};
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Bounded wait on phase `parity`.  The hint lets the hardware hold the warp until the phase completes: without it
// try_wait comes back early, and the polls of a CTA's waiting warps took two fifths of the instructions issued.
constexpr uint32_t kWaitHintNs = 1000000;
__device__ __forceinline__ bool held_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kWaitHintNs)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool held_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  if (held_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!held_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > limit_ns) return false;
  return true;
}

// ---- one 8-bit pair to f16 ----------------------------------------------------------------------
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// INT8 words have their sign bits flipped first (bias 128): 0x6400 | n is 1024 + n.
template <int FMT>
__device__ __forceinline__ uint32_t prepare_word(uint32_t w) {
  return FMT == QZ_INT8 ? w ^ 0x80808080u : w;
}
// the E4M3 pairs in a word's halves (as 16-bit halves of a register: a shift and a cast cost an instruction more)
__device__ __forceinline__ void e4m3_pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
}
// the two pairs of a prepared word's bytes: 0 and 1, 2 and 3
template <int FMT>
__device__ __forceinline__ void pairs_in_word(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == QZ_INT8) {
    lo = sub_f16x2(prmt(w, 0x64646464u, 0x4140u), 0x64806480u);
    hi = sub_f16x2(prmt(w, 0x64646464u, 0x4342u), 0x64806480u);
  } else if constexpr (FMT == QZ_FP8_E5M2) {
    lo = prmt(w, 0u, 0x1404u);
    hi = prmt(w, 0u, 0x3424u);
  } else {
    e4m3_pairs(w, lo, hi);
  }
}
// bytes J and J + 1 of two words, the pairs (a, b) of each
template <int FMT, int J>
__device__ __forceinline__ void pairs_of_words(uint32_t a, uint32_t b, uint32_t& p0, uint32_t& p1) {
  if constexpr (FMT == QZ_INT8) {
    constexpr uint32_t kSel = J | (J << 4) | ((4 + J) << 8) | ((4 + J) << 12);  // (a, a, b, b)
    uint32_t d0, d1;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d0) : "r"(prmt(a, b, kSel)), "r"(0x00FF00FFu), "r"(0x64806480u));  // (t & m) ^ c
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d1) : "r"(prmt(a, b, kSel + 0x1111u)), "r"(0x00FF00FFu), "r"(0x64806480u));
    p0 = sub_f16x2(d0, 0x64806480u);
    p1 = sub_f16x2(d1, 0x64806480u);
  } else if constexpr (FMT == QZ_FP8_E5M2) {
    const uint32_t t = prmt(a, b, J | ((J + 1) << 4) | ((4 + J) << 8) | ((5 + J) << 12));  // (a, a', b, b')
    p0 = prmt(t, 0u, 0x2404u);
    p1 = t & 0xFF00FF00u;
  } else {
    e4m3_pairs(prmt(a, b, J | ((4 + J) << 4) | ((J + 1) << 8) | ((5 + J) << 12)), p0, p1);
  }
}
// Whether one of 16 codes stands for no finite number (E4M3: NaN; E5M2: NaN and Inf).  qz_cache_append writes none, but
// what lies at a position may be anything where a row does not see it, and the products take values by the tile: 0 x NaN.
template <int FMT>
__device__ __forceinline__ bool has_nonfinite(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  constexpr uint32_t kMask = FMT == QZ_FP8_E4M3 ? 0x7f7f7f7fu : 0x7c7c7c7cu, kOne = FMT == QZ_FP8_E4M3 ? 0x01010101u : 0x04040404u;
  return FMT != QZ_INT8 && ((((a & kMask) + kOne) | ((b & kMask) + kOne) | ((c & kMask) + kOne) | ((d & kMask) + kOne)) & 0x80808080u);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 4 elements of q at element offset `at` as bf16 pairs (zeros where !in)
__device__ __forceinline__ uint2 load_q4_raw(const AttentionArgs& a, bool in, int64_t at) {
  if (!in) return make_uint2(0u, 0u);
  if (a.q_vec) return __ldg(reinterpret_cast<const uint2*>(a.q + at));
  uint32_t x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = __ldg(a.q + at + e);
  return make_uint2(x[0] | (x[1] << 16), x[2] | (x[3] << 16));
}
// The power of two that brings a row whose largest magnitude is `top` into [2^14, 2^15), and its inverse;
// elements 2^-31 of the largest and less lose bits, 2^-39 of it at most.  NaN for a row that is not finite.
__device__ __forceinline__ float q_unit(float top, float& down) {
  const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100);
  down = __uint_as_float(static_cast<uint32_t>(127 - 14 + min(e, 127)) << 23);
  return is_finite_f(top) ? __uint_as_float(static_cast<uint32_t>(127 + 14 - min(e, 127)) << 23) : __uint_as_float(0x7fc00000u);
}
// 4 finished sums of a row, elements d .. d + 3: l and the sums relative to 2^top
__device__ __forceinline__ void store_row(const AttentionArgs& a, int64_t token, int head, int d, const float (&v)[4], float top, float l) {
  if (a.lse && d == 0) a.lse[token * a.ld_lse + head] = l == 0.0f ? kNone : (top + log2f(l)) * 0.69314718055994531f;
  if (d >= a.c.dim) return;
  const float r = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
  uint16_t* p = a.out + token * a.ld_out + head * a.hd_out + d;
  const uint32_t lo = bf16x2_bits(v[0] * r, v[1] * r), hi = bf16x2_bits(v[2] * r, v[3] * r);
  if (a.out_vec) {
    *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
  } else {
    p[0] = static_cast<uint16_t>(lo), p[1] = static_cast<uint16_t>(lo >> 16);
    p[2] = static_cast<uint16_t>(hi), p[3] = static_cast<uint16_t>(hi >> 16);
  }
}

// rows of 64 bytes (up to 64 elements) or 128 in the swizzle of that width; past the vector's end zeros
inline bool encode_codes(CUtensorMap* m, const AttentionArgs& a, const void* codes, int rows) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return false;
  const bool narrow = a.c.dim <= 64;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.c.dim), static_cast<cuuint64_t>(a.c.page), static_cast<cuuint64_t>(a.c.pages * a.c.heads)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.c.dim), static_cast<cuuint64_t>(a.c.page) * a.c.dim};
  const cuuint32_t box[3] = {narrow ? 64u : 128u, static_cast<cuuint32_t>(rows), 1}, es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool encode_maps(CacheMaps* m, const AttentionArgs& a, int rows) {
  return encode_codes(&m->k, a, a.c.k, rows) && encode_codes(&m->v, a, a.c.v, rows);
}

}  // namespace
}  // namespace qz
