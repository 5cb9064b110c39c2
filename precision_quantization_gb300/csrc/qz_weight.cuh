// qz_weight.cuh -- the 4-bit weights of the product kernels (MXFP4, NVFP4, grouped INT4): their
// device view, the value of one code, and the activations of the gated block.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "qz_device.cuh"

namespace qz {

struct WeightView {
  const uint8_t* codes;   // [rows, cols / 2], the even column in the low nibble
  const void* scales;     // [rows, cols / block]: E8M0, E4M3 or fp32
  const float* tscale;    // NVFP4 tensor scale, or null (1)
};

inline WeightView view_of(const qz_weight& w) {
  return WeightView{static_cast<const uint8_t*>(w.codes), w.scales,
                    w.format == QZ_NVFP4 ? w.tensor_scale_dev : nullptr};
}

// decode(code) of one nibble
template <int FMT>
__device__ __forceinline__ float nibble_value(uint32_t n) {
  if constexpr (FMT == QZ_INT4) {
    return static_cast<float>(static_cast<int>(n ^ 8u) - 8);
  } else {  // E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6: fields e (2 bits), m (1 bit)
    const uint32_t e = (n >> 1) & 3u, m = n & 1u;
    const float v = e ? __uint_as_float(((126u + e) << 23) | (m << 22)) : 0.5f * static_cast<float>(m);
    return (n & 8u) ? -v : v;
  }
}

// the scale of block b (a flat index over [rows, cols / block])
template <int FMT>
__device__ __forceinline__ float block_scale(const void* scales, int64_t b) {
  if constexpr (FMT == QZ_INT4) return __ldg(static_cast<const float*>(scales) + b);
  const uint32_t c = __ldg(static_cast<const uint8_t*>(scales) + b);
  if constexpr (FMT == QZ_MXFP4) return c == 255u ? __uint_as_float(0x7fc00000u) : exp2_pos(static_cast<int>(c) - 127);
  return dec_e4m3(c);
}

// The factor of the finished sum (the NVFP4 tensor scale).
template <int FMT>
__device__ __forceinline__ float sum_factor(const float* tscale) {
  if constexpr (FMT == QZ_NVFP4) return tscale ? __ldg(tscale) : 1.0f;
  return 1.0f;
}

// act(a) and act'(a).  SiLU: a p with p = 1 / (1 + exp(-a)); the tanh form of GELU is a p(2 z)
// too, z = sqrt(2 / pi) (a + 0.044715 a^3), because (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)).
// Infinite exp(-a) gives p = 0 and a p = -0, the limit.
template <int ACT>
__device__ __forceinline__ float act_gate(float a, float& slope) {  // p, and d(2 z) / da
  float t = a;
  slope = 1.0f;
  if constexpr (ACT == QZ_ACT_GELU_TANH) {
    constexpr float k2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float q = a * a;
    t = k2 * a * __fmaf_rn(0.044715f, q, 1.0f);
    slope = k2 * __fmaf_rn(3.0f * 0.044715f, q, 1.0f);
  }
  return __fdividef(1.0f, 1.0f + __expf(-t));
}
// __expf errs by 2 + |1.173 a| ulp at most and __fdividef by 2, so p is within about 2^-21 of
// its value for |a| <= 4 and the error stays far below the bf16 rounding of the result (2^-9)
// up to |a| = 88, where exp(-a) leaves fp32.  __fdividef(1, y) is 0 for y > 2^126, which is
// the limit of p there.
template <int ACT>
__device__ __forceinline__ float act_value(float a) {
  float slope;
  const float p = act_gate<ACT>(a, slope);
  // -inf: p = 0 and the limit is -0, not NaN
  return a == -__int_as_float(0x7f800000) ? -0.0f : a * p;
}
template <int ACT>
__device__ __forceinline__ float act_derivative(float a, float& value) {
  float slope;
  const float p = act_gate<ACT>(a, slope);
  const bool ninf = a == -__int_as_float(0x7f800000);
  value = ninf ? -0.0f : a * p;
  const float q = p * (1.0f - p);
  // where p has reached 0 or 1 the second term is 0 (its factors may be infinite)
  return q == 0.0f ? p : __fmaf_rn(a * slope, q, p);
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  uint16_t h;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
  return h;
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float bf16_float(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

}  // namespace qz
