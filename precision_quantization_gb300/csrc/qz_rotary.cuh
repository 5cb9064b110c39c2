// qz_rotary.cuh -- the rotation of one head's vector by its token's position (include/qz.h, qz_rotary),
// 16 elements a thread.
#pragma once

#include <cstdint>

#include "qz_device.cuh"
#include "qz_weight.cuh"

namespace qz {

struct RotaryView {
  const float *cos, *sin;  // null: no rotation
  int32_t positions, pairs;
  bool interleaved;
};

// A thread's elements: two pieces of 8, at o0 and o1.  Where the pairs come in whole pieces (VEC: pairs a
// multiple of 8, rows 16-byte aligned, dim a multiple of 16) the pieces hold both halves of their pairs:
// pieces u and u + pairs / 8 of the halves' layout, neighbours else.  Otherwise 16 elements in a row, and
// the halves' partners are loaded beside them.
template <bool VEC>
__device__ __forceinline__ void unit_offsets(const RotaryView& r, int u, int& o0, int& o1) {
  o0 = 16 * u;
  o1 = o0 + 8;
  if (VEC && r.cos && !r.interleaved && o0 < 2 * r.pairs) {
    o0 = 8 * u;
    o1 = o0 + r.pairs;
  }
}

template <int DT>
__device__ __forceinline__ void load8(const void* x, int64_t at, float* v) {
  if constexpr (DT == QZ_BF16) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
template <int DT>
__device__ __forceinline__ void store8v(void* y, int64_t at, const float* v) {
  if constexpr (DT == QZ_BF16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + at) =
        make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(y) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// One pair; the products are rounded apart (the library is compiled without contraction).
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

// The cos and sin that a unit of 16 elements needs (VEC): 8 pairs of one token.
struct Turns {
  float c[8], s[8];
};
__device__ __forceinline__ void load_turns(const RotaryView& r, int u, int64_t pos, float sign, Turns& t) {
  const bool in = pos >= 0 && pos < r.positions;
  const int64_t at = (in ? pos : 0) * r.pairs + 8 * u;
  load8<QZ_F32>(r.cos, at, t.c);
  load8<QZ_F32>(r.sin, at, t.s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.c[i] = in ? t.c[i] : __uint_as_float(0x7fc00000u);
    t.s[i] *= sign;
  }
}
// v: the two pieces of unit u, rotated in place (VEC); units from 2 pairs on pass
__device__ __forceinline__ void turn_unit(const RotaryView& r, const Turns& t, float (&v)[16]) {
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(v[2 * i], v[2 * i + 1], t.c[i], t.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(v[i], v[8 + i], t.c[i], t.s[i]);
  }
}
// Element d of the vector at x, rotated: any sizes and alignment.
template <int DT>
__device__ __forceinline__ float turned(const RotaryView& r, const void* x, int64_t base, int d, int64_t pos, float sign) {
  const float v = load_elem<DT>(x, base + d);
  if (!r.cos || d >= 2 * r.pairs) return v;
  const bool second = r.interleaved ? d & 1 : d >= r.pairs;
  const int i = r.interleaved ? d >> 1 : second ? d - r.pairs : d;
  const int e = r.interleaved ? d ^ 1 : second ? d - r.pairs : d + r.pairs;
  if (pos < 0 || pos >= r.positions) return __uint_as_float(0x7fc00000u);
  const float c = __ldg(r.cos + pos * r.pairs + i), s = __ldg(r.sin + pos * r.pairs + i) * sign;
  float a = v, b = load_elem<DT>(x, base + e);
  if (second) {
    const float t = a;
    a = b;
    b = t;
  }
  turn(a, b, c, s);
  return second ? b : a;
}

inline bool rotary_vec(const RotaryView& r, int64_t dim) {
  return dim % 16 == 0 && r.pairs % 8 == 0 && reinterpret_cast<uintptr_t>(r.cos) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(r.sin) % 16 == 0;
}
// rows of 16-byte pieces
inline bool rows_vec(const void* x, int64_t elem, int64_t tokens, int64_t ld, int64_t heads, int64_t hd) {
  return reinterpret_cast<uintptr_t>(x) % 16 == 0 && (tokens <= 1 || ld * elem % 16 == 0) && (heads <= 1 || hd * elem % 16 == 0);
}
RotaryView view_of(const qz_rotary_table* t);

}  // namespace qz
