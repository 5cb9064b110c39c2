// qz_rotary.cu -- rotation of queries and keys by their positions and its gradient (include/qz.h,
// qz_rotary), and the table of cosines and sines.
//
//   a' = a c - b s,  b' = b c + a s  per pair, c and s of the token's position; backward: -s
//
// One pass: x read, y written, and a table row per token that every head shares: bound by HBM, of which it reaches
// 70 %.  A thread takes the same elements of several heads, for one look at the table, in 16-byte pieces; four loads each
// of 1024 threads are more in flight than HBM needs, so that what is missing is likely that every thread loads, waits and
// stores once and ends (no persistent form was tried).  GPU times:
//   bf16, 8192 tokens x 32 heads x 128, adjacent pairs (139 MB)   29.2 us, 4.75 TB/s  (one head a thread, 64-bit places: 39)
//   fp32, backward of 4093 x 40 x 80, 10 pairs (105 MB)           22.6 us, 4.65 TB/s  (rotary_quad_kernel)
//   one token                                                     2.3 us, all of it launch
#include "qz_rotary.cuh"

#include <climits>
#include <cstdint>
#include <type_traits>

#include "qz_cache.h"
#include "qz_internal.h"

namespace qz {
namespace {

constexpr int kRotThreads = 256;

struct RotaryArgs {
  RotaryView r;
  const void* x;
  void* y;
  int64_t ld_x, hd_x, ld_y, hd_y;
  const int32_t* positions;
  int32_t tokens, heads, dim;
  int32_t units;  // threads of a vector
  float sign;
};

// A thread's token, element group and first head: I is 32 bits wide where all of the threads' numbers are (a
// division in 64 bits costs as much as the rest).
template <class I>
__device__ __forceinline__ bool place(const RotaryArgs& a, int groups, int64_t& t, int& u, int& h) {
  const I i = static_cast<I>(blockIdx.x) * kRotThreads + threadIdx.x, row = i / static_cast<I>(a.units);
  u = static_cast<int>(i - row * static_cast<I>(a.units));
  const I token = row / static_cast<I>(groups);
  h = static_cast<int>(row - token * static_cast<I>(groups));
  t = static_cast<int64_t>(token);
  return t < a.tokens;
}

// Whole pieces (rotary_vec): a thread rotates the same 16 elements of kHeads heads of one token, whose cos and sin
// it loads once.
constexpr int kHeads = 2;
template <int DT, class I>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryArgs a) {
  const int groups = (a.heads + kHeads - 1) / kHeads;
  int64_t t;
  int u, h0;
  if (!place<I>(a, groups, t, u, h0)) return;
  int o0, o1;
  unit_offsets<true>(a.r, u, o0, o1);
  float v[kHeads][16];
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {  // heads h0, h0 + groups
    const int h = min(h0 + k * groups, a.heads - 1);
    const int64_t base = t * a.ld_x + h * a.hd_x;
    load8<DT>(a.x, base + o0, v[k]);
    load8<DT>(a.x, base + o1, v[k] + 8);
  }
  if (16 * u < 2 * a.r.pairs) {
    Turns turns;
    load_turns(a.r, u, a.positions ? __ldg(a.positions + t) : t, a.sign, turns);
#pragma unroll
    for (int k = 0; k < kHeads; ++k) turn_unit(a.r, turns, v[k]);
  }
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    const int h = h0 + k * groups;
    if (h >= a.heads) break;
    const int64_t base = t * a.ld_y + h * a.hd_y;
    store8v<DT>(a.y, base + o0, v[k]);
    store8v<DT>(a.y, base + o1, v[k] + 8);
  }
}

// Four elements in a row of kQuadHeads heads, any number of pairs: their partners are loaded beside them, so that y
// is not x.  (fp32, 4093 tokens of 40 heads of 80 elements, 10 pairs: 62 us by single elements.)
constexpr int kQuadHeads = 4;
template <int DT>
__device__ __forceinline__ void load4(const void* x, int64_t at, float (&v)[4]) {
  if constexpr (DT == QZ_BF16) {
    const uint2 b = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x) + at));
    v[0] = __uint_as_float(b.x << 16), v[1] = __uint_as_float(b.x & 0xffff0000u);
    v[2] = __uint_as_float(b.y << 16), v[3] = __uint_as_float(b.y & 0xffff0000u);
  } else {
    const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(x) + at));
    v[0] = b.x, v[1] = b.y, v[2] = b.z, v[3] = b.w;
  }
}
template <int DT, class I>
__global__ void __launch_bounds__(kRotThreads) rotary_quad_kernel(const RotaryArgs a) {
  const int groups = (a.heads + kQuadHeads - 1) / kQuadHeads, pairs = a.r.pairs;
  int64_t t;
  int u, h0;
  if (!place<I>(a, groups, t, u, h0)) return;
  const int d = 4 * u;
  float v[kQuadHeads][4];
#pragma unroll
  for (int k = 0; k < kQuadHeads; ++k) load4<DT>(a.x, t * a.ld_x + min(h0 + k * groups, a.heads - 1) * a.hd_x + d, v[k]);
  if (d < 2 * pairs) {
    const int64_t pos = a.positions ? __ldg(a.positions + t) : t;
    const bool in = pos >= 0 && pos < a.r.positions;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int z = d + e;
      if (z >= 2 * pairs) break;
      const bool second = a.r.interleaved ? z & 1 : z >= pairs;
      const int i = a.r.interleaved ? z >> 1 : second ? z - pairs : z, other = a.r.interleaved ? z ^ 1 : second ? z - pairs : z + pairs;
      const float c = in ? __ldg(a.r.cos + pos * pairs + i) : __uint_as_float(0x7fc00000u);
      const float s = (in ? __ldg(a.r.sin + pos * pairs + i) : 0.0f) * a.sign;
#pragma unroll
      for (int k = 0; k < kQuadHeads; ++k) {
        const float w = load_elem<DT>(a.x, t * a.ld_x + min(h0 + k * groups, a.heads - 1) * a.hd_x + other);
        // x1 c - x2 s, or x2 c + x1 s
        v[k][e] = second ? __fadd_rn(__fmul_rn(v[k][e], c), __fmul_rn(w, s)) : __fsub_rn(__fmul_rn(v[k][e], c), __fmul_rn(w, s));
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kQuadHeads; ++k) {
    const int h = h0 + k * groups;
    if (h >= a.heads) break;
    const int64_t at = t * a.ld_y + h * a.hd_y + d;
    if constexpr (DT == QZ_BF16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) = make_uint2(bf16x2_bits(v[k][0], v[k][1]), bf16x2_bits(v[k][2], v[k][3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) = make_float4(v[k][0], v[k][1], v[k][2], v[k][3]);
  }
}

// Any sizes, strides and alignment: a thread takes one pair, or one element past the pairs.
template <int DT, class I>
__global__ void __launch_bounds__(kRotThreads) rotary_any_kernel(const RotaryArgs a) {
  int64_t t;
  int u, h;
  if (!place<I>(a, a.heads, t, u, h)) return;
  const int64_t from = t * a.ld_x + h * a.hd_x, to = t * a.ld_y + h * a.hd_y;
  if (u >= a.r.pairs) {
    const int d = u + a.r.pairs;
    store_elem<DT>(a.y, to + d, load_elem<DT>(a.x, from + d));
    return;
  }
  const int d0 = a.r.interleaved ? 2 * u : u, d1 = a.r.interleaved ? d0 + 1 : u + a.r.pairs;
  const int64_t pos = a.positions ? __ldg(a.positions + t) : t;
  float v0 = load_elem<DT>(a.x, from + d0), v1 = load_elem<DT>(a.x, from + d1);
  if (pos < 0 || pos >= a.r.positions) {
    v0 = v1 = __uint_as_float(0x7fc00000u);
  } else {
    turn(v0, v1, __ldg(a.r.cos + pos * a.r.pairs + u), __ldg(a.r.sin + pos * a.r.pairs + u) * a.sign);
  }
  store_elem<DT>(a.y, to + d0, v0);
  store_elem<DT>(a.y, to + d1, v1);
}

__global__ void __launch_bounds__(kRotThreads) rotary_fill_kernel(const double* turns, int64_t positions, int64_t pairs,
                                                                  double amplitude, float* cos_out, float* sin_out) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRotThreads + threadIdx.x; i < positions * pairs;
       i += static_cast<int64_t>(gridDim.x) * kRotThreads) {
    double s, c;
    sincos(static_cast<double>(i / pairs) * turns[i % pairs], &s, &c);
    cos_out[i] = static_cast<float>(amplitude * c);
    sin_out[i] = static_cast<float>(amplitude * s);
  }
}

qz_status run_rotary(const qz_rotary_table* table, int32_t dtype, const void* x, int64_t ld_x, int64_t hd_x, int64_t tokens,
                     int64_t heads, int64_t dim, const int32_t* positions, void* y, int64_t ld_y, int64_t hd_y, float sign,
                     cudaStream_t s) {
  if (!table) return QZ_ERR_NULL;
  if (dtype != QZ_BF16 && dtype != QZ_F32) return QZ_ERR_ENUM;
  qz_status st;
  if ((st = check_vectors(tokens, heads, dim, ld_x, hd_x)) != QZ_OK || (st = check_vectors(tokens, heads, dim, ld_y, hd_y)) != QZ_OK ||
      (st = check_rotary_table(table, dim)) != QZ_OK)
    return st;
  if (tokens == 0 || heads == 0 || dim == 0) return QZ_OK;
  if (!x || !y) return QZ_ERR_NULL;
  if (moves_in_place(x, ld_x, hd_x, y, ld_y, hd_y, tokens, heads)) return QZ_ERR_SHAPE;
  const int64_t e = dtype == QZ_BF16 ? 2 : 4;
  if (!is_aligned(x, e) || !is_aligned(y, e) || !is_aligned(positions, 4)) return QZ_ERR_ALIGN;
  RotaryArgs a{};
  a.r = view_of(table);
  a.x = x, a.y = y;
  a.ld_x = ld_x, a.hd_x = hd_x, a.ld_y = ld_y, a.hd_y = hd_y;
  a.positions = positions;
  a.tokens = static_cast<int32_t>(tokens), a.heads = static_cast<int32_t>(heads), a.dim = static_cast<int32_t>(dim);
  a.sign = sign;
  const bool vec = rotary_vec(a.r, dim) && rows_vec(x, e, tokens, ld_x, heads, hd_x) && rows_vec(y, e, tokens, ld_y, heads, hd_y);
  // four-element pieces: 16 bytes of fp32, 8 of bf16
  const auto quads = [&](const void* p, int64_t ld, int64_t hd) {
    return is_aligned(p, 4 * e) && (tokens <= 1 || ld % 4 == 0) && (heads <= 1 || hd % 4 == 0);
  };
  const bool quad = !vec && x != y && dim % 4 == 0 && quads(x, ld_x, hd_x) && quads(y, ld_y, hd_y);
  a.units = static_cast<int32_t>(vec ? dim / 16 : quad ? dim / 4 : dim - table->pairs);
  const int each = vec ? kHeads : quad ? kQuadHeads : 1;
  const int64_t threads = tokens * ((heads + each - 1) / each) * a.units, blocks = (threads + kRotThreads - 1) / kRotThreads;
  if (blocks > INT32_MAX) return QZ_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(blocks);
  const bool small = blocks * kRotThreads <= INT32_MAX;
  const auto run = [&](auto dt, auto index) {
    constexpr int DT = decltype(dt)::value;
    using I = decltype(index);
    if (vec) rotary_kernel<DT, I><<<grid, kRotThreads, 0, s>>>(a);
    else if (quad) rotary_quad_kernel<DT, I><<<grid, kRotThreads, 0, s>>>(a);
    else rotary_any_kernel<DT, I><<<grid, kRotThreads, 0, s>>>(a);
  };
  using Bf16 = std::integral_constant<int, QZ_BF16>;
  using F32 = std::integral_constant<int, QZ_F32>;
  if (dtype == QZ_BF16) small ? run(Bf16{}, uint32_t{}) : run(Bf16{}, uint64_t{});
  else small ? run(F32{}, uint32_t{}) : run(F32{}, uint64_t{});
  return launch_status();
}

}  // namespace

RotaryView view_of(const qz_rotary_table* t) {
  RotaryView r{};
  if (!t || t->pairs == 0) return r;
  r.cos = t->cos, r.sin = t->sin;
  r.positions = static_cast<int32_t>(t->positions), r.pairs = t->pairs;
  r.interleaved = t->interleaved != 0;
  return r;
}

qz_status check_rotary_table(const qz_rotary_table* t, int64_t dim) {
  if (t->pairs < 0 || 2 * static_cast<int64_t>(t->pairs) > dim || t->positions < (t->pairs > 0 ? 1 : 0)) return QZ_ERR_SHAPE;
  if (t->positions > INT32_MAX) return QZ_ERR_UNSUPPORTED;
  if (t->pairs > 0 && (!t->cos || !t->sin)) return QZ_ERR_NULL;
  if (!is_aligned(t->cos, 4) || !is_aligned(t->sin, 4)) return QZ_ERR_ALIGN;
  return QZ_OK;
}

}  // namespace qz

using namespace qz;

extern "C" qz_status qz_rotary_fill(const double* turns, int64_t positions, int64_t pairs, double amplitude, float* cos,
                                    float* sin, qz_stream_t stream) {
  if (positions < 0 || pairs < 0) return QZ_ERR_SHAPE;
  if (positions > INT32_MAX || pairs > INT32_MAX) return QZ_ERR_UNSUPPORTED;
  if (positions == 0 || pairs == 0) return QZ_OK;
  if (!turns || !cos || !sin) return QZ_ERR_NULL;
  if (!is_aligned(turns, 8) || !is_aligned(cos, 4) || !is_aligned(sin, 4)) return QZ_ERR_ALIGN;
  const int64_t blocks = (positions * pairs + kRotThreads - 1) / kRotThreads;
  rotary_fill_kernel<<<static_cast<unsigned>(blocks < 65536 ? blocks : 65536), kRotThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      turns, positions, pairs, amplitude, cos, sin);
  return launch_status();
}

extern "C" qz_status qz_rotary(const qz_rotary_table* table, int32_t dtype, const void* x, int64_t ld_x, int64_t hd_x,
                               int64_t tokens, int64_t heads, int64_t dim, const int32_t* positions, void* y, int64_t ld_y,
                               int64_t hd_y, qz_stream_t stream) {
  return run_rotary(table, dtype, x, ld_x, hd_x, tokens, heads, dim, positions, y, ld_y, hd_y, 1.0f,
                    reinterpret_cast<cudaStream_t>(stream));
}

extern "C" qz_status qz_rotary_backward(const qz_rotary_table* table, int32_t dtype, const void* dy, int64_t ld_dy,
                                        int64_t hd_dy, int64_t tokens, int64_t heads, int64_t dim, const int32_t* positions,
                                        void* dx, int64_t ld_dx, int64_t hd_dx, qz_stream_t stream) {
  return run_rotary(table, dtype, dy, ld_dy, hd_dy, tokens, heads, dim, positions, dx, ld_dx, hd_dx, -1.0f,
                    reinterpret_cast<cudaStream_t>(stream));
}
