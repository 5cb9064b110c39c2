// qz_rotary.cu -- rotation of queries and keys by their positions and its gradient (include/qz.h,
// qz_rotary), and the table of cosines and sines.
#include "qz_rotary.cuh"

#include <climits>
#include <cstdint>

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

// VEC: a thread rotates the same 16 elements of kHeads heads of one token, whose cos and sin it loads once.
constexpr int kHeads = 4;
template <int DT>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryArgs a) {
  const int groups = (a.heads + kHeads - 1) / kHeads;
  const int64_t per_token = static_cast<int64_t>(groups) * a.units;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRotThreads + threadIdx.x;
  const int64_t t = i / per_token;
  if (t >= a.tokens) return;
  const int rest = static_cast<int>(i - t * per_token), u = rest % a.units, h0 = rest / a.units;
  int o0, o1;
  unit_offsets<true>(a.r, u, o0, o1);
  float v[kHeads][16];
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {  // heads h0, h0 + groups, ...
    const int h = h0 + k * groups;
    if (h >= a.heads) break;
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

// Any sizes, strides and alignment: a thread takes one pair, or one element past the pairs.
template <int DT>
__global__ void __launch_bounds__(kRotThreads) rotary_any_kernel(const RotaryArgs a) {
  const int64_t per_token = static_cast<int64_t>(a.heads) * a.units;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRotThreads + threadIdx.x;
  const int64_t t = i / per_token;
  if (t >= a.tokens) return;
  const int rest = static_cast<int>(i - t * per_token), u = rest % a.units, h = rest / a.units;
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
  a.units = static_cast<int32_t>(vec ? dim / 16 : dim - table->pairs);
  const int64_t threads = tokens * (vec ? (heads + kHeads - 1) / kHeads : heads) * a.units;
  const int64_t blocks = (threads + kRotThreads - 1) / kRotThreads;
  if (blocks > INT32_MAX) return QZ_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (vec) {
    if (dtype == QZ_BF16) rotary_kernel<QZ_BF16><<<grid, kRotThreads, 0, s>>>(a);
    else rotary_kernel<QZ_F32><<<grid, kRotThreads, 0, s>>>(a);
  } else {
    if (dtype == QZ_BF16) rotary_any_kernel<QZ_BF16><<<grid, kRotThreads, 0, s>>>(a);
    else rotary_any_kernel<QZ_F32><<<grid, kRotThreads, 0, s>>>(a);
  }
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
