// qz_norm.cu -- layer norm over rows and its gradients (include/qz.h, qz_layer_norm).
//
//   mean = sum x / C,  v = sum (x - mean)^2 / C,  rstd = 1 / sqrt(v + eps),
//   n = (x - mean) rstd,  y = n w + b;
//   t = dy w,  dx = rstd (t - sum t / C - n sum (t n) / C),  dw = sum_rows dy n,  db = sum_rows dy.
//
// Bound by HBM: the forward pass reads x and writes y, the backward pass reads dy and x and
// writes dx; everything else is per row or per column.  So a row is read once and held in
// registers, 16 values a thread (kPer), by 32 to 1024 threads (TPR, the smallest power of two
// that covers the row): the squares are taken about the mean from the registers, a second pass
// over the chip, not over memory.  Rows longer than 16384 are read again from L2 instead.
#include <climits>
#include <cstdint>

#include "qz_device.cuh"
#include "qz_internal.h"
#include "qz_weight.cuh"

namespace qz {
namespace {

constexpr int kPer = 16;           // values of a row per thread
constexpr int kMaxParts = 304;     // partial column sums in the workspace: two per SM
constexpr int kMaxHeld = 1024 * kPer;

struct NormArgs {
  const void *x, *dy;
  void* y;  // y or dx
  int64_t ld_x, ld_dy, ld_y, rows, cols;
  const float *weight, *bias, *mean_in, *rstd_in;
  float *mean, *rstd;
  float eps;
  float* parts;  // [gridDim.x][2][cols] partial dweight, dbias; null: not computed
};

// 16 values of a row per thread in chunks of E consecutive ones: chunk i of thread l starts at
// column E (i TPR + l).  E = 16 bytes' worth where rows are 16-byte aligned, else 1.
template <int DT, int E>
struct RowRegs {
  static constexpr int kChunks = kPer / E;
  static constexpr int kWords = DT == QZ_BF16 && E > 1 ? kPer / 2 : kPer;
  uint32_t raw[kWords];

  template <int TPR>
  __device__ __forceinline__ void load(const void* base, int64_t off, int l, int cols) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = E * (i * TPR + l);
      if constexpr (E == 1) {
        if constexpr (DT == QZ_BF16) raw[i] = c < cols ? static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(base) + off + c)) << 16 : 0u;
        else raw[i] = c < cols ? __ldg(static_cast<const uint32_t*>(base) + off + c) : 0u;
      } else {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (c < cols) v = ld16B(static_cast<const char*>(base) + (off + c) * (16 / E));
        raw[4 * i] = v.x;
        raw[4 * i + 1] = v.y;
        raw[4 * i + 2] = v.z;
        raw[4 * i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (DT == QZ_BF16 && E > 1) {
      const uint32_t w = raw[j >> 1];
      return __uint_as_float((j & 1) ? w & 0xffff0000u : w << 16);
    } else {
      return __uint_as_float(raw[j]);
    }
  }
  template <int TPR>
  static __device__ __forceinline__ int column(int j, int l) { return E * ((j / E) * TPR + l) + j % E; }

  template <int TPR>
  static __device__ __forceinline__ void store(void* base, int64_t off, int l, int cols, const float (&v)[kPer]) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = E * (i * TPR + l);
      if (c >= cols) continue;
      if constexpr (E == 1) {
        store_elem<DT>(base, off + c, v[i]);
      } else {
        uint4 o;
        if constexpr (DT == QZ_BF16)
          o = make_uint4(bf16x2_bits(v[8 * i], v[8 * i + 1]), bf16x2_bits(v[8 * i + 2], v[8 * i + 3]),
                         bf16x2_bits(v[8 * i + 4], v[8 * i + 5]), bf16x2_bits(v[8 * i + 6], v[8 * i + 7]));
        else
          o = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                         __float_as_uint(v[4 * i + 3]));
        *reinterpret_cast<uint4*>(static_cast<char*>(base) + (off + c) * (16 / E)) = o;
      }
    }
  }
};

// The parameters of this thread's columns (`dflt` where there are none, and past the row's end), in
// 16-byte loads where the row's chunks allow them.
template <int E, int TPR>
__device__ __forceinline__ void load_params(float (&w)[kPer], const float* base, float dflt, int l, int cols) {
  if constexpr (E == 1) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int c = j * TPR + l;
      w[j] = base && c < cols ? __ldg(base + c) : dflt;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPer; j += 4) {
      const int c = E * ((j / E) * TPR + l) + j % E;
      float4 v = make_float4(dflt, dflt, dflt, dflt);
      if (base && c < cols) v = __ldg(reinterpret_cast<const float4*>(base + c));
      w[j] = v.x;
      w[j + 1] = v.y;
      w[j + 2] = v.z;
      w[j + 3] = v.w;
    }
  }
}

// Sums of (a, b) over the TPR threads of a row: shuffles, then the warps' sums through shared
// memory behind a barrier of the row's threads alone (number 1 + group).  `buf` alternates, so
// the next row's sums need no second barrier.
template <int TPR>
__device__ __forceinline__ void row_sums(float& a, float& b, float2* buf, int group) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(kFull, a, o);
    b += __shfl_xor_sync(kFull, b, o);
  }
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int w = (threadIdx.x % TPR) / 32;
    if ((threadIdx.x & 31) == 0) buf[w] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(TPR) : "memory");
    float2 s = (threadIdx.x & 31) < W ? buf[threadIdx.x & 31] : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      s.x += __shfl_xor_sync(kFull, s.x, o);
      s.y += __shfl_xor_sync(kFull, s.y, o);
    }
    a = s.x;
    b = s.y;
  }
}

template <int DT, int E, int TPR>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_forward_kernel(const NormArgs a) {
  constexpr int kBlock = TPR < 256 ? 256 : TPR, G = kBlock / TPR;
  using R = RowRegs<DT, E>;
  __shared__ float2 sums[G][2][TPR > 32 ? TPR / 32 : 1];
  const int group = threadIdx.x / TPR, l = threadIdx.x % TPR, cols = static_cast<int>(a.cols);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * G + group;
  if (row >= a.rows) return;
  R x;
  x.template load<TPR>(a.x, row * a.ld_x, l, cols);
  float s = 0.0f, none = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) s += x.get(j);
  row_sums<TPR>(s, none, sums[group][0], group);
  const float inv = 1.0f / static_cast<float>(cols), mean = s * inv;
  float q = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (R::template column<TPR>(j, l) < cols) {
      const float d = x.get(j) - mean;
      q = __fmaf_rn(d, d, q);
    }
  row_sums<TPR>(q, none, sums[group][1], group);
  const float rstd = 1.0f / sqrtf(q * inv + a.eps);
  if (l == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  float y[kPer], w[kPer], b[kPer];
  load_params<E, TPR>(w, a.weight, 1.0f, l, cols);
  load_params<E, TPR>(b, a.bias, 0.0f, l, cols);
#pragma unroll
  for (int j = 0; j < kPer; ++j) y[j] = __fmaf_rn((x.get(j) - mean) * rstd, w[j], b[j]);
  R::template store<TPR>(a.y, row * a.ld_y, l, cols, y);
}

// A thread keeps its 16 columns from row to row, so the column sums of dy n and dy stay in its
// registers; at the end a block adds its groups' sums in group order and writes one partial.
template <int DT, int E, int TPR, bool PARAMS>
__global__ void __launch_bounds__(TPR < 512 ? 512 : TPR) norm_backward_kernel(const NormArgs a) {
  constexpr int kBlock = TPR < 512 ? 512 : TPR, G = kBlock / TPR;
  using R = RowRegs<DT, E>;
  extern __shared__ float columns[];  // [2][cols] where G > 1
  __shared__ float2 sums[G][2][TPR > 32 ? TPR / 32 : 1];
  const int group = threadIdx.x / TPR, l = threadIdx.x % TPR, cols = static_cast<int>(a.cols);
  const float inv = 1.0f / static_cast<float>(cols);
  float w[kPer], dw[kPer] = {}, db[kPer] = {};
  load_params<E, TPR>(w, a.weight, 1.0f, l, cols);
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + group;
  R x, dy;
  float mean = 0.0f, rstd = 0.0f;
  const auto fetch = [&](int64_t r) {
    x.template load<TPR>(a.x, r * a.ld_x, l, cols);
    dy.template load<TPR>(a.dy, r * a.ld_dy, l, cols);
    mean = __ldg(a.mean_in + r);
    rstd = __ldg(a.rstd_in + r);
  };
  if (row < a.rows) fetch(row);
  for (int flip = 0; row < a.rows; row += step, flip ^= 1) {
    float t[kPer], n[kPer], s1 = 0.0f, s2 = 0.0f;
    const float rs = rstd;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float d = dy.get(j);  // 0 past the row's end
      n[j] = (x.get(j) - mean) * rstd;
      t[j] = d * w[j];
      if (R::template column<TPR>(j, l) < cols) {
        s1 += t[j];
        s2 = __fmaf_rn(t[j], n[j], s2);
        if constexpr (PARAMS) {
          dw[j] = __fmaf_rn(d, n[j], dw[j]);
          db[j] += d;
        }
      }
    }
    if (row + step < a.rows) fetch(row + step);  // in flight during the sums
    row_sums<TPR>(s1, s2, sums[group][flip], group);
    s1 *= inv;
    s2 *= inv;
#pragma unroll
    for (int j = 0; j < kPer; ++j) t[j] = rs * (t[j] - s1 - n[j] * s2);
    R::template store<TPR>(a.y, row * a.ld_y, l, cols, t);
  }
  if constexpr (PARAMS) {
    float* out = a.parts + static_cast<int64_t>(blockIdx.x) * 2 * cols;
    if constexpr (G > 1) {
      for (int g = 0; g < G; ++g) {
        if (group == g) {
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const int c = R::template column<TPR>(j, l);
            if (c < cols) {
              columns[c] = g ? columns[c] + dw[j] : dw[j];
              columns[cols + c] = g ? columns[cols + c] + db[j] : db[j];
            }
          }
        }
        __syncthreads();
      }
      for (int i = threadIdx.x; i < 2 * cols; i += kBlock) out[i] = columns[i];
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int c = R::template column<TPR>(j, l);
        if (c < cols) {
          out[c] = dw[j];
          out[cols + c] = db[j];
        }
      }
    }
  }
}

// Sum of the blocks' partials: 32 columns a block, eight threads a column over every eighth part.
__global__ void __launch_bounds__(256) norm_parts_kernel(const float* parts, int n_parts, int64_t cols, float* dw, float* db) {
  __shared__ float s[8][33];
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;
  const int k = threadIdx.x / 32;
  float v = 0.0f;
  if (i < 2 * cols)
    for (int p = k; p < n_parts; p += 8) v += parts[p * 2 * cols + i];
  s[k][threadIdx.x % 32] = v;
  __syncthreads();
  if (k == 0 && i < 2 * cols) {
#pragma unroll
    for (int j = 1; j < 8; ++j) v += s[j][threadIdx.x];
    if (i < cols) dw[i] = v;
    else db[i - cols] = v;
  }
}

// ---- rows longer than kMaxHeld: a block of 1024 threads a row, the row read again from L2 ------
constexpr int kLong = 1024;

template <int DT>
__global__ void __launch_bounds__(kLong) norm_forward_long_kernel(const NormArgs a) {
  __shared__ float2 sums[2][kLong / 32];
  const float inv = 1.0f / static_cast<float>(a.cols);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t off = row * a.ld_x;
    float s = 0.0f, none = 0.0f, q = 0.0f;
    for (int64_t c = threadIdx.x; c < a.cols; c += kLong) s += load_elem<DT>(a.x, off + c);
    row_sums<kLong>(s, none, sums[0], 0);
    const float mean = s * inv;
    for (int64_t c = threadIdx.x; c < a.cols; c += kLong) {
      const float d = load_elem<DT>(a.x, off + c) - mean;
      q = __fmaf_rn(d, d, q);
    }
    row_sums<kLong>(q, none, sums[1], 0);
    const float rstd = 1.0f / sqrtf(q * inv + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int64_t c = threadIdx.x; c < a.cols; c += kLong) {
      const float w = a.weight ? __ldg(a.weight + c) : 1.0f, b = a.bias ? __ldg(a.bias + c) : 0.0f;
      store_elem<DT>(a.y, row * a.ld_y + c, __fmaf_rn((load_elem<DT>(a.x, off + c) - mean) * rstd, w, b));
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(kLong) norm_backward_long_kernel(const NormArgs a) {
  __shared__ float2 sums[2][kLong / 32];
  const float inv = 1.0f / static_cast<float>(a.cols);
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
    const float mean = __ldg(a.mean_in + row), rstd = __ldg(a.rstd_in + row);
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < a.cols; c += kLong) {
      const float t = load_elem<DT>(a.dy, row * a.ld_dy + c) * (a.weight ? __ldg(a.weight + c) : 1.0f);
      s1 += t;
      s2 = __fmaf_rn(t, (load_elem<DT>(a.x, row * a.ld_x + c) - mean) * rstd, s2);
    }
    row_sums<kLong>(s1, s2, sums[flip], 0);
    s1 *= inv;
    s2 *= inv;
    for (int64_t c = threadIdx.x; c < a.cols; c += kLong) {
      const float t = load_elem<DT>(a.dy, row * a.ld_dy + c) * (a.weight ? __ldg(a.weight + c) : 1.0f);
      const float n = (load_elem<DT>(a.x, row * a.ld_x + c) - mean) * rstd;
      store_elem<DT>(a.y, row * a.ld_y + c, rstd * (t - s1 - n * s2));
    }
  }
}
// partial column sums of rows blockIdx.y, + gridDim.y, ...: a thread a column
template <int DT>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormArgs a) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float d = load_elem<DT>(a.dy, row * a.ld_dy + c);
    dw = __fmaf_rn(d, (load_elem<DT>(a.x, row * a.ld_x + c) - __ldg(a.mean_in + row)) * __ldg(a.rstd_in + row), dw);
    db += d;
  }
  float* out = a.parts + static_cast<int64_t>(blockIdx.y) * 2 * a.cols;
  out[c] = dw;
  out[a.cols + c] = db;
}

__global__ void __launch_bounds__(256) zero_columns_kernel(float* dw, float* db, int64_t cols) {
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; c < cols; c += static_cast<int64_t>(gridDim.x) * 256)
    dw[c] = db[c] = 0.0f;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int DT, int E, int TPR>
qz_status run_forward(const NormArgs& a, cudaStream_t s) {
  constexpr int kBlock = TPR < 256 ? 256 : TPR, G = kBlock / TPR;
  const int64_t grid = (a.rows + G - 1) / G;
  norm_forward_kernel<DT, E, TPR><<<static_cast<unsigned>(grid), kBlock, 0, s>>>(a);
  return launch_status();
}

template <int DT, int E, int TPR>
qz_status run_backward(const NormArgs& a, int parts, cudaStream_t s) {
  constexpr int kBlock = TPR < 512 ? 512 : TPR, G = kBlock / TPR;
  const int smem = a.parts && G > 1 ? static_cast<int>(a.cols) * 8 : 0;
  if (a.parts) norm_backward_kernel<DT, E, TPR, true><<<parts, kBlock, smem, s>>>(a);
  else norm_backward_kernel<DT, E, TPR, false><<<parts, kBlock, smem, s>>>(a);
  return launch_status();
}

template <int DT, int E>
qz_status run_held(const NormArgs& a, bool backward, int parts, cudaStream_t s) {
  int tpr = 32;
  while (tpr * kPer < a.cols) tpr *= 2;
  switch (tpr) {
    case 32: return backward ? run_backward<DT, E, 32>(a, parts, s) : run_forward<DT, E, 32>(a, s);
    case 64: return backward ? run_backward<DT, E, 64>(a, parts, s) : run_forward<DT, E, 64>(a, s);
    case 128: return backward ? run_backward<DT, E, 128>(a, parts, s) : run_forward<DT, E, 128>(a, s);
    case 256: return backward ? run_backward<DT, E, 256>(a, parts, s) : run_forward<DT, E, 256>(a, s);
    case 512: return backward ? run_backward<DT, E, 512>(a, parts, s) : run_forward<DT, E, 512>(a, s);
    default: return backward ? run_backward<DT, E, 1024>(a, parts, s) : run_forward<DT, E, 1024>(a, s);
  }
}

template <int DT>
qz_status run_norm(const NormArgs& a, bool backward, int parts, cudaStream_t s) {
  constexpr int E = DT == QZ_BF16 ? 8 : 4;
  if (a.cols <= kMaxHeld) {
    const bool vec = aligned(a.weight, 16) && aligned(a.bias, 16) && a.cols % E == 0 && a.ld_x % E == 0 && a.ld_y % E == 0 && a.ld_dy % E == 0 && aligned(a.x, 16) &&
                     aligned(a.y, 16) && aligned(a.dy, 16);
    return vec ? run_held<DT, E>(a, backward, parts, s) : run_held<DT, 1>(a, backward, parts, s);
  }
  const int grid = static_cast<int>(a.rows < 2 * sm_count() ? a.rows : 2 * sm_count());
  if (!backward) {
    norm_forward_long_kernel<DT><<<grid, kLong, 0, s>>>(a);
    return launch_status();
  }
  norm_backward_long_kernel<DT><<<grid, kLong, 0, s>>>(a);
  if (a.parts) norm_columns_kernel<DT><<<dim3(static_cast<unsigned>((a.cols + 255) / 256), parts), 256, 0, s>>>(a);
  return launch_status();
}

// blocks of the backward pass, one partial column sum each
int parts_for(int64_t rows, int64_t cols) {
  int64_t per = 1;  // rows a block works on at once
  if (cols <= kMaxHeld) {
    int tpr = 32;
    while (tpr * kPer < cols) tpr *= 2;
    per = tpr < 512 ? 512 / tpr : 1;
  }
  const int64_t want = (rows + per - 1) / per;
  return static_cast<int>(want < kMaxParts ? want : kMaxParts);
}

qz_status check_rows(int32_t dtype, int64_t rows, int64_t cols) {
  if (dtype != QZ_BF16 && dtype != QZ_F32) return QZ_ERR_ENUM;
  if (rows < 0 || cols < 0 || (cols == 0 && rows > 0)) return QZ_ERR_SHAPE;
  if (rows >= (int64_t{1} << 31) || cols >= (int64_t{1} << 31)) return QZ_ERR_UNSUPPORTED;
  return QZ_OK;
}
qz_status check_ld(int64_t rows, int64_t cols, int64_t ld) {
  return ld < cols || (rows > 0 && ld > (INT64_MAX / 8) / rows) ? QZ_ERR_SHAPE : QZ_OK;
}

}  // namespace
}  // namespace qz

using namespace qz;

extern "C" qz_status qz_layer_norm(int32_t dtype, const void* x, int64_t ld_x, int64_t rows, int64_t cols,
                                   const float* weight, const float* bias, float eps, void* y, int64_t ld_y,
                                   float* mean, float* rstd, qz_stream_t stream) {
  qz_status st = check_rows(dtype, rows, cols);
  if (st != QZ_OK) return st;
  if (!(eps >= 0.0f)) return QZ_ERR_SHAPE;
  if ((st = check_ld(rows, cols, ld_x)) != QZ_OK || (st = check_ld(rows, cols, ld_y)) != QZ_OK) return st;
  if (rows == 0) return QZ_OK;
  if (!x || !y) return QZ_ERR_NULL;
  const size_t e = dtype == QZ_BF16 ? 2 : 4;
  if (!aligned(x, e) || !aligned(y, e) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
    return QZ_ERR_ALIGN;
  NormArgs a{};
  a.x = x;
  a.y = y;
  a.ld_x = ld_x;
  a.ld_y = ld_y;
  a.rows = rows;
  a.cols = cols;
  a.weight = weight;
  a.bias = bias;
  a.mean = mean;
  a.rstd = rstd;
  a.eps = eps;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == QZ_BF16 ? run_norm<QZ_BF16>(a, false, 0, s) : run_norm<QZ_F32>(a, false, 0, s);
}

extern "C" size_t qz_layer_norm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return static_cast<size_t>(parts_for(rows, cols)) * 2 * static_cast<size_t>(cols) * sizeof(float);
}

extern "C" qz_status qz_layer_norm_backward(int32_t dtype, const void* dy, int64_t ld_dy, const void* x,
                                            int64_t ld_x, int64_t rows, int64_t cols, const float* mean,
                                            const float* rstd, const float* weight, void* dx, int64_t ld_dx,
                                            float* dweight, float* dbias, void* ws, size_t ws_bytes,
                                            qz_stream_t stream) {
  qz_status st = check_rows(dtype, rows, cols);
  if (st != QZ_OK) return st;
  if ((st = check_ld(rows, cols, ld_dy)) != QZ_OK || (st = check_ld(rows, cols, ld_x)) != QZ_OK ||
      (st = check_ld(rows, cols, ld_dx)) != QZ_OK)
    return st;
  if ((dweight == nullptr) != (dbias == nullptr)) return QZ_ERR_NULL;
  if (!aligned(dweight, 4) || !aligned(dbias, 4)) return QZ_ERR_ALIGN;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dweight && cols) {
      zero_columns_kernel<<<static_cast<int>(cols < 262144 ? (cols + 255) / 256 : 1024), 256, 0, s>>>(dweight, dbias, cols);
      return launch_status();
    }
    return QZ_OK;
  }
  if (!dy || !x || !mean || !rstd || !dx) return QZ_ERR_NULL;
  const size_t e = dtype == QZ_BF16 ? 2 : 4;
  if (!aligned(dy, e) || !aligned(x, e) || !aligned(dx, e) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(weight, 4))
    return QZ_ERR_ALIGN;
  if (dweight) {
    if (!ws || ws_bytes < qz_layer_norm_backward_workspace(rows, cols)) return QZ_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return QZ_ERR_ALIGN;
  }
  NormArgs a{};
  a.x = x;
  a.dy = dy;
  a.y = dx;
  a.ld_x = ld_x;
  a.ld_dy = ld_dy;
  a.ld_y = ld_dx;
  a.rows = rows;
  a.cols = cols;
  a.weight = weight;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.parts = dweight ? static_cast<float*>(ws) : nullptr;
  const int parts = parts_for(rows, cols);
  st = dtype == QZ_BF16 ? run_norm<QZ_BF16>(a, true, parts, s) : run_norm<QZ_F32>(a, true, parts, s);
  if (st != QZ_OK || !dweight) return st;
  norm_parts_kernel<<<static_cast<unsigned>((2 * cols + 31) / 32), 256, 0, s>>>(a.parts, parts, cols, dweight, dbias);
  return launch_status();
}
