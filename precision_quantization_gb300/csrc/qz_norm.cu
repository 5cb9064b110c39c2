// qz_norm.cu -- layer norm over rows and its gradients (include/qz.h, qz_layer_norm).
//
//   mean = sum x / C,  v = sum (x - mean)^2 / C,  rstd = 1 / sqrt(v + eps),
//   n = (x - mean) rstd,  y = n w + b;
//   t = dy w,  dx = rstd (t - sum t / C - n sum (t n) / C),  dw = sum_rows dy n,  db = sum_rows dy.
//
// Bound by HBM: the forward pass reads x and writes y, the backward pass reads dy and x and
// writes dx; everything else is per row or per column.  So a row is read once and held in
// registers, 16 values a thread (kPer), by 32 to 1024 threads (TPR, see threads_per_row): the squares are taken about the mean from the registers, a second pass
// over the chip, not over memory.  The backward pass is persistent, for the column sums, and each
// thread copies its own pieces of the next rows into shared memory (cp.async, kAhead rows ahead).
// Rows longer than 16384 are read again from L2 instead.
//
// Measured, 8192 x 4096 bf16, a pass among others: forward 28.7 us, 4.7 TB/s, bound by L1 (the
// parameters, 8 bytes a column against 4 of x and y) and the two sums one after the other; backward
// 42 us, 4.8 TB/s, 4 of them the join of the blocks' column sums.  (fp32: 42 and 68 us on the GPU.)
// Rows that are not 16-byte aligned take one value a load: 8192 x 4095 bf16 49 and 105 us.
#include <climits>
#include <cstdint>

#include "qz_device.cuh"
#include "qz_internal.h"
#include "qz_pipe.cuh"
#include "qz_weight.cuh"

namespace qz {
namespace {

constexpr int kPer = 16;           // values of a row per thread
constexpr int kMaxParts = 152;     // partial column sums in the workspace: one per SM
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

  // The ring: piece i of thread x of the block in slot d at ((d kChunks + i) threads + x) 16 bytes.
  template <int TPR>
  static __device__ __forceinline__ void copy(uint32_t slot, int threads, const void* base, int64_t off, int l, int cols) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = E * (i * TPR + l);
      if (c < cols)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + (i * threads + threadIdx.x) * 16u),
                     "l"(static_cast<const char*>(base) + (off + c) * (16 / E))
                     : "memory");
    }
  }
  template <int TPR>
  __device__ __forceinline__ void take(const unsigned char* slot, int threads, int l, int cols) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (E * (i * TPR + l) < cols) v = *reinterpret_cast<const uint4*>(slot + (i * threads + threadIdx.x) * 16);
      raw[4 * i] = v.x;
      raw[4 * i + 1] = v.y;
      raw[4 * i + 2] = v.z;
      raw[4 * i + 3] = v.w;
    }
  }
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
  // values 2 i and 2 i + 1
  __device__ __forceinline__ uint64_t pair(int i) const { return pk(get(2 * i), get(2 * i + 1)); }
  // whether they lie in the row; the chunks of E > 1 do wholly or not at all
  template <int TPR>
  static __device__ __forceinline__ uint64_t inside(int i, int l, int cols, uint64_t v) {
    if constexpr (E > 1) return column<TPR>(2 * i, l) < cols ? v : 0ull;
    float a, b;
    upk(v, a, b);
    return pk(column<TPR>(2 * i, l) < cols ? a : 0.0f, column<TPR>(2 * i + 1, l) < cols ? b : 0.0f);
  }
  template <int TPR>
  static __device__ __forceinline__ int column(int j, int l) { return E * ((j / E) * TPR + l) + j % E; }

  template <int TPR>
  static __device__ __forceinline__ void store(void* base, int64_t off, int l, int cols, const uint64_t (&y)[kPer / 2]) {
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) upk(y[i], v[2 * i], v[2 * i + 1]);
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
__device__ __forceinline__ void load_params(uint64_t (&p)[kPer / 2], const float* base, float dflt, int l, int cols) {
  float w[kPer];
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
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) p[i] = pk(w[2 * i], w[2 * i + 1]);
}

// Sums over the TPR threads of a row: shuffles, then the warps' sums through shared memory behind a
// barrier of the row's threads alone (number 1 + group).  `buf` alternates between the sums of a
// row, or of two rows, so no second barrier is needed.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*buf)[N], int group) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int w = (threadIdx.x % TPR) / 32;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[w][i] = v[i];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(TPR) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (W & (W - 1)) == 0 ? buf[threadIdx.x % W][i] : (threadIdx.x & 31) < W ? buf[threadIdx.x & 31][i] : 0.0f;
#pragma unroll
    for (int o = (W & (W - 1)) == 0 ? W / 2 : 16; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
  }
}
// 1 / sqrt(v): the approximation (2 ulp) and one Newton step
__device__ __forceinline__ float rsqrt_of(float v) {
  const float r = rsqrtf(v);
  const float e = __fmaf_rn(-v * r, r, 1.0f);
  // (an infinite r, from v = 0, stays: its correction would be NaN)
  return fabsf(e) <= 1.0f ? __fmaf_rn(0.5f * r, e, r) : r;
}

constexpr int kAhead = 5;  // rows a thread copies ahead at most
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Threads a row takes: the smallest of these that hold it.  (Powers of two alone left half of them idle
// just above one: 4092 x 8200 bf16, forward 72 -> 43 us, backward 152 -> 72 us with 640 for 1024.)
int threads_per_row(int64_t cols) {
  for (int t : {32, 64, 128, 192, 256, 384, 512, 640, 768})
    if (t * kPer >= cols) return t;
  return 1024;
}
// threads of a block of the backward pass
constexpr int norm_block(int tpr) { return tpr == 192 || tpr == 384 ? 384 : tpr < 512 ? 512 : tpr; }
template <int TPR>
constexpr int kNormBlock = norm_block(TPR);
// threads of a block of the forward pass
template <int TPR>
constexpr int kForwardBlock = TPR < 192 ? 256 : TPR;
// The backward pass's ring: a slot is one row of x and dy for every group of the block, and there are
// as many (kAhead + 1 at most) as fit 192 KiB.
template <int DT, int TPR>
constexpr int kNormSlot = 2 * kNormBlock<TPR> * kPer * (DT == QZ_BF16 ? 2 : 4);
template <int DT, int TPR>
constexpr int kNormRoom = 192 * 1024 / kNormSlot<DT, TPR>;
template <int DT, int TPR>
constexpr int kNormSlots = kNormRoom<DT, TPR> > kAhead + 1 ? kAhead + 1 : kNormRoom<DT, TPR>;

// ROWS rows per group of threads and launch: the forward pass keeps nothing from row to row but the
// parameters, which come from L1 and there take more of the wavefronts than the rows themselves; two
// rows share them and the chains of their sums (8192 x 4096 bf16: 33 -> 28.7 us).  (A persistent form with
// the rows copied ahead, as the backward pass has it, was slower: 43 us.)
template <int DT, int E, int TPR, int ROWS>
__global__ void __launch_bounds__(kForwardBlock<TPR>, (ROWS == 2 ? 1024 : 1536) / kForwardBlock<TPR>)
norm_forward_kernel(const NormArgs a) {
  constexpr int kBlock = kForwardBlock<TPR>, G = kBlock / TPR, kChunks = kPer / E;
  using R = RowRegs<DT, E>;
  __shared__ float sums[G][2][TPR > 32 ? TPR / 32 : 1][ROWS];
  const int group = threadIdx.x / TPR, l = threadIdx.x % TPR, cols = static_cast<int>(a.cols);
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * G + group) * ROWS;
  if (row >= a.rows) return;
  R x[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) x[k].template load<TPR>(a.x, (row + k < a.rows ? row + k : row) * a.ld_x, l, cols);
  float s[ROWS], mean[ROWS], rstd[ROWS];
  const float inv = 1.0f / static_cast<float>(cols);
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    s[k] = 0.0f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) s[k] += x[k].get(j);
  }
  row_sums<TPR>(s, sums[group][0], group);
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    mean[k] = s[k] * inv;
    s[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (E * (i * TPR + l) < cols) {  // a chunk lies wholly in the row or not at all
#pragma unroll
        for (int j = E * i; j < E * i + E; ++j) {
          const float d = x[k].get(j) - mean[k];
          s[k] = __fmaf_rn(d, d, s[k]);
        }
      }
    }
  }
  row_sums<TPR>(s, sums[group][1], group);
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    rstd[k] = rsqrt_of(s[k] * inv + a.eps);
    if (l == 0 && row + k < a.rows) {
      if (a.mean) a.mean[row + k] = mean[k];
      if (a.rstd) a.rstd[row + k] = rstd[k];
    }
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = E * (i * TPR + l);
    if (c >= cols) continue;
    float w[E], b[E];
    if constexpr (E == 1) {
      w[0] = a.weight ? __ldg(a.weight + c) : 1.0f;
      b[0] = a.bias ? __ldg(a.bias + c) : 0.0f;
    } else {
#pragma unroll
      for (int j = 0; j < E; j += 4) {
        float4 v = make_float4(1.0f, 1.0f, 1.0f, 1.0f), u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (a.weight) v = __ldg(reinterpret_cast<const float4*>(a.weight + c + j));
        if (a.bias) u = __ldg(reinterpret_cast<const float4*>(a.bias + c + j));
        w[j] = v.x; w[j + 1] = v.y; w[j + 2] = v.z; w[j + 3] = v.w;
        b[j] = u.x; b[j + 1] = u.y; b[j + 2] = u.z; b[j + 3] = u.w;
      }
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      if (row + k >= a.rows) break;
      const int64_t at = (row + k) * a.ld_y + c;
      float y[E];
#pragma unroll
      for (int j = 0; j < E; ++j) y[j] = __fmaf_rn((x[k].get(E * i + j) - mean[k]) * rstd[k], w[j], b[j]);
      if constexpr (E == 1) {
        store_elem<DT>(a.y, at, y[0]);
      } else {
        uint4 o;
        if constexpr (DT == QZ_BF16) o = make_uint4(bf16x2_bits(y[0], y[1]), bf16x2_bits(y[2], y[3]), bf16x2_bits(y[E - 4], y[E - 3]), bf16x2_bits(y[E - 2], y[E - 1]));
        else o = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
        *reinterpret_cast<uint4*>(static_cast<char*>(a.y) + at * (16 / E)) = o;
      }
    }
  }
}

// Rows a group works on at once: a row's sums are a chain of shuffles and a barrier, some 1000 cycles
// whatever the row's length, which two rows share where the ring has room for them (backward pass
// of 8192 x 4096 bf16: 52 -> 40 us).
template <int SLOTS>
constexpr int kNormRows = SLOTS >= 4 ? 2 : 1;

// A thread keeps its 16 columns from row to row, so the column sums of dy n and dy stay in its
// registers; at the end a block adds its groups' sums in group order and writes one partial.
template <int DT, int E, int TPR, bool PARAMS>
__global__ void __launch_bounds__(kNormBlock<TPR>) norm_backward_kernel(const NormArgs a) {
  constexpr int kBlock = kNormBlock<TPR>, G = kBlock / TPR, kSlots = kNormSlots<DT, TPR>, kSlotBytes = kNormSlot<DT, TPR> / 2;  // of one tensor
  constexpr int kRows = kNormRows<kSlots>;
  using R = RowRegs<DT, E>;
  extern __shared__ __align__(16) unsigned char norm_ring_smem[];
  __shared__ float sums[G][2][TPR > 32 ? TPR / 32 : 1][2 * kRows];
  const int group = threadIdx.x / TPR, l = threadIdx.x % TPR, cols = static_cast<int>(a.cols);
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + group, ahead = row;
  int slot = 0, to = 0;
  const auto copy_next = [&]() {
    if constexpr (E > 1) {
      if (ahead < a.rows) {
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(norm_ring_smem)) + to * (2 * kSlotBytes);
        R::template copy<TPR>(at, kBlock, a.x, ahead * a.ld_x, l, cols);
        R::template copy<TPR>(at + kSlotBytes, kBlock, a.dy, ahead * a.ld_dy, l, cols);
      }
      copies_commit();
      ahead += step;
      to = to == kSlots - 1 ? 0 : to + 1;
    }
  };
  // row k of this round: this thread's own pieces, which no other thread reads
  const auto take = [&](int k, R& x, R& dy) {
    if constexpr (E > 1) {
      const int d = slot + k;
      const unsigned char* at = norm_ring_smem + (d >= kSlots ? d - kSlots : d) * (2 * kSlotBytes);
      x.template take<TPR>(at, kBlock, l, cols);
      dy.template take<TPR>(at + kSlotBytes, kBlock, l, cols);
    } else {
      const int64_t r = row + k * step;
      x.template load<TPR>(a.x, r * a.ld_x, l, cols);
      dy.template load<TPR>(a.dy, r * a.ld_dy, l, cols);
    }
  };
  for (int i = 0; i < kSlots - kRows; ++i) copy_next();
  const float inv = 1.0f / static_cast<float>(cols);
  uint64_t w[kPer / 2], dw[kPer / 2] = {}, db[kPer / 2] = {};
  load_params<E, TPR>(w, a.weight, 1.0f, l, cols);
  // mean and rstd one round ahead
  float mean[kRows], rstd[kRows], mean1[kRows], rstd1[kRows];
  const auto stats = [&](int64_t r, float (&m)[kRows], float (&v)[kRows]) {
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t i = r + k * step < a.rows ? r + k * step : a.rows - 1;
      m[k] = __ldg(a.mean_in + i);
      v[k] = __ldg(a.rstd_in + i);
    }
  };
  if (row < a.rows) stats(row, mean1, rstd1);
  for (int flip = 0; row < a.rows; row += kRows * step, flip ^= 1) {
    if constexpr (E > 1) {
#pragma unroll
      for (int k = 0; k < kRows; ++k) copy_next();
      copies_wait<kSlots - kRows>();
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      mean[k] = mean1[k];
      rstd[k] = rstd1[k];
    }
    stats(row + kRows * step, mean1, rstd1);
    float s[2 * kRows], lo, hi;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      s[2 * k] = s[2 * k + 1] = 0.0f;
      if (row + k * step >= a.rows) continue;
      R x, dy;
      take(k, x, dy);
      uint64_t a1 = 0ull, a2 = 0ull;
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) {
        const uint64_t d = dy.pair(i);  // 0 past the row's end, and so t and what it is summed into
        const uint64_t n = R::template inside<TPR>(i, l, cols, mul2(add2(x.pair(i), pk(-mean[k], -mean[k])), pk(rstd[k], rstd[k])));
        const uint64_t t = mul2(d, w[i]);
        a1 = add2(a1, t);
        a2 = fma2(t, n, a2);
        if constexpr (PARAMS) {
          dw[i] = fma2(d, n, dw[i]);
          db[i] = add2(db[i], d);
        }
      }
      upk(a1, lo, hi);
      s[2 * k] = lo + hi;
      upk(a2, lo, hi);
      s[2 * k + 1] = lo + hi;
    }
    row_sums<TPR>(s, sums[group][flip], group);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t r = row + k * step;
      if (r >= a.rows) break;
      R x, dy;
      take(k, x, dy);
      // rstd (t - m1 - n m2) with n = (x - mean) rstd
      const float m1 = -s[2 * k] * inv, m2 = -s[2 * k + 1] * inv * rstd[k];
      uint64_t o[kPer / 2];
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i)
        o[i] = mul2(pk(rstd[k], rstd[k]), add2(fma2(add2(x.pair(i), pk(-mean[k], -mean[k])), pk(m2, m2), mul2(dy.pair(i), w[i])), pk(m1, m1)));
      R::template store<TPR>(a.y, r * a.ld_y, l, cols, o);
    }
    slot += kRows;
    if (slot >= kSlots) slot -= kSlots;
  }
  if constexpr (E > 1) copies_wait<0>();
  if constexpr (PARAMS) {
    float fw[kPer], fb[kPer];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      upk(dw[i], fw[2 * i], fw[2 * i + 1]);
      upk(db[i], fb[2 * i], fb[2 * i + 1]);
    }
    float* out = a.parts + static_cast<int64_t>(blockIdx.x) * 2 * cols;
    if constexpr (G > 1) {
      // every group's sums side by side, then each column's in group order; the ring is idle
      constexpr int kWide = TPR * kPer;
      float* columns = reinterpret_cast<float*>(norm_ring_smem);  // [G][2][kWide]
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kPer; j += E > 1 ? 4 : 1) {
        float* at = columns + group * 2 * kWide + R::template column<TPR>(j, l);
        if constexpr (E > 1) {
          *reinterpret_cast<float4*>(at) = make_float4(fw[j], fw[j + 1], fw[j + 2], fw[j + 3]);
          *reinterpret_cast<float4*>(at + kWide) = make_float4(fb[j], fb[j + 1], fb[j + 2], fb[j + 3]);
        } else {
          at[0] = fw[j];
          at[kWide] = fb[j];
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * cols; i += kBlock) {
        const float* at = columns + (i < cols ? i : i - cols + kWide);
        float v = at[0];
#pragma unroll
        for (int g = 1; g < G; ++g) v += at[g * 2 * kWide];
        out[i] = v;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int c = R::template column<TPR>(j, l);
        if (c < cols) {
          out[c] = fw[j];
          out[cols + c] = fb[j];
        }
      }
    }
  }
}

// Sum of the blocks' partials: 32 columns a block, 32 threads a column over every 32nd part.
__global__ void __launch_bounds__(1024) norm_parts_kernel(const float* parts, int n_parts, int64_t cols, float* dw, float* db) {
  __shared__ float s[32][33];
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;
  const int k = threadIdx.x / 32;
  float v = 0.0f;
  if (i < 2 * cols) {
#pragma unroll 4
    for (int p = k; p < n_parts; p += 32) v += parts[p * 2 * cols + i];
  }
  s[k][threadIdx.x % 32] = v;
  __syncthreads();
  v = s[threadIdx.x % 32][k];  // column k of the block, summed over a warp
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + k;
  if (threadIdx.x % 32 == 0 && c < 2 * cols) {
    if (c < cols) dw[c] = v;
    else db[c - cols] = v;
  }
}

// ---- rows longer than kMaxHeld: a block of 1024 threads a row, the row read again from L2 ------
constexpr int kLong = 1024;

template <int DT>
__global__ void __launch_bounds__(kLong) norm_forward_long_kernel(const NormArgs a) {
  __shared__ float sums[2][kLong / 32][1];
  const float inv = 1.0f / static_cast<float>(a.cols);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t off = row * a.ld_x;
    float s[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < a.cols; c += kLong) s[0] += load_elem<DT>(a.x, off + c);
    row_sums<kLong>(s, sums[0], 0);
    const float mean = s[0] * inv;
    s[0] = 0.0f;
    for (int64_t c = threadIdx.x; c < a.cols; c += kLong) {
      const float d = load_elem<DT>(a.x, off + c) - mean;
      s[0] = __fmaf_rn(d, d, s[0]);
    }
    row_sums<kLong>(s, sums[1], 0);
    const float rstd = rsqrt_of(s[0] * inv + a.eps);
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
  __shared__ float sums[2][kLong / 32][2];
  const float inv = 1.0f / static_cast<float>(a.cols);
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
    const float mean = __ldg(a.mean_in + row), rstd = __ldg(a.rstd_in + row);
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < a.cols; c += kLong) {
      const float t = load_elem<DT>(a.dy, row * a.ld_dy + c) * (a.weight ? __ldg(a.weight + c) : 1.0f);
      s[0] += t;
      s[1] = __fmaf_rn(t, (load_elem<DT>(a.x, row * a.ld_x + c) - mean) * rstd, s[1]);
    }
    row_sums<kLong>(s, sums[flip], 0);
    const float s1 = s[0] * inv, s2 = s[1] * inv;
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
  constexpr int kBlock = kForwardBlock<TPR>, G = kBlock / TPR;
  // two rows a group where the GPU stays full with them
  if (TPR <= 512 && a.rows >= static_cast<int64_t>(2 * sm_count()) * (2048 / kBlock) * G) {
    constexpr int kRows = TPR <= 512 ? 2 : 1;
    norm_forward_kernel<DT, E, TPR, kRows><<<static_cast<unsigned>((a.rows + kRows * G - 1) / (kRows * G)), kBlock, 0, s>>>(a);
  } else {
    norm_forward_kernel<DT, E, TPR, 1><<<static_cast<unsigned>((a.rows + G - 1) / G), kBlock, 0, s>>>(a);
  }
  return launch_status();
}

template <int DT, int E, int TPR>
qz_status run_backward(const NormArgs& a, int parts, cudaStream_t s) {
  constexpr int kBlock = kNormBlock<TPR>, G = kBlock / TPR;
  constexpr int kColumns = G > 1 ? 2 * kBlock * kPer * 4 : 0, kRing = E > 1 ? kNormSlots<DT, TPR> * kNormSlot<DT, TPR> : 0;
  constexpr int kSmem = kRing > kColumns ? kRing : kColumns;
  const void* k = a.parts ? reinterpret_cast<const void*>(&norm_backward_kernel<DT, E, TPR, true>)
                          : reinterpret_cast<const void*>(&norm_backward_kernel<DT, E, TPR, false>);
  if (kSmem && !set_dyn_smem(k, kSmem)) return QZ_ERR_CUDA;
  if (a.parts) norm_backward_kernel<DT, E, TPR, true><<<parts, kBlock, kSmem, s>>>(a);
  else norm_backward_kernel<DT, E, TPR, false><<<parts, kBlock, kSmem, s>>>(a);
  return launch_status();
}

template <int DT, int E>
qz_status run_held(const NormArgs& a, bool backward, int parts, cudaStream_t s) {
  const int tpr = threads_per_row(a.cols);
  if (!backward) {
    switch (tpr) {
      case 32: return run_forward<DT, E, 32>(a, s);
      case 64: return run_forward<DT, E, 64>(a, s);
      case 128: return run_forward<DT, E, 128>(a, s);
      case 192: return run_forward<DT, E, 192>(a, s);
      case 256: return run_forward<DT, E, 256>(a, s);
      case 384: return run_forward<DT, E, 384>(a, s);
      case 512: return run_forward<DT, E, 512>(a, s);
      case 640: return run_forward<DT, E, 640>(a, s);
      case 768: return run_forward<DT, E, 768>(a, s);
      default: return run_forward<DT, E, 1024>(a, s);
    }
  }
  // 192 and 384 threads make blocks of 384: fp32 rows gain (16320 x 2056: 88 -> 70 us; 8176 x 4104: 92 ->
  // 70), bf16 rows have more instructions a byte and want the warps (68 -> 86 us; 84 -> 92)
  if constexpr (DT == QZ_F32) {
    if (tpr == 192) return run_backward<DT, E, 192>(a, parts, s);
    if (tpr == 384) return run_backward<DT, E, 384>(a, parts, s);
  }
  switch (tpr) {
    case 32: return run_backward<DT, E, 32>(a, parts, s);
    case 64: return run_backward<DT, E, 64>(a, parts, s);
    case 128: return run_backward<DT, E, 128>(a, parts, s);
    case 192:
    case 256: return run_backward<DT, E, 256>(a, parts, s);
    case 384:
    case 512: return run_backward<DT, E, 512>(a, parts, s);
    case 640: return run_backward<DT, E, 640>(a, parts, s);
    case 768: return run_backward<DT, E, 768>(a, parts, s);
    default: return run_backward<DT, E, 1024>(a, parts, s);
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
    const int tpr = threads_per_row(cols);
    per = norm_block(tpr) / tpr;  // the same with 192 threads as with 256, with 384 as with 512
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
  norm_parts_kernel<<<static_cast<unsigned>((2 * cols + 31) / 32), 1024, 0, s>>>(a.parts, parts, cols, dweight, dbias);
  return launch_status();
}
