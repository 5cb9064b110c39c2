// qz_product.cu -- products with 4-bit weights (include/qz.h, "Products with quantized weights"):
// argument checks, the choice of kernel, the elementwise part of the gated block's backward pass,
// and the plain tile kernel that takes every shape, stride and alignment.
//
//   forward   out[t][r] = sum_c x[t][c] W[r][c]            (one weight, or gate and up together)
//   backward  out[t][c] = sum_r dy[t][r] W[r][c]           (summed over one or two weights)
#include <climits>
#include <cstdint>

#include "qz_device.cuh"
#include "qz_internal.h"
#include "qz_product.h"
#include "qz_product_plan.h"
#include "qz_weight.cuh"

namespace qz {
namespace {

// ---- the plain tile kernel ------------------------------------------------------------------
// A CTA computes 64 tokens x 64 outputs in fp32 FMAs, 32 summands at a time through shared
// memory, weights decoded as they are loaded.  It is bound by the FMA pipe and the decoding and
// serves the calls whose strides or alignment the other kernels do not take (gated 4096 tokens of
// 2 x 16384 x 4096 here: 45 ms, 24 TFLOP/s, against 0.66 ms on the tensor cores).
constexpr int kTileT = 64, kTileN = 64, kTileK = 32;

template <int FMT>
__device__ __forceinline__ float weight_at(const WeightView& w, int64_t cols, int log2_block, int64_t r, int64_t c) {
  const uint32_t b = __ldg(w.codes + (r * cols + c) / 2);
  return nibble_value<FMT>((c & 1) ? b >> 4 : b & 15u) *
         block_scale<FMT>(w.scales, r * (cols >> log2_block) + (c >> log2_block));
}

template <int FMT, int MODE>
__global__ void __launch_bounds__(256) product_tile_kernel(const ProductArgs p, int tiles_n) {
  constexpr int NW = MODE == kModeGated ? 2 : 1;    // weights read with each x
  constexpr int NA = MODE == kModeLinear ? 1 : 2;   // sums per output, one per weight (own tensor scales)
  __shared__ float xs[kTileK][kTileT + 1];
  __shared__ float ws[NW][kTileK][kTileN + 1];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / tiles_n) * kTileT;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x % tiles_n) * kTileN;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t nout = MODE == kModeBackward ? p.cols : p.rows, nsum = MODE == kModeBackward ? p.rows : p.cols;
  float acc[NA][4][4] = {};
#pragma unroll
  for (int pass = 0; pass < (MODE == kModeBackward ? 2 : 1); ++pass) {
    if (pass >= p.n_weights) break;
    const uint16_t* x = pass ? p.x1 : p.x0;
    for (int64_t k0 = 0; k0 < nsum; k0 += kTileK) {
      for (int i = threadIdx.x; i < kTileK * kTileT; i += 256) {
        const int k = i % kTileK, t = i / kTileK;
        xs[k][t] = (k0 + k < nsum && t0 + t < p.tokens) ? bf16_float(__ldg(x + (t0 + t) * p.ld_x + k0 + k)) : 0.0f;
      }
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        const WeightView& w = (v || pass) ? p.w1 : p.w0;
        for (int i = threadIdx.x; i < kTileK * kTileN; i += 256) {
          // columns of W run fastest over the threads
          const int k = MODE == kModeBackward ? i / kTileN : i % kTileK;
          const int n = MODE == kModeBackward ? i % kTileN : i / kTileK;
          float val = 0.0f;
          if (k0 + k < nsum && n0 + n < nout)
            val = MODE == kModeBackward ? weight_at<FMT>(w, p.cols, p.log2_block, k0 + k, n0 + n)
                                        : weight_at<FMT>(w, p.cols, p.log2_block, n0 + n, k0 + k);
          ws[v][k][n] = val;
        }
      }
      __syncthreads();
      const int kn = static_cast<int>(min(static_cast<int64_t>(kTileK), nsum - k0));
      for (int k = 0; k < kn; ++k) {
        float a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = xs[k][ty + 16 * i];
#pragma unroll
        for (int v = 0; v < NW; ++v)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float b = ws[v][k][tx + 16 * j];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[v + pass][i][j] = __fmaf_rn(a[i], b, acc[v + pass][i][j]);
          }
      }
      __syncthreads();
    }
  }
  const float f0 = sum_factor<FMT>(p.w0.tscale);
  const float f1 = NA == 2 && p.n_weights == 2 ? sum_factor<FMT>(p.w1.tscale) : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (t >= p.tokens || n >= nout) continue;
      float a = acc[0][i][j] * f0;
      if (MODE == kModeBackward && p.n_weights == 2) a = __fmaf_rn(acc[NA - 1][i][j], f1, a);
      if constexpr (MODE == kModeGated) {
        const float u = acc[NA - 1][i][j] * f1;
        const float v = p.act == QZ_ACT_SILU ? act_value<QZ_ACT_SILU>(a) : act_value<QZ_ACT_GELU_TANH>(a);
        static_cast<uint16_t*>(p.y)[t * p.ld_y + n] = bf16_bits(v * u);
        if (p.g_out) {
          p.g_out[t * p.ld_gu + n] = bf16_bits(a);
          p.u_out[t * p.ld_gu + n] = bf16_bits(u);
        }
      } else if (p.out_f32) {
        static_cast<float*>(p.y)[t * p.ld_y + n] = a;
      } else {
        static_cast<uint16_t*>(p.y)[t * p.ld_y + n] = bf16_bits(a);
      }
    }
}

template <int FMT>
qz_status run_tile(const ProductArgs& p, cudaStream_t s) {
  const int64_t nout = p.mode == kModeBackward ? p.cols : p.rows;
  const int64_t tn = (nout + kTileN - 1) / kTileN, tt = (p.tokens + kTileT - 1) / kTileT;
  if (tn * tt >= (int64_t{1} << 31)) return QZ_ERR_UNSUPPORTED;
  const int grid = static_cast<int>(tn * tt), n = static_cast<int>(tn);
  if (p.mode == kModeLinear) product_tile_kernel<FMT, kModeLinear><<<grid, 256, 0, s>>>(p, n);
  else if (p.mode == kModeGated) product_tile_kernel<FMT, kModeGated><<<grid, 256, 0, s>>>(p, n);
  else product_tile_kernel<FMT, kModeBackward><<<grid, 256, 0, s>>>(p, n);
  return launch_status();
}

qz_status launch_few(const ProductArgs& p, cudaStream_t s) {
  const bool whole = few_whole(p);
  if (p.format == QZ_MXFP4) return whole ? launch_product_few_mxfp4(p, s) : launch_product_few_mxfp4_ragged(p, s);
  if (p.format == QZ_NVFP4) return whole ? launch_product_few_nvfp4(p, s) : launch_product_few_nvfp4_ragged(p, s);
  return whole ? launch_product_few_int4(p, s) : launch_product_few_int4_ragged(p, s);
}

// `count` of a forward product's tokens from `first` on
ProductArgs some_tokens(ProductArgs p, int64_t first, int64_t count) {
  p.tokens = count;
  p.x0 += first * p.ld_x;
  p.y = static_cast<char*>(p.y) + first * p.ld_y * (p.out_f32 ? 4 : 2);
  if (p.g_out) {
    p.g_out += first * p.ld_gu;
    p.u_out += first * p.ld_gu;
  }
  return p;
}

// The streaming kernel or the tiles, by what they are estimated to take.  Where the activations' staging costs
// little against the start of a tile (3 tokens of 4096 columns 5.6 us, on the tiles 9.0 and more) nothing is estimated.
bool few_pays(const ProductArgs& p) {
  return p.tokens * ((p.cols + 4095) / 4096) <= 4 || few_us(p) <= tiles_us(p);
}

qz_status launch_product(const ProductArgs& p, cudaStream_t s) {
  if (product_few_applicable(p)) {
    if (few_pays(p)) return launch_few(p, s);
  } else if (p.format == QZ_INT4 && p.mode != kModeBackward && p.tokens > 1 && p.tokens <= 16) {
    // INT4, at most 16 tokens that do not fit shared memory together: two halves of 8 read the weights
    // twice and may still beat the tiles (16 tokens, groups of 128, 32768 x 8192: 93 us against 166;
    // 512 x 8192: 26 against 18)
    const int64_t half = (p.tokens + 1) / 2;
    const ProductArgs a = some_tokens(p, 0, half), b = some_tokens(p, half, p.tokens - half);
    if (product_few_applicable(a) && 2 * few_us(a) <= tiles_us(p)) {
      const qz_status st = launch_few(a, s);
      return st == QZ_OK ? launch_few(b, s) : st;
    }
  }
  if (product_tc_applicable(p)) {
    if (p.format == QZ_MXFP4) return launch_product_tc_mxfp4(p, s);
    if (p.format == QZ_NVFP4) return launch_product_tc_nvfp4(p, s);
    return launch_product_tc_int4(p, s);
  }
  if (p.format == QZ_MXFP4) return run_tile<QZ_MXFP4>(p, s);
  if (p.format == QZ_NVFP4) return run_tile<QZ_NVFP4>(p, s);
  return run_tile<QZ_INT4>(p, s);
}

// ---- dg = dh u act'(g), du = dh act(g) --------------------------------------------------------
// Elementwise: three reads and two writes of 2 bytes per element, bound by HBM.  Eight elements
// a thread when rows and leading dimensions allow 16-byte access, one otherwise.  4096 x 16384:
// 99 us, 6.8 TB/s.
struct GateGradArgs {
  const uint16_t *dh, *g, *u;
  uint16_t *dg, *du;
  int64_t tokens, rows, ld_dh, ld_gu, ld_dgu;
};

template <int ACT, bool VEC>
__global__ void __launch_bounds__(256) gate_grad_kernel(const GateGradArgs a) {
  constexpr int V = VEC ? 8 : 1;
  const int64_t per = (a.rows + V - 1) / V, n = a.tokens * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t t = i / per, r = (i - t * per) * V;
    const uint16_t* ph = a.dh + t * a.ld_dh + r;
    const int64_t gu = t * a.ld_gu + r, dd = t * a.ld_dgu + r;
    if constexpr (VEC) {
      const uint4 vh = ld16B(ph), vg = ld16B(a.g + gu), vu = ld16B(a.u + gu);
      const uint32_t h4[4] = {vh.x, vh.y, vh.z, vh.w}, g4[4] = {vg.x, vg.y, vg.z, vg.w}, u4[4] = {vu.x, vu.y, vu.z, vu.w};
      uint32_t og[4], ou[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float rg[2], ru[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float dh = __uint_as_float(e ? h4[q] & 0xffff0000u : h4[q] << 16);
          const float g = __uint_as_float(e ? g4[q] & 0xffff0000u : g4[q] << 16);
          const float u = __uint_as_float(e ? u4[q] & 0xffff0000u : u4[q] << 16);
          float v;
          const float d = act_derivative<ACT>(g, v);
          rg[e] = dh * u * d;
          ru[e] = dh * v;
        }
        og[q] = bf16x2_bits(rg[0], rg[1]);
        ou[q] = bf16x2_bits(ru[0], ru[1]);
      }
      *reinterpret_cast<uint4*>(a.dg + dd) = make_uint4(og[0], og[1], og[2], og[3]);
      *reinterpret_cast<uint4*>(a.du + dd) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
    } else {
      const float dh = bf16_float(__ldg(ph)), g = bf16_float(__ldg(a.g + gu)), u = bf16_float(__ldg(a.u + gu));
      float v;
      const float d = act_derivative<ACT>(g, v);
      a.dg[dd] = bf16_bits(dh * u * d);
      a.du[dd] = bf16_bits(dh * v);
    }
  }
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

qz_status launch_gate_grad(const GateGradArgs& a, int act, cudaStream_t s) {
  const bool vec = a.rows % 8 == 0 && a.ld_dh % 8 == 0 && a.ld_gu % 8 == 0 && a.ld_dgu % 8 == 0 && aligned(a.dh, 16) &&
                   aligned(a.g, 16) && aligned(a.u, 16) && aligned(a.dg, 16) && aligned(a.du, 16);
  const int64_t n = a.tokens * ((a.rows + (vec ? 7 : 0)) / (vec ? 8 : 1));
  const void* k;
  if (act == QZ_ACT_SILU)
    k = vec ? reinterpret_cast<const void*>(&gate_grad_kernel<QZ_ACT_SILU, true>)
            : reinterpret_cast<const void*>(&gate_grad_kernel<QZ_ACT_SILU, false>);
  else
    k = vec ? reinterpret_cast<const void*>(&gate_grad_kernel<QZ_ACT_GELU_TANH, true>)
            : reinterpret_cast<const void*>(&gate_grad_kernel<QZ_ACT_GELU_TANH, false>);
  const int grid = grid_for(k, (n + 255) / 256, s);
  void* args[] = {const_cast<GateGradArgs*>(&a)};
  return cudaLaunchKernel(k, dim3(grid), dim3(256), args, 0, s) == cudaSuccess ? launch_status() : QZ_ERR_CUDA;
}

}  // namespace

bool product_few_applicable(const ProductArgs& p) {
  // whole chunks of 32 columns (16 bytes of codes); an INT4 group of 16 would change inside one's sum
  if (p.mode == kModeBackward || p.tokens > few_tokens(p.format) || p.cols == 0 || p.cols % 32 != 0) return false;
  if (p.format == QZ_INT4 && p.log2_block < 5) return false;
  if (p.rows >= (int64_t{1} << 30) || p.cols >= (int64_t{1} << 30) || few_depth(p) == 0) return false;
  // (NVFP4: the scales of 32 columns are loaded together)
  const size_t n = p.format == QZ_NVFP4 ? 2 : 1;
  return p.ld_x % 8 == 0 && aligned(p.x0, 16) && aligned(p.w0.codes, 16) && aligned(p.w0.scales, n) &&
         (p.n_weights == 1 || (aligned(p.w1.codes, 16) && aligned(p.w1.scales, n)));
}

bool few_whole(const ProductArgs& p) {
  const size_t n = p.format == QZ_MXFP4 || (p.format == QZ_INT4 && p.log2_block == 7) ? 8 : 16;
  return p.cols % 256 == 0 && aligned(p.w0.scales, n) && (p.n_weights == 1 || aligned(p.w1.scales, n));
}

bool product_tc_applicable(const ProductArgs& p) {
  const auto a16 = [](const void* q) { return aligned(q, 16); };
  const int64_t big = int64_t{1} << 30;
  return p.cols % 32 == 0 && p.cols > 0 && p.rows > 0 && p.cols < big && p.rows < big && p.tokens < big && p.ld_x % 8 == 0 &&
         a16(p.x0) && a16(p.w0.codes) && (p.n_weights == 1 || a16(p.w1.codes)) &&
         (p.mode != kModeBackward || p.n_weights == 1 || a16(p.x1));
}

namespace {

// ---- checks -------------------------------------------------------------------------------------
constexpr int64_t kMaxDim = int64_t{1} << 31;

qz_status check_weight(const qz_weight* w) {
  if (!w) return QZ_ERR_NULL;
  if (w->format != QZ_MXFP4 && w->format != QZ_NVFP4 && w->format != QZ_INT4) return QZ_ERR_ENUM;
  const int bs = w->block_size;
  if (w->format == QZ_INT4 ? (bs != 16 && bs != 32 && bs != 64 && bs != 128) : bs != (w->format == QZ_MXFP4 ? 32 : 16))
    return QZ_ERR_UNSUPPORTED;
  if (w->rows < 0 || w->cols < 0 || w->cols % bs != 0) return QZ_ERR_SHAPE;
  if (w->rows >= kMaxDim || w->cols >= kMaxDim) return QZ_ERR_UNSUPPORTED;
  return QZ_OK;
}
qz_status check_weight_buffers(const qz_weight* w) {
  if (w->rows * w->cols == 0) return QZ_OK;
  if (!w->codes || !w->scales) return QZ_ERR_NULL;
  if (w->format == QZ_INT4 && !aligned(w->scales, 4)) return QZ_ERR_ALIGN;
  if (w->format == QZ_NVFP4 && w->tensor_scale_dev && !aligned(w->tensor_scale_dev, 4)) return QZ_ERR_ALIGN;
  return QZ_OK;
}
// a [tokens, width] matrix with leading dimension ld
qz_status check_matrix(int64_t tokens, int64_t width, int64_t ld) {
  if (tokens < 0 || ld < width) return QZ_ERR_SHAPE;
  if (tokens >= kMaxDim) return QZ_ERR_UNSUPPORTED;
  if (tokens > 0 && ld > (INT64_MAX / 8) / tokens) return QZ_ERR_SHAPE;
  return QZ_OK;
}
// The leading dimension of one row means nothing: it may be odd, or beyond the strides that TMA takes (2^40 bytes).
int64_t pitch_of(int64_t tokens, int64_t width, int64_t ld) { return tokens == 1 ? (width + 7) / 8 * 8 : ld; }
qz_status check_pointer(const void* p, size_t a) {
  if (!p) return QZ_ERR_NULL;
  return aligned(p, a) ? QZ_OK : QZ_ERR_ALIGN;
}
int log2_of(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}
ProductArgs args_of(const qz_weight& w, int mode, int64_t tokens) {
  ProductArgs p{};
  p.mode = mode;
  p.format = w.format;
  p.log2_block = log2_of(w.block_size);
  p.n_weights = 1;
  p.w0 = view_of(w);
  p.rows = w.rows;
  p.cols = w.cols;
  p.tokens = tokens;
  return p;
}
bool same_kind(const qz_weight& a, const qz_weight& b) {
  return a.format == b.format && a.block_size == b.block_size && a.rows == b.rows && a.cols == b.cols;
}

#define QZ_TRY(expr)                        \
  do {                                      \
    const qz_status st_ = (expr);           \
    if (st_ != QZ_OK) return st_;           \
  } while (0)

}  // namespace
}  // namespace qz

using namespace qz;

extern "C" qz_status qz_linear(const qz_weight* w, const void* x, int64_t ld_x, int64_t tokens, void* y,
                               int64_t ld_y, int32_t out_dtype, qz_stream_t stream) {
  QZ_TRY(check_weight(w));
  if (out_dtype != QZ_BF16 && out_dtype != QZ_F32) return QZ_ERR_ENUM;
  QZ_TRY(check_matrix(tokens, w->cols, ld_x));
  QZ_TRY(check_matrix(tokens, w->rows, ld_y));
  if (tokens == 0 || w->rows == 0) return QZ_OK;
  QZ_TRY(check_weight_buffers(w));
  if (w->cols) QZ_TRY(check_pointer(x, 2));
  QZ_TRY(check_pointer(y, out_dtype == QZ_BF16 ? 2 : 4));
  ProductArgs p = args_of(*w, kModeLinear, tokens);
  p.x0 = static_cast<const uint16_t*>(x);
  p.ld_x = pitch_of(tokens, w->cols, ld_x);
  p.y = y;
  p.ld_y = ld_y;
  p.out_f32 = out_dtype == QZ_F32;
  return launch_product(p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" qz_status qz_linear_backward(const qz_weight* w, const void* dy, int64_t ld_dy, int64_t tokens,
                                        void* dx, int64_t ld_dx, int32_t out_dtype, qz_stream_t stream) {
  QZ_TRY(check_weight(w));
  if (out_dtype != QZ_BF16 && out_dtype != QZ_F32) return QZ_ERR_ENUM;
  QZ_TRY(check_matrix(tokens, w->rows, ld_dy));
  QZ_TRY(check_matrix(tokens, w->cols, ld_dx));
  if (tokens == 0 || w->cols == 0) return QZ_OK;
  QZ_TRY(check_weight_buffers(w));
  if (w->rows) QZ_TRY(check_pointer(dy, 2));
  QZ_TRY(check_pointer(dx, out_dtype == QZ_BF16 ? 2 : 4));
  ProductArgs p = args_of(*w, kModeBackward, tokens);
  p.x0 = static_cast<const uint16_t*>(dy);
  p.ld_x = pitch_of(tokens, w->rows, ld_dy);
  p.y = dx;
  p.ld_y = ld_dx;
  p.out_f32 = out_dtype == QZ_F32;
  return launch_product(p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" qz_status qz_gated_ffn(const qz_weight* gate, const qz_weight* up, int32_t act, const void* x,
                                  int64_t ld_x, int64_t tokens, void* h, int64_t ld_h, void* g_out,
                                  void* u_out, int64_t ld_gu, qz_stream_t stream) {
  QZ_TRY(check_weight(gate));
  QZ_TRY(check_weight(up));
  if (act != QZ_ACT_SILU && act != QZ_ACT_GELU_TANH) return QZ_ERR_ENUM;
  if (!same_kind(*gate, *up)) return QZ_ERR_SHAPE;
  QZ_TRY(check_matrix(tokens, gate->cols, ld_x));
  QZ_TRY(check_matrix(tokens, gate->rows, ld_h));
  if (g_out || u_out) QZ_TRY(check_matrix(tokens, gate->rows, ld_gu));
  if (tokens == 0 || gate->rows == 0) return QZ_OK;
  QZ_TRY(check_weight_buffers(gate));
  QZ_TRY(check_weight_buffers(up));
  if (gate->cols) QZ_TRY(check_pointer(x, 2));
  QZ_TRY(check_pointer(h, 2));
  if (g_out || u_out) {
    QZ_TRY(check_pointer(g_out, 2));
    QZ_TRY(check_pointer(u_out, 2));
  }
  ProductArgs p = args_of(*gate, kModeGated, tokens);
  p.n_weights = 2;
  p.w1 = view_of(*up);
  p.act = act;
  p.x0 = static_cast<const uint16_t*>(x);
  p.ld_x = pitch_of(tokens, gate->cols, ld_x);
  p.y = h;
  p.ld_y = ld_h;
  p.g_out = static_cast<uint16_t*>(g_out);
  p.u_out = static_cast<uint16_t*>(u_out);
  p.ld_gu = ld_gu;
  return launch_product(p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" qz_status qz_gated_ffn_backward(const qz_weight* gate, const qz_weight* up, int32_t act,
                                           const void* dh, int64_t ld_dh, const void* g, const void* u,
                                           int64_t ld_gu, int64_t tokens, void* dg, void* du, int64_t ld_dgu,
                                           void* dx, int64_t ld_dx, qz_stream_t stream) {
  QZ_TRY(check_weight(gate));
  QZ_TRY(check_weight(up));
  if (act != QZ_ACT_SILU && act != QZ_ACT_GELU_TANH) return QZ_ERR_ENUM;
  if (!same_kind(*gate, *up)) return QZ_ERR_SHAPE;
  QZ_TRY(check_matrix(tokens, gate->rows, ld_dh));
  QZ_TRY(check_matrix(tokens, gate->rows, ld_gu));
  QZ_TRY(check_matrix(tokens, gate->rows, ld_dgu));
  QZ_TRY(check_matrix(tokens, gate->cols, ld_dx));
  if (tokens == 0) return QZ_OK;
  QZ_TRY(check_weight_buffers(gate));
  QZ_TRY(check_weight_buffers(up));
  if (gate->rows)
    for (const void* q : {dh, g, u, static_cast<const void*>(dg), static_cast<const void*>(du)}) QZ_TRY(check_pointer(q, 2));
  if (gate->cols) QZ_TRY(check_pointer(dx, 2));
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (gate->rows) {
    GateGradArgs a{static_cast<const uint16_t*>(dh), static_cast<const uint16_t*>(g), static_cast<const uint16_t*>(u),
                   static_cast<uint16_t*>(dg), static_cast<uint16_t*>(du), tokens, gate->rows, ld_dh, ld_gu, ld_dgu};
    QZ_TRY(launch_gate_grad(a, act, s));
  }
  if (gate->cols == 0) return QZ_OK;
  ProductArgs p = args_of(*gate, kModeBackward, tokens);
  p.n_weights = 2;
  p.w1 = view_of(*up);
  p.x0 = static_cast<const uint16_t*>(dg);
  p.x1 = static_cast<const uint16_t*>(du);
  p.ld_x = pitch_of(tokens, gate->rows, ld_dgu);
  p.y = dx;
  p.ld_y = ld_dx;
  return launch_product(p, s);
}
