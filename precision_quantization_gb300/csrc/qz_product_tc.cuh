// qz_product_tc.cuh -- products with 4-bit weights on the tcgen05 tensor cores (more than a few
// tokens), included once per weight format.
//
//   forward   D[r][t] = sum_c W[r][c] x[t][c]          backward  D[c][t] = sum_r W[r][c] dy[t][r]
//
// The weights are the MMA's A operand (M: 128 outputs a CTA, one tensor-memory lane each), the
// activations its B operand (N: up to 256 tokens, one fp32 tensor-memory column each).  E2M1
// times its block scale has at most 6 significant bits and so is exact in bf16; an INT4 weight
// q s is held as the sum of two bf16 values (16 bits of it) and takes two MMAs.  So kind::f16
// with fp32 accumulation gives the sums of include/qz.h without a rounding of the weights.
//
// Roles of a CTA of 16 warps (every wait is bounded):
//   warp 0       streams the tokens' 64-wide steps into a shared-memory ring by TMA
//   warp 2       streams the 4-bit codes into a ring of their own by TMA
//   warps 4-11   decode: 256 threads take 32 weights of every step each (16 bytes of codes),
//                turn them into bf16 and store them in the layout the MMA reads
//   warp 1       issues the MMAs, four 16-wide ones a step (one thread)
//   warps 12-15  read finished accumulators from tensor memory, apply the activation and store
// Two forms.  PAIR: two CTAs on neighbouring SMs share one 256 x 256 tile (cta_group::2: each
// decodes its own 128 outputs and loads half of the tokens, so the shared-memory traffic per MMA
// halves), persistent over the tiles, the epilogue of a tile beside the next tile's MMAs (two
// accumulators of 256 columns).  Alone: a CTA has a tile of 128 outputs and one slice of the sum;
// the CTAs of a cluster hold the slices of one tile, exchange their partial sums through
// distributed shared memory and add them in slice order, so few tokens still fill the GPU and
// equal inputs give equal results.
#pragma once

#include <cuda.h>  // CUtensorMap and its enumerators (types only; the encoder is looked up)
#include <cudaTypedefs.h>

#include <algorithm>

#include "qz_device.cuh"
#include "qz_internal.h"
#include "qz_pipe.cuh"
#include "qz_product.h"
#include "qz_weight.cuh"

namespace qz {
namespace {

constexpr int kBM = 128;            // outputs per CTA (MMA rows, tensor-memory lanes)
constexpr int kBK = 64;             // summands per step: 128 bytes of bf16, one swizzle row
constexpr int kThreadsTc = 512;
constexpr int kDecWarp0 = 4, kDecWarps = 8, kEpiWarp0 = 12, kEpiWarps = 4;
constexpr uint32_t kABytes = kBM * kBK * 2;        // 16 KiB of decoded weights
constexpr uint32_t kCodeBytes = kBM * kBK / 2;     // 4 KiB of codes per step
constexpr uint32_t kTmemCols = 512;                // two accumulators of 256 columns
constexpr uint64_t kTcWaitNs = 1000000000ull;      // 1 s: far beyond any step's latency
constexpr int kMaxBStages = 8, kCodeSlots = 10;    // code ring: ten steps
constexpr int kMaxAStages = 4;

template <int FMT>
struct TcFormat {
  static constexpr int kTerms = FMT == QZ_INT4 ? 2 : 1;  // bf16 terms per weight
  static constexpr int kAStages = FMT == QZ_INT4 ? 3 : 4;
};
template <int FMT>
constexpr uint32_t kARing = TcFormat<FMT>::kAStages * TcFormat<FMT>::kTerms * kABytes;
constexpr uint32_t kSmemMax = 227 * 1024 - 2048;   // dynamic; the barriers are static
template <int FMT>
constexpr uint32_t kBRoom = kSmemMax - 1024 - kARing<FMT> - kCodeSlots * kCodeBytes;

struct TcArgs {
  CUtensorMap map_x0, map_x1;  // bf16 [tokens][sum], box 64 x (tokens of a CTA's load)
  CUtensorMap map_w0, map_w1;  // codes [rows][cols / 2] bytes
  const void *scales0, *scales1;
  const float *tscale0, *tscale1;
  ProductArgs p;
  int nout, nsum;         // outputs and summands (per weight)
  int blocks_row;         // scales per weight row
  int steps_w, steps;     // steps per weight, in all (backward: both weights one after the other)
  int n;                  // tokens per tile (a multiple of 32)
  int b_stages;
  int tiles_n, tiles;
  int slices, slice_steps;  // Alone: slices of the sum (the cluster), steps per slice
};

// ---- PTX ------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// arrive on a barrier of this CTA or (shared::cluster address) of another in the cluster
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
template <int CG>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// completion of every MMA issued so far arrives on `bar`, in both CTAs of a pair
template <int CG>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
}
// 8 consecutive fp32 columns of this thread's tensor-memory lane
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void sts16(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle (byte offsets in 16-byte units, version 1).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: fp32 accumulator, bf16 operands, B K-major, A K-major or MN-major.
__device__ __forceinline__ uint32_t idesc_of(int m, int n, bool a_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!try_wait_cluster(bar, parity)) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kTcWaitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

// After a wait has given up: let the copies already issued land before their memory is released.
// The last one went to the stage before `s`; `ph` is the parity of stage s's next use.
__device__ __forceinline__ void let_land(uint64_t* full, int s, uint32_t ph, int stages, uint32_t issued) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t k = 0; k < min(issued, static_cast<uint32_t>(stages)); ++k) {
    if (--s < 0) {
      s = stages - 1;
      ph ^= 1u;
    }
    while (!try_wait_cluster(smem_addr(&full[s]), ph) && globaltimer_ns() - t0 < kTcWaitNs) {
    }
  }
}

// ---- decoding -------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Byte q of a word as two 4-bit fields at bits 0 and 16 (even and odd nibble); t0 = word &
// 0x0F0F0F0F, t1 = (word >> 4) & 0x0F0F0F0F.  Selectors 8 give the sign of byte 0, which is 0.
template <int Q>
__device__ __forceinline__ uint32_t nibble_pair(uint32_t t0, uint32_t t1) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(t0), "r"(t1), "n"(0x8080 | Q | ((4 + Q) << 8)));
  return d;
}
// The E2M1 pair as bf16 times 2^-126: the sign goes to bit 15, the exponent and mantissa bits to
// bits 6-8, and bf16's own exponent (biased 127 against 1) and subnormals do the rest.
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t d) { return (d * 0x1040u) & 0x81C081C0u; }

// The scale(s) of one thread's 32 weights.  raw: an E8M0 byte, two E4M3 bytes, or fp32 (two for
// groups of 16).
template <int FMT>
struct Scales {
  uint32_t a, b;
};
template <int FMT>
__device__ __forceinline__ Scales<FMT> load_scales(const void* base, int64_t row_blocks, int col, int log2_block, bool in) {
  Scales<FMT> s{0u, 0u};  // outside the weight: finite (its codes are 0)
  if (!in) return s;
  const int64_t i = row_blocks + (col >> log2_block);
  if constexpr (FMT == QZ_MXFP4) {
    s.a = __ldg(static_cast<const uint8_t*>(base) + i);
  } else if constexpr (FMT == QZ_NVFP4) {
    s.a = __ldg(static_cast<const uint8_t*>(base) + i);
    s.b = __ldg(static_cast<const uint8_t*>(base) + i + 1);
  } else {
    s.a = __ldg(static_cast<const uint32_t*>(base) + i);
    s.b = log2_block == 4 ? __ldg(static_cast<const uint32_t*>(base) + i + 1) : s.a;
  }
  return s;
}

// 32 weights (16 bytes of codes) to bf16, stored as four 16-byte chunks of line `line`:
// chunk 4 half + j at its swizzled place.
template <int FMT>
__device__ __forceinline__ void decode32(const uint4 codes, const Scales<FMT> s, uint32_t dst, uint32_t line_addr, int line, int half) {
  const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t f0, f1;  // bf16 pairs: the factor of the first and the second 16 weights
  bool big = false;
  uint32_t extra = 0x3F803F80u;
  if constexpr (FMT == QZ_MXFP4) {
    // 2^(E - 127) 2^126 as bf16 has exponent field E + 126; fields above 254 take a second factor
    const uint32_t e = min(s.a + 126u, 254u);
    f0 = s.a == 255u ? 0x7FC07FC0u : (e << 7) * 0x00010001u;
    f1 = f0;
    big = s.a > 128u && s.a != 255u;
    if (big) extra = ((s.a - 128u + 127u) << 7) * 0x00010001u;
  } else if constexpr (FMT == QZ_NVFP4) {
    // an E4M3 byte at bits 4-10 is its value times 2^-120 as bf16; 2^127 and 2^111 bring it to
    // 2^118 times its value (below 2^127), so a weight comes out as 2^-8 of its own
    uint32_t c = (s.a << 4) | (s.b << 20);
    c = mul_bf16x2(mul_bf16x2(c, 0x7F007F00u), 0x77007700u);
    f0 = (c & 0xffffu) * 0x00010001u;
    f1 = (c >> 16) * 0x00010001u;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t t0 = cw[j] & 0x0F0F0F0Fu, t1 = (cw[j] >> 4) & 0x0F0F0F0Fu;
    uint32_t d[4] = {nibble_pair<0>(t0, t1), nibble_pair<1>(t0, t1), nibble_pair<2>(t0, t1), nibble_pair<3>(t0, t1)};
    const uint32_t at = dst + line_addr + static_cast<uint32_t>(((4 * half + j) ^ (line & 7)) << 4);
    if constexpr (FMT == QZ_INT4) {
      const float sc = __uint_as_float(j < 2 ? s.a : s.b);
      uint32_t lo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // bf16 128 + (n ^ 8), less 136: the two's complement value, exactly
        uint32_t v;
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"((d[q] ^ 0x00080008u) | 0x43004300u), "r"(0xC308C308u));
        const float w0 = __uint_as_float(v << 16) * sc, w1 = __uint_as_float(v & 0xffff0000u) * sc;
        d[q] = bf16x2_bits(w0, w1);  // the first term; what it leaves of w is exact in fp32
        lo[q] = bf16x2_bits(w0 - __uint_as_float(d[q] << 16), w1 - __uint_as_float(d[q] & 0xffff0000u));
      }
      sts16(at, d);
      sts16(at + kABytes, lo);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) d[q] = mul_bf16x2(e2m1_pair(d[q]), j < 2 ? f0 : f1);
      if (FMT == QZ_MXFP4 && big) {
#pragma unroll
        for (int q = 0; q < 4; ++q) d[q] = mul_bf16x2(d[q], extra);
      }
      sts16(at, d);
    }
  }
}

// ---- epilogue ---------------------------------------------------------------------------------
__device__ __forceinline__ void store_rows2(uint16_t* y, int64_t ld, int64_t t, int row, int rows, bool vec, float a, float b) {
  uint16_t* q = y + t * ld + row;
  if (vec && row + 1 < rows) {
    *reinterpret_cast<uint32_t*>(q) = bf16x2_bits(a, b);
  } else {
    if (row < rows) q[0] = bf16_bits(a);
    if (row + 1 < rows) q[1] = bf16_bits(b);
  }
}
// Neighbouring lanes hold neighbouring outputs of the tokens t and t + 1 (a and b): after the
// exchange the even lane stores both outputs of t, the odd lane both of t + 1.
__device__ __forceinline__ void store_pair(uint16_t* y, int64_t ld, int64_t t, int64_t tokens, int row, int rows, bool vec,
                                           float a, float b, int lane) {
  const bool odd = lane & 1;
  const float got = __shfl_xor_sync(kFull, odd ? a : b, 1);
  const int64_t tt = t + (odd ? 1 : 0);
  if (tt < tokens) store_rows2(y, ld, tt, row & ~1, rows, vec, odd ? got : a, odd ? b : got);
}

struct StoreFlags {
  bool y_vec, gu_vec;
};
// 8 finished sums of this thread's lane, tokens t0 .. t0 + 7.  m0: first output of the CTA's tile.
template <int FMT, int MODE>
__device__ __forceinline__ void store8(const TcArgs& a, StoreFlags f, const float (&v)[8], float f0, float f1, int m0, int quarter,
                                       int lane, int64_t t0) {
  const ProductArgs& p = a.p;
  const int64_t tokens = p.tokens;
  if (t0 >= tokens) return;
  if constexpr (MODE == kModeGated) {
    // lanes 0-15 hold gate sums, 16-31 the same outputs' up sums: each half takes one token of
    // a pair from the other
    const bool upper = lane >= 16;
    const int row = m0 + 16 * quarter + (lane & 15);
    uint16_t* y = static_cast<uint16_t*>(p.y);
    float g[4], u[4], h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float got = __shfl_xor_sync(kFull, upper ? v[2 * i] : v[2 * i + 1], 16);
      g[i] = (upper ? got : v[2 * i]) * f0;
      u[i] = (upper ? v[2 * i + 1] : got) * f1;
      h[i] = (p.act == QZ_ACT_SILU ? act_value<QZ_ACT_SILU>(g[i]) : act_value<QZ_ACT_GELU_TANH>(g[i])) * u[i];
    }
    // this lane now has tokens t0 + 2 i (+ 1 in the upper half); pairs of them two tokens apart
    const bool odd = lane & 1;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const int64_t t = t0 + 2 * i + (upper ? 1 : 0) + (odd ? 2 : 0);
      const auto put = [&](uint16_t* dst, int64_t ld, bool vec, const float (&w)[4]) {
        const float got = __shfl_xor_sync(kFull, odd ? w[i] : w[i + 1], 1);
        if (t < tokens) store_rows2(dst, ld, t, row & ~1, a.nout, vec, odd ? got : w[i], odd ? w[i + 1] : got);
      };
      put(y, p.ld_y, f.y_vec, h);
      if (p.g_out) {
        put(p.g_out, p.ld_gu, f.gu_vec, g);
        put(p.u_out, p.ld_gu, f.gu_vec, u);
      }
    }
  } else {
    const int row = m0 + 32 * quarter + lane;
    if (p.out_f32) {
      float* y = static_cast<float*>(p.y) + t0 * p.ld_y + row;
      if (row < a.nout) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (t0 + i < tokens) y[i * p.ld_y] = v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        store_pair(static_cast<uint16_t*>(p.y), p.ld_y, t0 + i, tokens, row, a.nout, f.y_vec, v[i], v[i + 1], lane);
    }
  }
}

// ---- the kernel ---------------------------------------------------------------------------------
// PAIR = true: CG = 2, persistent; false: CG = 1, one tile per cluster of a.slices CTAs.
template <int FMT, int MODE, bool PAIR>
__global__ void __launch_bounds__(kThreadsTc, 1) product_tc_kernel(const __grid_constant__ TcArgs a) {
  constexpr int CG = PAIR ? 2 : 1;
  constexpr int kTerms = TcFormat<FMT>::kTerms, kAStages = TcFormat<FMT>::kAStages;
  constexpr int kStepsPerCode = MODE == kModeBackward ? 1 : 2;      // steps of one code box
  constexpr int kSlots = kCodeSlots / kStepsPerCode;
  constexpr int kOut = MODE == kModeGated ? kBM / 2 : kBM;          // outputs per CTA
  extern __shared__ uint8_t tc_raw[];
  __shared__ __align__(8) uint64_t b_full[kMaxBStages], b_empty[kMaxBStages], a_full[kMaxAStages], a_empty[kMaxAStages];
  __shared__ __align__(8) uint64_t c_full[kCodeSlots], c_empty[kCodeSlots], d_full[2], d_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = !PAIR || rank == 0;
  const uint32_t base = (smem_addr(tc_raw) + 1023u) & ~1023u;
  const uint32_t a_base = base, c_base = base + kARing<FMT>, b_base = c_base + kCodeSlots * kCodeBytes;
  const int b_rows = a.n / CG;                       // tokens that this CTA loads
  const uint32_t b_bytes = static_cast<uint32_t>(b_rows) * kBK * 2;
  const int b_stages = a.b_stages;

  if (tid == 0) {
    for (int s = 0; s < kMaxBStages; ++s) {
      mbar_init(smem_addr(&b_full[s]), 1);
      mbar_init(smem_addr(&b_empty[s]), 1);
    }
    for (int s = 0; s < kMaxAStages; ++s) {
      mbar_init(smem_addr(&a_full[s]), kDecWarps * CG);
      mbar_init(smem_addr(&a_empty[s]), 1);
    }
    for (int s = 0; s < kCodeSlots; ++s) {
      mbar_init(smem_addr(&c_full[s]), 1);
      mbar_init(smem_addr(&c_empty[s]), kDecWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&d_full[s]), 1);
      mbar_init(smem_addr(&d_empty[s]), kEpiWarps * CG);
    }
    mbar_init(smem_addr(&drain), 1);
    mbar_init_fence();
    s_abort = 0;
  }
  if (warp == 3) {
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)), "r"(kTmemCols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)), "r"(kTmemCols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // every CTA's barriers exist before another signals them
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  // this CTA's tiles: PAIR: cluster id, + clusters, ...; else one
  const int first = PAIR ? static_cast<int>(blockIdx.x) / 2 : static_cast<int>(blockIdx.x) / a.slices;
  const int tile_end = PAIR ? a.tiles : first + 1;
  const int tile_step = PAIR ? static_cast<int>(gridDim.x) / 2 : 1;
  const int st_begin = PAIR ? 0 : static_cast<int>(rank) * a.slice_steps;
  const int st_end = PAIR ? a.steps : min(a.steps, st_begin + a.slice_steps);
  const auto tile_m0 = [&](int t) { return (t / a.tiles_n) * (kOut * CG) + (PAIR ? static_cast<int>(rank) * kOut : 0); };
  const auto tile_n0 = [&](int t) { return (t % a.tiles_n) * a.n; };

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, issued = 0;
      bool ok = true;
      for (int t = first; t < tile_end && ok; t += tile_step) {
        const int n0 = tile_n0(t) + (PAIR ? static_cast<int>(rank) * b_rows : 0);
        for (int st = st_begin; st < st_end; ++st) {
          if (!(ok = tc_wait(smem_addr(&b_empty[s]), ph ^ 1u, &s_abort))) break;
          const uint32_t fb = PAIR ? map_to_rank(smem_addr(&b_full[s]), 0) : smem_addr(&b_full[s]);
          if (leader) mbar_expect_tx(smem_addr(&b_full[s]), b_bytes * CG);
          const bool second = MODE == kModeBackward && st >= a.steps_w;
          tma_load<CG>(b_base + s * b_bytes, second ? &a.map_x1 : &a.map_x0, (second ? st - a.steps_w : st) * kBK, n0, fb);
          ++issued;
          if (++s == b_stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (s_abort && leader) let_land(b_full, s, ph, b_stages, issued);
    }
    __syncwarp();
  } else if (warp == 2) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, issued = 0;
      bool ok = true;
      for (int t = first; t < tile_end && ok; t += tile_step) {
        const int m0 = tile_m0(t);
        for (int st = st_begin; st < st_end; st += kStepsPerCode) {
          if (!(ok = tc_wait(smem_addr(&c_empty[s]), ph ^ 1u, &s_abort))) break;
          const uint32_t fb = smem_addr(&c_full[s]), dst = c_base + s * (kStepsPerCode * kCodeBytes);
          mbar_expect_tx(fb, kStepsPerCode * kCodeBytes);
          if constexpr (MODE == kModeBackward) {
            // 64 weight rows x 128 columns (64 bytes)
            const bool second = st >= a.steps_w;
            tma_load<1>(dst, second ? &a.map_w1 : &a.map_w0, m0 / 2, (second ? st - a.steps_w : st) * kBK, fb);
          } else if constexpr (MODE == kModeGated) {
            // 16 gate rows, the same 16 up rows, ...: 128 columns (64 bytes) each
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              tma_load<1>(dst + q * 2048u, &a.map_w0, st * (kBK / 2), m0 + 16 * q, fb);
              tma_load<1>(dst + q * 2048u + 1024u, &a.map_w1, st * (kBK / 2), m0 + 16 * q, fb);
            }
          } else {
            tma_load<1>(dst, &a.map_w0, st * (kBK / 2), m0, fb);
          }
          ++issued;
          if (++s == kSlots) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (s_abort) let_land(c_full, s, ph, kSlots, issued);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      const uint32_t idesc = idesc_of(kBM * CG, a.n, MODE == kModeBackward);
      int bs = 0, as = 0, buf = 0;
      uint32_t bph = 0, aph = 0, dph = 3u;  // dph: parity bit per accumulator of the next "empty" wait
      bool ok = true;
      for (int t = first; t < tile_end && ok; t += tile_step) {
        for (int st = st_begin; st < st_end; ++st) {
          // a sum starts: the tile's first step, or (backward) the second weight's
          const bool start = st == st_begin || (MODE == kModeBackward && st == a.steps_w);
          if (start) {
            if (st != st_begin) {
              tc_commit<CG>(smem_addr(&d_full[buf]));
              buf ^= 1;
            }
            if (!(ok = tc_wait(smem_addr(&d_empty[buf]), (dph >> buf) & 1u, &s_abort))) break;
            dph ^= 1u << buf;
          }
          if (!(ok = tc_wait(smem_addr(&b_full[bs]), bph, &s_abort) && tc_wait(smem_addr(&a_full[as]), aph, &s_abort))) break;
          tc_fence_after();
          const uint32_t at = a_base + as * (kTerms * kABytes);
          const uint64_t bd = desc_sw128(b_base + bs * b_bytes, 16u, 1024u);
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j) {
#pragma unroll
            for (int k = 0; k < kTerms; ++k) {
              // K-major A: lines of 128 bytes, 32 bytes a 16-wide step; MN-major A: two slabs of
              // 64 outputs, 8 KiB apart, 16 lines (2 KiB) a step
              const uint64_t ad = MODE == kModeBackward ? desc_sw128(at + k * kABytes, 8192u, 1024u) + 128u * j
                                                        : desc_sw128(at + k * kABytes, 16u, 1024u) + 2u * j;
              tc_mma<CG>(tmem + static_cast<uint32_t>(buf) * 256u, ad, bd + 2u * j, idesc, !(start && j == 0 && k == 0));
            }
          }
          tc_commit<CG>(smem_addr(&a_empty[as]));
          tc_commit<CG>(smem_addr(&b_empty[bs]));
          if (++as == kAStages) {
            as = 0;
            aph ^= 1u;
          }
          if (++bs == b_stages) {
            bs = 0;
            bph ^= 1u;
          }
        }
        if (!ok) break;
        if (st_begin < st_end) {
          tc_commit<CG>(smem_addr(&d_full[buf]));
          buf ^= 1;
        }
      }
      // every MMA issued has completed before tensor memory and shared memory are released
      tc_commit<CG>(smem_addr(&drain));
    }
    __syncwarp();
  } else if (warp >= kDecWarp0 && warp < kDecWarp0 + kDecWarps) {
    // thread i: line i % 128 (an output; backward: a slab's weight row), half i / 128 of its 64
    const int i = tid - kDecWarp0 * 32, line = i & 127, half = i >> 7;
    const uint32_t line_addr = 128u * line;
    const uint32_t full0 = PAIR ? map_to_rank(smem_addr(&a_full[0]), 0) : smem_addr(&a_full[0]);
    int as = 0, cs = 0;
    uint32_t aph = 0, cph = 0;
    bool ok = true;
    for (int t = first; t < tile_end && ok; t += tile_step) {
      const int m0 = tile_m0(t);
      // the scales of step st, (row, first column) of this thread's 32 weights
      const auto scales_of = [&](int st) {
        int row, col;
        const void* base;
        if constexpr (MODE == kModeBackward) {
          const bool second = st >= a.steps_w;
          row = (second ? st - a.steps_w : st) * kBK + (line & 63);
          col = m0 + 64 * (line >> 6) + 32 * half;
          base = second ? a.scales1 : a.scales0;
        } else {
          col = st * kBK + 32 * half;
          if constexpr (MODE == kModeGated) {
            row = m0 + 16 * (line >> 5) + (line & 15);
            base = (line & 16) ? a.scales1 : a.scales0;
          } else {
            row = m0 + line;
            base = a.scales0;
          }
        }
        const bool in = st < st_end && row < (MODE == kModeBackward ? a.nsum : a.nout) && col < a.p.cols;
        return load_scales<FMT>(base, static_cast<int64_t>(row) * a.blocks_row, col, a.p.log2_block, in);
      };
      constexpr int kAhead = 4;  // steps that the scales are loaded ahead
      Scales<FMT> sc[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) sc[k] = scales_of(st_begin + k);
      for (int st0 = st_begin; st0 < st_end && ok; st0 += kAhead) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int st = st0 + k;
          if (st >= st_end) break;
          const int sub = kStepsPerCode == 2 ? k & 1 : 0;  // slices start at even steps
          if (sub == 0 && !__all_sync(kFull, tc_wait(smem_addr(&c_full[cs]), cph, &s_abort))) {
            ok = false;
            break;
          }
          // the code box has 64-byte lines, 64-byte swizzle: 16-byte chunk c of line l is at
          // c ^ (l / 2 % 4)
          const int cl = MODE == kModeBackward ? line & 63 : line;
          const int c = MODE == kModeBackward ? 2 * (line >> 6) + half : 2 * sub + half;
          const uint4 codes = lds16(c_base + cs * (kStepsPerCode * kCodeBytes) + 64u * cl + static_cast<uint32_t>((c ^ ((cl >> 1) & 3)) << 4));
          const Scales<FMT> now = sc[k];
          sc[k] = scales_of(st + kAhead);
          if (sub == kStepsPerCode - 1 || st + 1 == st_end) {
            __syncwarp();
            if (lane == 0) arrive_cluster(smem_addr(&c_empty[cs]));
            if (++cs == kSlots) {
              cs = 0;
              cph ^= 1u;
            }
          }
          if (!__all_sync(kFull, tc_wait(smem_addr(&a_empty[as]), aph ^ 1u, &s_abort))) {
            ok = false;
            break;
          }
          decode32<FMT>(codes, now, a_base + as * (kTerms * kABytes), line_addr, line, half);
          fence_proxy_async();  // the stores, before the tensor cores read them
          __syncwarp();
          if (lane == 0) arrive_cluster(full0 + 8u * as);
          if (++as == kAStages) {
            as = 0;
            aph ^= 1u;
          }
        }
      }
    }
  } else if (PAIR && warp >= kEpiWarp0) {
    const int quarter = warp & 3;
    const StoreFlags fl{(reinterpret_cast<uintptr_t>(a.p.y) & 3u) == 0 && (a.p.ld_y & 1) == 0,
                        (reinterpret_cast<uintptr_t>(a.p.g_out) & 3u) == 0 && (reinterpret_cast<uintptr_t>(a.p.u_out) & 3u) == 0 && (a.p.ld_gu & 1) == 0};
    constexpr float kUnit = FMT == QZ_NVFP4 ? 256.0f : 1.0f;  // decoded NVFP4 weights are 2^-8 of their value
    const float f0 = sum_factor<FMT>(a.tscale0) * kUnit, f1 = a.p.n_weights == 2 ? sum_factor<FMT>(a.tscale1) * kUnit : 0.0f;
    const bool two = MODE == kModeBackward && a.p.n_weights == 2;
    int buf = 0;
    uint32_t fph = 0;  // parity bit per accumulator
    bool ok = true;
    for (int t = first; t < tile_end; t += tile_step) {
      const int m0 = tile_m0(t), n0 = tile_n0(t);
      for (int k = 0; k < (two ? 2 : 1) && ok; ++k) {
        const int b = buf ^ k;
        ok = __all_sync(kFull, tc_wait(smem_addr(&d_full[b]), (fph >> b) & 1u, &s_abort));
        fph ^= 1u << b;
      }
      tc_fence_after();
      const uint32_t ta = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
      for (int c = 0; c < a.n && n0 + c < a.p.tokens; c += 8) {
        float v[8];
        if (ok) {
          tmem_ld8(ta + 256u * buf + c, v);
          if (two) {
            float w[8];
            tmem_ld8(ta + 256u * (buf ^ 1) + c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fmaf_rn(w[i], f1, v[i] * f0);
          } else if (MODE != kModeGated) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= f0;
          }
        } else {  // a wait gave up: NaN instead of a wrong result
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(0x7fc00000u);
        }
        store8<FMT, MODE>(a, fl, v, f0, f1, m0, quarter, lane, n0 + c);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        for (int k = 0; k < (two ? 2 : 1); ++k) {
          const uint32_t bar = smem_addr(&d_empty[buf ^ k]);
          arrive_cluster(map_to_rank(bar, 0));
        }
      }
      if (!two) buf ^= 1;
    }
  }

  // every MMA has completed (or its wait has given up) before shared and tensor memory go
  __syncthreads();
  const bool done = __all_sync(kFull, st_begin >= st_end || tc_wait(smem_addr(&drain), 0u, &s_abort)) && !s_abort;
  tc_fence_after();
  if constexpr (!PAIR) {
    // ---- the slices of the tile: partial sums to the CTA that finishes their columns ----------
    const int slices = a.slices, cols = a.n / slices;  // columns this CTA finishes
    const int quarter = warp & 3, part = warp >> 2;    // 16 warps: four column parts a quarter
    const uint32_t ta = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    constexpr float kUnit = FMT == QZ_NVFP4 ? 256.0f : 1.0f;
    const float f0 = sum_factor<FMT>(a.tscale0) * kUnit, f1 = a.p.n_weights == 2 ? sum_factor<FMT>(a.tscale1) * kUnit : 0.0f;
    const bool has0 = MODE == kModeBackward ? st_begin < min(st_end, a.steps_w) : st_begin < st_end;
    const bool has1 = MODE == kModeBackward && max(st_begin, a.steps_w) < st_end;
    const int m0 = tile_m0(first), n0 = tile_n0(first);
    // 8 columns of this CTA's own partial sums; the backward pass joins its weights' here
    const auto own = [&](int c, float (&v)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      if (!done) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(0x7fc00000u);
        return;
      }
      if (has0) tmem_ld8(ta + c, v);
      if constexpr (MODE == kModeBackward) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= f0;
        if (has1) {
          float w[8];
          tmem_ld8(ta + (has0 ? 256u : 0u) + c, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __fmaf_rn(w[i], f1, v[i]);
        }
      }
    };
    if (slices > 1) {
      cluster_sync();  // every slice's rings are idle: their memory takes the partial sums
      for (int c = 8 * part; c < a.n; c += 32) {
        const int dst = c / cols;
        if (dst == static_cast<int>(rank) || n0 + c >= a.p.tokens) continue;
        float v[8];
        own(c, v);
        const uint32_t to = map_to_rank(base + ((rank * cols + (c - dst * cols)) * kBM + 32 * quarter + lane) * 4u, dst);
#pragma unroll
        for (int i = 0; i < 8; ++i) st_cluster(to + i * (kBM * 4u), v[i]);
      }
      cluster_sync();
    }
    const StoreFlags fl{(reinterpret_cast<uintptr_t>(a.p.y) & 3u) == 0 && (a.p.ld_y & 1) == 0,
                        (reinterpret_cast<uintptr_t>(a.p.g_out) & 3u) == 0 && (reinterpret_cast<uintptr_t>(a.p.u_out) & 3u) == 0 && (a.p.ld_gu & 1) == 0};
    const int c_begin = static_cast<int>(rank) * cols;
    for (int c = 8 * part; c < cols && n0 + c_begin + c < a.p.tokens; c += 32) {
      float mine[8], v[8];
      own(c_begin + c, mine);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      for (int s = 0; s < slices; ++s) {  // slice order
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float w = mine[i];
          if (s != static_cast<int>(rank))
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w) : "r"(base + ((s * cols + c + i) * kBM + 32 * quarter + lane) * 4u) : "memory");
          v[i] += w;
        }
      }
      if constexpr (MODE == kModeLinear) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= f0;
      }
      store8<FMT, MODE>(a, fl, v, f0, f1, m0, quarter, lane, n0 + c_begin + c);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while another may still signal it
  if (warp == 3) {
    tc_fence_after();
    if constexpr (CG == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// ---- host side ----------------------------------------------------------------------------------
inline bool encode(CUtensorMap* m, bool codes, const void* base, int64_t inner, int64_t outer, int64_t pitch, int box_in, int box_out) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_in), static_cast<cuuint32_t>(box_out)}, es[2] = {1, 1};
  return enc(m, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
             box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, codes ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int MODE, bool PAIR>
qz_status run_tc(const TcArgs& a, int grid, cudaStream_t s) {
  const void* k = reinterpret_cast<const void*>(&product_tc_kernel<FMT, MODE, PAIR>);
  if (!set_dyn_smem(k, static_cast<int>(kSmemMax))) return QZ_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = PAIR ? 2u : static_cast<unsigned>(a.slices);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreadsTc);
  cfg.dynamicSmemBytes = kSmemMax;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<TcArgs*>(&a)};
  if (cudaLaunchKernelExC(&cfg, k, args) != cudaSuccess) {
    cudaGetLastError();
    return QZ_ERR_CUDA;
  }
  return launch_status();
}

// The form and its tiles.  Estimated in SM cycles: a step's MMAs take 2 cycles a token column
// (128 x n x 64 at 8192 FLOP a cycle; about 2.8 where one CTA loads all the tokens, the
// shared-memory bandwidth), its decoding about 300; a tile of the second form starts with an empty
// pipeline and ends with the exchange.
struct Plan {
  bool pair;
  int n, tiles_n, tiles, slices, slice_steps, grid;
};
inline Plan plan_of(int64_t nout, int out_per_cta, int64_t tokens, int steps, int even, int terms) {
  const int sms = sm_count();
  Plan best{};
  double best_cost = 1e30;
  const int64_t tn256 = (tokens + 255) / 256;
  const int n = static_cast<int>(((tokens + tn256 - 1) / tn256 + 31) / 32 * 32);
  const int64_t tiles_n = (tokens + n - 1) / n;
  {
    const int64_t tiles = (nout + 2 * out_per_cta - 1) / (2 * out_per_cta) * tiles_n;
    const int64_t pairs = std::max(1, sms / 2);
    const double cost = static_cast<double>((tiles + pairs - 1) / pairs) * steps * std::max(2.0 * n, 300.0) * terms + 6000;
    if (tiles < (int64_t{1} << 30)) {
      best = Plan{true, n, static_cast<int>(tiles_n), static_cast<int>(tiles), 1, steps, static_cast<int>(2 * std::min(tiles, pairs))};
      best_cost = cost;
    }
  }
  for (int s = 1; s <= 8; s *= 2) {
    const int ns = n % (8 * s) ? (n + 8 * s - 1) / (8 * s) * (8 * s) : n;  // columns divide into eights per slice
    const int64_t tiles = (nout + out_per_cta - 1) / out_per_cta * tiles_n;
    int per = (steps + s - 1) / s;
    per += per % even;
    const int64_t clusters = std::max(1, s == 1 ? sms : (s == 2 ? sms * 9 / 10 : sms * 5 / 6) / s);
    const double cost = static_cast<double>((tiles + clusters - 1) / clusters) * (per * std::max(2.8 * ns, 300.0) * terms + 5000 + (s > 1 ? 2000 + 16.0 * ns : 0));
    if (ns <= 256 && tiles * s < (int64_t{1} << 30) && cost < best_cost) {
      best = Plan{false, ns, static_cast<int>(tiles_n), static_cast<int>(tiles), s, per, static_cast<int>(tiles * s)};
      best_cost = cost;
    }
  }
  return best;
}

template <int FMT>
qz_status launch_tc(const ProductArgs& p, cudaStream_t s) {
  TcArgs a{};
  const bool back = p.mode == kModeBackward;
  a.p = p;
  a.scales0 = p.w0.scales;
  a.scales1 = p.w1.scales;
  a.tscale0 = p.w0.tscale;
  a.tscale1 = p.w1.tscale;
  a.nout = static_cast<int>(back ? p.cols : p.rows);
  a.nsum = static_cast<int>(back ? p.rows : p.cols);
  a.blocks_row = static_cast<int>(p.cols >> p.log2_block);
  a.steps_w = (a.nsum + kBK - 1) / kBK;
  a.steps = back ? a.steps_w * p.n_weights : a.steps_w;
  const Plan plan = plan_of(a.nout, p.mode == kModeGated ? kBM / 2 : kBM, p.tokens, a.steps, back ? 1 : 2, TcFormat<FMT>::kTerms);
  if (plan.grid == 0) return QZ_ERR_UNSUPPORTED;
  a.n = plan.n;
  a.tiles_n = plan.tiles_n;
  a.tiles = plan.tiles;
  a.slices = plan.slices;
  a.slice_steps = plan.slice_steps;
  const int b_rows = plan.pair ? plan.n / 2 : plan.n;
  a.b_stages = static_cast<int>(std::min<uint32_t>(kMaxBStages, kBRoom<FMT> / (static_cast<uint32_t>(b_rows) * kBK * 2)));
  const int code_rows = back ? 64 : (p.mode == kModeGated ? 16 : 128);
  bool ok = encode(&a.map_x0, false, p.x0, a.nsum, p.tokens, p.ld_x * 2, kBK, b_rows) &&
            encode(&a.map_w0, true, p.w0.codes, p.cols / 2, p.rows, p.cols / 2, 64, code_rows);
  if (p.n_weights == 2) ok = ok && encode(&a.map_w1, true, p.w1.codes, p.cols / 2, p.rows, p.cols / 2, 64, code_rows);
  if (p.n_weights == 2 && back) ok = ok && encode(&a.map_x1, false, p.x1, a.nsum, p.tokens, p.ld_x * 2, kBK, b_rows);
  if (!ok) return QZ_ERR_CUDA;
  if (plan.pair) {
    if (p.mode == kModeLinear) return run_tc<FMT, kModeLinear, true>(a, plan.grid, s);
    if (p.mode == kModeGated) return run_tc<FMT, kModeGated, true>(a, plan.grid, s);
    return run_tc<FMT, kModeBackward, true>(a, plan.grid, s);
  }
  if (p.mode == kModeLinear) return run_tc<FMT, kModeLinear, false>(a, plan.grid, s);
  if (p.mode == kModeGated) return run_tc<FMT, kModeGated, false>(a, plan.grid, s);
  return run_tc<FMT, kModeBackward, false>(a, plan.grid, s);
}

}  // namespace
}  // namespace qz
