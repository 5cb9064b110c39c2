// qz_product_tc.cuh -- products with 4-bit weights on the tcgen05 tensor cores (more than a few
// tokens), included once per weight format.
//
//   forward   D[r][t] = sum_c W[r][c] x[t][c]          backward  D[c][t] = sum_r W[r][c] dy[t][r]
//
// The weights are the MMA's A operand (M: 128 outputs a CTA, one tensor-memory lane each), the
// activations its B operand (N: up to 256 tokens, one fp32 tensor-memory column each).  E2M1
// times its block scale has at most 6 significant bits and so is exact in bf16: kind::f16 with fp32
// accumulation gives the sums of include/qz.h without a rounding of the weights.  An INT4 weight q s
// is held as the sum of two bf16 values (2^-17 of it at most away) and takes two MMAs; three would
// hold it and take half as long again.
//
// Roles of a CTA's warps (every wait is bounded):
//   warp 0       streams the tokens' boxes (128 summands, INT4 64) into a ring by TMA
//   warp 2       streams the 4-bit codes' boxes into a ring of their own by TMA
//   decoders     three groups of four warps that take the boxes in turn: a thread turns a line's
//                codes into bf16 and stores them in the layout the MMA reads
//   warp 1       issues the MMAs, eight 16-wide ones a box (one thread)
//   the rest     read finished accumulators from tensor memory, apply the activation and store
// A box is the unit of every hand-over: a wait or a commit of the issuing thread takes some 60 to
// 140 cycles even when nothing is to be waited for, which 64-wide steps paid twice as often.
// Two forms.  PAIR: two CTAs on neighbouring SMs share one 256 x 256 tile (cta_group::2: each
// decodes its own 128 outputs and loads half of the tokens, so the shared-memory traffic per MMA
// halves), persistent over the tiles, the epilogue of a tile beside the next tile's MMAs (two
// accumulators of 256 columns).  Alone: a CTA has a tile of 128 outputs and one slice of the sum;
// the CTAs of a cluster hold the slices of one tile, exchange their partial sums through
// distributed shared memory and add them in slice order, so few tokens still fill the GPU and
// equal inputs give equal results.
//
// Measured, NVFP4, passes one after the other for seconds: gated 4096 tokens, 2 x 16384 x 4096: 659 us,
// 1.67 PFLOP/s, at 1552 MHz under the power cap, bound by the tensor cores (the library's product of
// that size on bf16 weights, measured likewise: 610 us at 1507 MHz); 2048 tokens backward, 8192 x 4096:
// 94 us, 1.46 PFLOP/s at 1972 MHz, the last round of tiles (the library 86).  MXFP4, gated 77 tokens,
// 2 x 10240 x 4096: 33 us on the GPU in two launches, bound by the decoders (842 cycles a box against
// 384 of MMAs) and the starts.
#pragma once

#include <cuda.h>  // CUtensorMap and its enumerators (types only; the encoder is looked up)
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "qz_device.cuh"
#include "qz_internal.h"
#include "qz_pipe.cuh"
#include "qz_product.h"
#include "qz_product_plan.h"
#include "qz_weight.cuh"

namespace qz {
namespace {

constexpr int kBK = 64;             // summands per step: 128 bytes of bf16, one swizzle row
constexpr int kDecWarp0 = 4;
constexpr uint32_t kABytes = kBM * kBK * 2;        // 16 KiB of decoded weights
constexpr uint32_t kTmemCols = 512;                // two accumulators of 256 columns
constexpr uint64_t kTcWaitNs = 1000000000ull;      // 1 s: far beyond any step's latency
constexpr int kMaxBStages = 8, kMaxGroups = 3, kMaxBoxes = 6;

template <int FMT>
struct TcFormat {
  static constexpr int kTerms = FMT == QZ_INT4 ? 2 : 1;      // bf16 terms per weight
  static constexpr int kSteps = FMT == QZ_INT4 ? 1 : 2;      // 64-wide steps of a box: eight MMAs
  static constexpr int kBoxK = kSteps * kBK;
  static_assert(kBoxK == box_of(FMT));
  static constexpr uint32_t kBoxBytes = kBM * kBoxK / 2;     // of codes
  static constexpr int kGroups = 3;                          // decoder groups of four warps
  // Stages of decoded weights: one box per group.  Both this ring and the code ring hold a whole
  // number of rounds of the groups, so a slot belongs to one group, which is never a lap ahead of
  // another on it (a parity wait could not tell the laps apart).
  static constexpr uint32_t kStageBytes = kSteps * kTerms * kABytes;  // 32 KiB
  static constexpr int kEpiWarp0 = kDecWarp0 + 4 * kGroups;
  // Eight epilogue warps (a tile's columns in two halves) where a box is 128 summands; INT4's MMAs
  // take twice as long per tile.
  static constexpr int kEpiWarps = FMT == QZ_INT4 ? 4 : 8;
  static constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
};
constexpr uint32_t kSmemMax = 227 * 1024 - 2048;   // dynamic; the barriers are static
template <int FMT>
constexpr uint32_t kRingRoom = kSmemMax - 1024 - TcFormat<FMT>::kGroups * TcFormat<FMT>::kStageBytes;  // codes and tokens

struct TcArgs {
  CUtensorMap map_x0, map_x1;  // bf16 [tokens][sum], box 64 x (tokens of a CTA's load)
  CUtensorMap map_w0, map_w1;  // codes [rows][cols / 2] bytes
  const void *scales0, *scales1;
  const float *tscale0, *tscale1;
  ProductArgs p;
  int nout, nsum;         // outputs and summands (per weight)
  int blocks_row;         // scales per weight row
  int boxes_w, boxes;     // boxes per weight (past the sum's end copies give zeros), in all
                          // (backward: both weights' one after the other)
  int n;                  // tokens per tile (a multiple of 32)
  int code_slots, b_stages;  // slots of the code ring (a multiple of the groups), of the tokens' ring
  int scales_vec;         // 1: the scales of 64 columns are one aligned load; 2: those of 128 are
  int tiles_n, tiles, m_base;  // tiles of tokens, in all; the first output of the first
  int slices, slice_boxes;  // Alone: slices of the sum (the cluster), boxes per slice
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
__device__ __forceinline__ void arrive_local(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrive on a barrier of another CTA of the cluster (a shared::cluster address).  What it announces
// is read by the tensor core of this SM, behind a proxy fence, and by no thread of the other CTA,
// so the default scope does; release.cluster waits for every load in flight (1100 cycles a step).
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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
// 8 consecutive fp32 columns of this thread's tensor-memory lane: the load, and the wait for every
// load before it, which hands the registers on (so nothing reads them earlier)
__device__ __forceinline__ void tmem_load8(uint32_t taddr, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait8(float (&v)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])::"memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  tmem_load8(taddr, v);
  tmem_wait8(v);
}
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void sts16(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
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

// Bounded wait on phase `parity`.
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kTcWaitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// One lane of a converged warp.  The compiler knows that at most one thread passes, and so feeds
// the uniform operands of tcgen05 and TMA instructions without a loop over the lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
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
    while (!mbar_try_wait(smem_addr(&full[s]), ph) && globaltimer_ns() - t0 < kTcWaitNs) {
    }
  }
}

// ---- decoding -------------------------------------------------------------------------------
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

// The scales of one 64-wide step of a line: two E8M0 bytes, four E4M3 bytes, or fp32 (of each 16
// columns).
template <int FMT>
struct Scales {
  uint32_t v[FMT == QZ_INT4 ? 4 : 1];
};
// Those of 64 columns from `col` on; p: the scales of the row.  Outside the weight they are 0 (finite; the
// codes there are 0).
template <int FMT>
__device__ __forceinline__ Scales<FMT> load_scales(const uint8_t* p, int col, int cols, int log2_block, bool vec) {
  Scales<FMT> s{};
  if (p == nullptr || col >= cols) return s;
  if constexpr (FMT == QZ_INT4) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p) + (col >> log2_block);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + 16 * i < cols) s.v[i] = __ldg(q + ((16 * i) >> log2_block));
  } else {
    constexpr int kN = FMT == QZ_MXFP4 ? 2 : 4;  // bytes
    p += static_cast<uint32_t>(col) / (64 / kN);
    if (vec) {
      if constexpr (FMT == QZ_MXFP4) s.v[0] = __ldg(reinterpret_cast<const uint16_t*>(p));
      else s.v[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
#pragma unroll
      for (int q = 0; q < kN; ++q)
        if (col + (64 / kN) * q < cols) s.v[0] |= static_cast<uint32_t>(__ldg(p + q)) << (8 * q);
    }
  }
  return s;
}
// Those of a box's two steps, 128 columns, as one aligned load (cols % 128 == 0).
template <int FMT>
__device__ __forceinline__ void load_scales_box(const uint8_t* p, int col, Scales<FMT> (&s)[2]) {
  static_assert(FMT != QZ_INT4, "two-step boxes");
  if (p == nullptr) {
    s[0] = s[1] = Scales<FMT>{};
  } else if constexpr (FMT == QZ_MXFP4) {
    const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(p + static_cast<uint32_t>(col) / 32u));
    s[0].v[0] = v;  // the second step's bytes lie above the first's
    s[1].v[0] = v >> 16;
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + static_cast<uint32_t>(col) / 16u));
    s[0].v[0] = v.x;
    s[1].v[0] = v.y;
  }
}

// 32 weights (16 bytes of codes; half h of a line's 64) to bf16, stored as chunks 4 h .. 4 h + 3
// of the line at `dst`, each at its swizzled place (x: line % 8).  ANY: E4M3 scales may be NaN (0x7F) or negative.
template <int FMT, bool ANY>
__device__ __forceinline__ void decode32(const uint4 codes, const Scales<FMT>& s, uint32_t dst, int x, int h) {
  const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t f0, f1;  // bf16 pairs: the factor of the first and the second 16 weights
  uint32_t extra = 0x3F803F80u;
  bool big = false;
  if constexpr (FMT == QZ_MXFP4) {
    // 2^(E - 127) 2^126 as bf16 has exponent field E + 126; what exceeds 254 is a second factor
    const uint32_t E = (s.v[0] >> (8 * h)) & 255u;
    f0 = E == 255u ? 0x7FC07FC0u : (min(E + 126u, 254u) << 7) * 0x00010001u;
    f1 = f0;
    big = E > 128u;
    if (big) extra = ((E - 1u) << 7) * 0x00010001u;  // 2^(E - 128); NaN stays NaN
  } else if constexpr (FMT == QZ_NVFP4) {
    // an E4M3 byte at bits 4-10 is its value times 2^-120 as bf16; 2^127 and 2^111 bring it to
    // 2^118 times its value (below 2^127), so a weight comes out as 2^-8 of its own
    const uint32_t b = s.v[0] >> (16 * h);
    if constexpr (ANY) {
      const float v0 = dec_e4m3(b & 255u) * 0x1p118f, v1 = dec_e4m3((b >> 8) & 255u) * 0x1p118f;
      f0 = bf16x2_bits(v0, v0);
      f1 = bf16x2_bits(v1, v1);
    } else {
      uint32_t c = ((b & 255u) << 4) | ((b & 0xff00u) << 12);
      c = mul_bf16x2(mul_bf16x2(c, 0x7F007F00u), 0x77007700u);
      f0 = (c & 0xffffu) * 0x00010001u;
      f1 = (c >> 16) * 0x00010001u;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t t0 = cw[j] & 0x0F0F0F0Fu, t1 = (cw[j] >> 4) & 0x0F0F0F0Fu;
    uint32_t d[4] = {nibble_pair<0>(t0, t1), nibble_pair<1>(t0, t1), nibble_pair<2>(t0, t1), nibble_pair<3>(t0, t1)};
    const uint32_t at = dst + static_cast<uint32_t>(((4 * h + j) ^ x) << 4);
    if constexpr (FMT == QZ_INT4) {
      const float sc = __uint_as_float(s.v[2 * h + (j >> 1)]);
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
// Neighbouring lanes hold neighbouring outputs r of two tokens t and t' (a and b), as a bf16 pair:
// after the exchange the even lane has both outputs of t, the odd lane both of t'.
__device__ __forceinline__ uint32_t exchange_pair(float a, float b, bool odd) {
  const uint32_t own = bf16x2_bits(a, b), other = __shfl_xor_sync(kFull, own, 1);
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(own), "r"(other), "r"(odd ? 0x3276u : 0x5410u));
  return r;
}
__device__ __forceinline__ void store_pair(uint16_t* q, uint32_t v, int row, int rows, bool vec) {
  if (vec && row + 1 < rows) {
    *reinterpret_cast<uint32_t*>(q) = v;
  } else {
    if (row < rows) q[0] = static_cast<uint16_t>(v);
    if (row + 1 < rows) q[1] = static_cast<uint16_t>(v >> 16);
  }
}

// A tile's stores: where this lane's values go, and whether every one of them is an aligned pair
// inside the matrices (then no store is tested).
struct StorePlan {
  bool whole;                // of the CTA's tile and this call's columns
  bool y_vec, gu_vec;
  int row;                   // this lane's first output (even), or its one output (fp32)
  uint32_t token_off;        // its token within a group of eight
};
template <int MODE>
__device__ __forceinline__ StorePlan store_plan(const TcArgs& a, int m0, int quarter, int lane, int64_t t_begin, int64_t t_end) {
  const ProductArgs& p = a.p;
  StorePlan f;
  f.y_vec = (reinterpret_cast<uintptr_t>(p.y) & 3u) == 0 && (p.ld_y & 1) == 0;
  f.gu_vec = (reinterpret_cast<uintptr_t>(p.g_out) & 3u) == 0 && (reinterpret_cast<uintptr_t>(p.u_out) & 3u) == 0 && (p.ld_gu & 1) == 0;
  const int first = MODE == kModeGated ? m0 + 16 * quarter : m0 + 32 * quarter;
  f.whole = t_end <= p.tokens && first + (MODE == kModeGated ? 16 : 32) <= a.nout && f.y_vec && (f.gu_vec || !p.g_out);
  if (MODE == kModeGated) {
    f.row = first + (lane & 14);
    f.token_off = (lane >> 4) + 2 * (lane & 1);
  } else if (p.out_f32) {
    f.row = first + lane;
    f.token_off = 0;
  } else {
    f.row = first + (lane & 30);
    f.token_off = lane & 1;
  }
  return f;
}

// 8 finished sums of this thread's lane, tokens t0 .. t0 + 7.
template <int MODE>
__device__ __forceinline__ void store8(const TcArgs& a, const StorePlan& f, const float (&v)[8], float f0, float f1, int lane, int64_t t0) {
  const ProductArgs& p = a.p;
  const int64_t tokens = p.tokens;
  const bool odd = lane & 1;
  if constexpr (MODE == kModeGated) {
    // lanes 0-15 hold gate sums, 16-31 the same outputs' up sums: each half takes one token of
    // a pair from the other, so lane l ends with tokens 2 i (+ 1 in the upper half)
    const bool upper = lane >= 16;
    float g[4], u[4], h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float got = __shfl_xor_sync(kFull, upper ? v[2 * i] : v[2 * i + 1], 16);
      g[i] = (upper ? got : v[2 * i]) * f0;
      u[i] = (upper ? v[2 * i + 1] : got) * f1;
    }
    if (p.act == QZ_ACT_SILU) {
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = act_value<QZ_ACT_SILU>(g[i]) * u[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = act_value<QZ_ACT_GELU_TANH>(g[i]) * u[i];
    }
    const int64_t t = t0 + f.token_off;
    const auto put = [&](uint16_t* dst, int64_t ld, bool vec, const float (&w)[4]) {
      const uint32_t e0 = exchange_pair(w[0], w[1], odd), e1 = exchange_pair(w[2], w[3], odd);
      uint16_t* q = dst + t * ld + f.row;
      if (f.whole) {
        *reinterpret_cast<uint32_t*>(q) = e0;
        *reinterpret_cast<uint32_t*>(q + 4 * ld) = e1;
      } else {
        if (t < tokens) store_pair(q, e0, f.row, a.nout, vec);
        if (t + 4 < tokens) store_pair(q + 4 * ld, e1, f.row, a.nout, vec);
      }
    };
    put(static_cast<uint16_t*>(p.y), p.ld_y, f.y_vec, h);
    if (p.g_out) {
      put(p.g_out, p.ld_gu, f.gu_vec, g);
      put(p.u_out, p.ld_gu, f.gu_vec, u);
    }
  } else if (p.out_f32) {
    float* y = static_cast<float*>(p.y) + t0 * p.ld_y + f.row;
    if (f.row < a.nout) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t0 + i < tokens) y[i * p.ld_y] = v[i];
    }
  } else {
    uint16_t* q = static_cast<uint16_t*>(p.y) + (t0 + f.token_off) * p.ld_y + f.row;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t e = exchange_pair(v[2 * i], v[2 * i + 1], odd);
      if (f.whole) *reinterpret_cast<uint32_t*>(q + 2 * i * p.ld_y) = e;
      else if (t0 + f.token_off + 2 * i < tokens) store_pair(q + 2 * i * p.ld_y, e, f.row, a.nout, f.y_vec);
    }
  }
}

// ---- the decoder warps -------------------------------------------------------------------------
struct DecodeLoop {
  int group, line, lane, first, tile_end, tile_step, bx_begin, bx_end, m_rank;
  uint32_t a_stage, c_full, c_empty, a_empty, a_full;
  const uint8_t* codes;
  volatile int* abort;
};
// Group g of four warps takes every kGroups-th box; thread i of it line i of each: an output
// (backward: weight row i % 64 of a step, outputs 64 (i / 64) .. + 63).  VEC: the scales of a box
// (INT4, backward: of 64 columns) are one aligned load.  It is a parameter of the whole loop: where
// two ways of loading met, the loaded registers would be copied and so be waited for at once.
template <int FMT, int MODE, bool PAIR, bool VEC>
__device__ __forceinline__ void decode_boxes(const TcArgs& a, const DecodeLoop& d) {
  constexpr int kSteps = TcFormat<FMT>::kSteps, kBoxK = TcFormat<FMT>::kBoxK, kGroups = TcFormat<FMT>::kGroups;
  constexpr int kTerms = TcFormat<FMT>::kTerms, kOut = MODE == kModeGated ? kBM / 2 : kBM, CG = PAIR ? 2 : 1;
  constexpr uint32_t kBoxBytes = TcFormat<FMT>::kBoxBytes;
  const int line = d.line, x = line & 7, cols = static_cast<int>(a.p.cols);
  // the code box has 64-byte lines with a 64-byte swizzle, 16-byte chunk c of line l at
  // c ^ (l / 2 % 4), or 32-byte ones (c ^ (l / 4 % 2)); a thread's chunks are 2 k and 2 k + 1 of
  // step k (backward: of its slab), so eight lanes' 16-byte loads take different banks
  constexpr uint32_t kLine = MODE == kModeBackward ? 64u : kBoxK / 2;
  const int cl = MODE == kModeBackward ? line & 63 : line, cx = kLine == 64 ? (cl >> 1) & 3 : (cl >> 2) & 1;
  const int per_tile = d.bx_end - d.bx_begin;
  int t = d.first, bx = d.bx_begin + d.group;  // this group's box
  int cs = d.group;
  uint32_t aph = 0, cph = 0;
  constexpr int kScaleBytes = FMT == QZ_INT4 ? 4 : 1;
  const int64_t pitch = static_cast<int64_t>(a.blocks_row) * kScaleBytes;
  const uint8_t* row_scales = nullptr;  // forward: of this thread's line in tile `row_tile` (null: outside)
  int row_tile = -1;
  Scales<FMT> next[kSteps] = {};
  const auto settle = [&]() {  // a box past the tile's end: the next tiles'
    while (t < d.tile_end && bx >= d.bx_end) {
      bx -= per_tile;
      t += d.tile_step;
    }
  };
  const auto load_next = [&]() {  // the scales of box bx in tile t
    const int m0 = a.m_base + (t / a.tiles_n) * (kOut * CG) + d.m_rank;
    if constexpr (MODE == kModeBackward) {
      const bool second = bx >= a.boxes_w;
      const int row = (second ? bx - a.boxes_w : bx) * kBoxK + (line & 63), col = m0 + 64 * (line >> 6);
      const uint8_t* base = static_cast<const uint8_t*>(second ? a.scales1 : a.scales0) + row * pitch;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
        next[k] = load_scales<FMT>(t < d.tile_end && row + 64 * k < a.nsum ? base + 64 * k * pitch : nullptr, col, cols, a.p.log2_block, VEC);
    } else {
      if (row_tile != t) {
        row_tile = t;
        const int row = MODE == kModeGated ? m0 + 16 * (line >> 5) + (line & 15) : m0 + line;
        const void* base = MODE == kModeGated && (line & 16) ? a.scales1 : a.scales0;
        row_scales = t < d.tile_end && row < a.nout ? static_cast<const uint8_t*>(base) + row * pitch : nullptr;
      }
      const int col = bx * kBoxK;
      if constexpr (kSteps == 2 && VEC) {
        load_scales_box<FMT>(row_scales, col, next);
      } else {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) next[k] = load_scales<FMT>(row_scales, col + 64 * k, cols, a.p.log2_block, VEC);
      }
    }
  };
  settle();
  load_next();
  while (t < d.tile_end) {
    Scales<FMT> now[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) now[k] = next[k];
    bx += kGroups;
    settle();
    load_next();  // of this group's next box, in flight during this one
    bool any = false;  // an E4M3 byte from 0x7F on
    if constexpr (FMT == QZ_NVFP4) {
#pragma unroll
      for (int k = 0; k < kSteps; ++k) any |= (((now[k].v[0] + 0x01010101u) | now[k].v[0]) & 0x80808080u) != 0u;
    }
    const bool ok = tc_wait(d.c_full + 8u * cs, cph, d.abort) && tc_wait(d.a_empty, aph ^ 1u, d.abort);
    const bool plain = __all_sync(kFull, ok && !any);  // (one vote a box, 1.5 per cent; a branch at each scale took 4)
    if (!plain && !__all_sync(kFull, ok)) break;
    const uint8_t* box = d.codes + cs * kBoxBytes + kLine * cl;
    uint4 codes[kSteps][2];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int c = 2 * (MODE == kModeBackward ? line >> 6 : k);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        codes[k][i] = *reinterpret_cast<const uint4*>(box + (MODE == kModeBackward ? 4096 * k : 0) + (((c + i) ^ cx) << 4));
    }
    const auto decode = [&](auto any) {
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const uint32_t dst = d.a_stage + k * (kTerms * kABytes) + 128u * line;
        decode32<FMT, decltype(any)::value>(codes[k][0], now[k], dst, x, 0);
        decode32<FMT, decltype(any)::value>(codes[k][1], now[k], dst, x, 1);
      }
    };
    if (FMT != QZ_NVFP4 || plain) decode(std::false_type{});
    else decode(std::true_type{});
    fence_proxy_async();  // the stores, before the tensor cores read them
    __syncwarp();
    if (d.lane == 0) {
      if constexpr (PAIR) arrive_remote(d.a_full);
      else arrive_local(d.a_full);
      arrive_local(d.c_empty + 8u * cs);
    }
    aph ^= 1u;
    cs += kGroups;
    if (cs >= a.code_slots) {
      cs -= a.code_slots;
      cph ^= 1u;
    }
  }
}

// ---- the kernel ---------------------------------------------------------------------------------
// PAIR = true: CG = 2, persistent; false: CG = 1, one tile per cluster of a.slices CTAs.
template <int FMT, int MODE, bool PAIR>
__global__ void __launch_bounds__(TcFormat<FMT>::kThreads, 1) product_tc_kernel(const __grid_constant__ TcArgs a) {
  constexpr int CG = PAIR ? 2 : 1;
  constexpr int kSteps = TcFormat<FMT>::kSteps, kBoxK = TcFormat<FMT>::kBoxK;
  constexpr uint32_t kBoxBytes = TcFormat<FMT>::kBoxBytes;
  constexpr int kTerms = TcFormat<FMT>::kTerms, kGroups = TcFormat<FMT>::kGroups, kEpiWarp0 = TcFormat<FMT>::kEpiWarp0;
  constexpr int kOut = MODE == kModeGated ? kBM / 2 : kBM;          // outputs per CTA
  extern __shared__ uint8_t tc_raw[];
  __shared__ __align__(8) uint64_t b_full[kMaxBStages], b_empty[kMaxBStages], a_full[kMaxGroups], a_empty[kMaxGroups];
  __shared__ __align__(8) uint64_t c_full[kMaxBoxes], c_empty[kMaxBoxes], d_full[2], d_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = !PAIR || rank == 0;
  const uint32_t base = (smem_addr(tc_raw) + 1023u) & ~1023u;
  const uint8_t* smem = tc_raw + (base - smem_addr(tc_raw));
  constexpr uint32_t kStageBytes = TcFormat<FMT>::kStageBytes;
  const int code_slots = a.code_slots, b_stages = a.b_stages;
  const uint32_t a_base = base, c_base = base + kGroups * kStageBytes, b_base = c_base + code_slots * kBoxBytes;
  const int b_rows = a.n / CG;                       // tokens that this CTA loads
  const uint32_t b_bytes = static_cast<uint32_t>(b_rows) * kBK * 2;  // of a step

  if (tid == 0) {
    for (int s = 0; s < kMaxBStages; ++s) {
      mbar_init(smem_addr(&b_full[s]), 1);
      mbar_init(smem_addr(&b_empty[s]), 1);
    }
    for (int s = 0; s < kMaxGroups; ++s) {
      mbar_init(smem_addr(&a_full[s]), 4 * CG);  // a group's warps, in both CTAs
      mbar_init(smem_addr(&a_empty[s]), 1);
    }
    for (int s = 0; s < kMaxBoxes; ++s) {
      mbar_init(smem_addr(&c_full[s]), 1);
      mbar_init(smem_addr(&c_empty[s]), 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&d_full[s]), 1);
      mbar_init(smem_addr(&d_empty[s]), TcFormat<FMT>::kEpiWarps * CG);
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
  const int bx_begin = PAIR ? 0 : static_cast<int>(rank) * a.slice_boxes;
  const int bx_end = PAIR ? a.boxes : min(a.boxes, bx_begin + a.slice_boxes);
  const auto tile_m0 = [&](int t) { return a.m_base + (t / a.tiles_n) * (kOut * CG) + (PAIR ? static_cast<int>(rank) * kOut : 0); };
  const auto tile_n0 = [&](int t) { return (t % a.tiles_n) * a.n; };

  if (warp == 0) {
    if (elect_one()) {
      int s = 0;
      uint32_t ph = 0, issued = 0;
      bool ok = true;
      for (int t = first; t < tile_end && ok; t += tile_step) {
        const int n0 = tile_n0(t) + (PAIR ? static_cast<int>(rank) * b_rows : 0);
        for (int bx = bx_begin; bx < bx_end; ++bx) {
          if (!(ok = tc_wait(smem_addr(&b_empty[s]), ph ^ 1u, &s_abort))) break;
          const uint32_t fb = PAIR ? map_to_rank(smem_addr(&b_full[s]), 0) : smem_addr(&b_full[s]);
          if (leader) mbar_expect_tx(smem_addr(&b_full[s]), kSteps * b_bytes * CG);
          const bool second = MODE == kModeBackward && bx >= a.boxes_w;
          const CUtensorMap* map = second ? &a.map_x1 : &a.map_x0;
          const int k0 = (second ? bx - a.boxes_w : bx) * kBoxK;
#pragma unroll
          for (int k = 0; k < kSteps; ++k) tma_load<CG>(b_base + (s * kSteps + k) * b_bytes, map, k0 + k * kBK, n0, fb);
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
    if (elect_one()) {
      int s = 0;
      uint32_t ph = 0, issued = 0;
      bool ok = true;
      for (int t = first; t < tile_end && ok; t += tile_step) {
        const int m0 = tile_m0(t);
        for (int bx = bx_begin; bx < bx_end; ++bx) {
          if (!(ok = tc_wait(smem_addr(&c_empty[s]), ph ^ 1u, &s_abort))) break;
          const uint32_t fb = smem_addr(&c_full[s]), dst = c_base + s * kBoxBytes;
          mbar_expect_tx(fb, kBoxBytes);
          if constexpr (MODE == kModeBackward) {
            // kBoxK weight rows x 128 columns (64 bytes)
            const bool second = bx >= a.boxes_w;
            tma_load<1>(dst, second ? &a.map_w1 : &a.map_w0, m0 / 2, (second ? bx - a.boxes_w : bx) * kBoxK, fb);
          } else if constexpr (MODE == kModeGated) {
            // 16 gate rows, the same 16 up rows, ...: kBoxK columns each
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              tma_load<1>(dst + q * (kBoxBytes / 4), &a.map_w0, bx * (kBoxK / 2), m0 + 16 * q, fb);
              tma_load<1>(dst + q * (kBoxBytes / 4) + kBoxBytes / 8, &a.map_w1, bx * (kBoxK / 2), m0 + 16 * q, fb);
            }
          } else {
            tma_load<1>(dst, &a.map_w0, bx * (kBoxK / 2), m0, fb);
          }
          ++issued;
          if (++s == code_slots) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (s_abort) let_land(c_full, s, ph, code_slots, issued);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader && elect_one()) {
      const uint32_t idesc = idesc_of(kBM * CG, a.n, MODE == kModeBackward);
      // K-major A: lines of 128 bytes, 32 bytes a 16-wide MMA; MN-major A: two slabs of 64 outputs,
      // 8 KiB apart, 16 lines (2 KiB) an MMA
      const uint64_t a_desc = MODE == kModeBackward ? desc_sw128(a_base, 8192u, 1024u) : desc_sw128(a_base, 16u, 1024u);
      constexpr uint32_t kAStep = MODE == kModeBackward ? 128u : 2u;
      const uint64_t b_desc = desc_sw128(b_base, 16u, 1024u);
      int bs = 0, g = 0, buf = 0;
      uint32_t bph = 0, aph = 0, dph = 3u;  // dph: parity bit per accumulator of the next "empty" wait
      bool ok = true;
      for (int t = first; t < tile_end && ok; t += tile_step) {
        for (int bx = bx_begin; bx < bx_end; ++bx) {
          // a sum starts: the tile's first box, or (backward) the second weight's
          const bool start = bx == bx_begin || (MODE == kModeBackward && bx == a.boxes_w);
          if (start) {
            if (bx != bx_begin) {
              tc_commit<CG>(smem_addr(&d_full[buf]));
              buf ^= 1;
            }
            if (!(ok = tc_wait(smem_addr(&d_empty[buf]), (dph >> buf) & 1u, &s_abort))) break;
            dph ^= 1u << buf;
          }
          if (!(ok = tc_wait(smem_addr(&b_full[bs]), bph, &s_abort) && tc_wait(smem_addr(&a_full[g]), aph, &s_abort))) break;
          tc_fence_after();
          const uint64_t ad = a_desc + g * (kStageBytes >> 4), bd = b_desc + bs * (kSteps * b_bytes >> 4);
          const uint32_t d = tmem + static_cast<uint32_t>(buf) * 256u;
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // kBoxK / 16 steps of kTerms MMAs
            const int j = i / kTerms, k = i % kTerms;
            tc_mma<CG>(d, ad + ((j >> 2) * kTerms + k) * (kABytes >> 4) + kAStep * (j & 3),
                       bd + (j >> 2) * (b_bytes >> 4) + 2u * (j & 3), idesc, !(start && i == 0));
          }
          tc_commit<CG>(smem_addr(&a_empty[g]));
          tc_commit<CG>(smem_addr(&b_empty[bs]));
          if (++g == kGroups) {
            g = 0;
            aph ^= 1u;
          }
          if (++bs == b_stages) {
            bs = 0;
            bph ^= 1u;
          }
        }
        if (!ok) break;
        if (bx_begin < bx_end) {
          tc_commit<CG>(smem_addr(&d_full[buf]));
          buf ^= 1;
        }
      }
      // every MMA issued has completed before tensor memory and shared memory are released (a slice without
      // boxes waits for nothing, so nothing may arrive there)
      if (bx_begin < bx_end) tc_commit<CG>(smem_addr(&drain));
    }
    __syncwarp();
  } else if (warp >= kDecWarp0 && warp < kEpiWarp0) {
    DecodeLoop d;
    d.group = (warp - kDecWarp0) >> 2;
    d.line = (tid - kDecWarp0 * 32) & 127;
    d.lane = lane;
    d.first = first;
    d.tile_end = tile_end;
    d.tile_step = tile_step;
    d.bx_begin = bx_begin;
    d.bx_end = bx_end;
    d.m_rank = PAIR ? static_cast<int>(rank) * kOut : 0;
    d.a_stage = a_base + d.group * kStageBytes;
    d.codes = smem + (c_base - base);
    d.c_full = smem_addr(&c_full[0]);
    d.c_empty = smem_addr(&c_empty[0]);
    d.a_empty = smem_addr(&a_empty[d.group]);
    d.a_full = PAIR ? map_to_rank(smem_addr(&a_full[d.group]), 0) : smem_addr(&a_full[d.group]);
    d.abort = &s_abort;
    if (a.scales_vec >= (MODE == kModeBackward || kSteps == 1 ? 1 : 2)) decode_boxes<FMT, MODE, PAIR, true>(a, d);
    else decode_boxes<FMT, MODE, PAIR, false>(a, d);
  } else if (PAIR && warp >= kEpiWarp0) {
    const int quarter = warp & 3;
    constexpr int kHalves = TcFormat<FMT>::kEpiWarps / 4;
    const int part = (warp - kEpiWarp0) >> 2;
    constexpr float kUnit = FMT == QZ_NVFP4 ? 256.0f : 1.0f;  // decoded NVFP4 weights are 2^-8 of their value
    const float f0 = sum_factor<FMT>(a.tscale0) * kUnit, f1 = a.p.n_weights == 2 ? sum_factor<FMT>(a.tscale1) * kUnit : 0.0f;
    const bool two = MODE == kModeBackward && a.p.n_weights == 2;
    const int c_begin = part * a.n / kHalves / 8 * 8, c_end = (part + 1) * a.n / kHalves / 8 * 8;
    const uint32_t ta = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
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
      const int end = min(c_end, static_cast<int>(min(a.p.tokens - n0, static_cast<int64_t>(a.n))));
      const StorePlan plan = store_plan<MODE>(a, m0, quarter, lane, n0 + c_begin, n0 + c_end);
      // the next eight columns are on their way while these are worked on
      float v[8], w[8];
      const auto fetch = [&](int c, float (&x)[8], float (&y)[8]) {
        tmem_load8(ta + 256u * buf + c, x);
        if (two) tmem_load8(ta + 256u * (buf ^ 1) + c, y);
      };
      if (ok && c_begin < end) fetch(c_begin, v, w);
      for (int c = c_begin; c < end; c += 8) {
        float r[8];
        if (ok) {
          tmem_wait8(v);
          if (two) {
            tmem_wait8(w);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = __fmaf_rn(w[i], f1, v[i] * f0);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = MODE == kModeGated ? v[i] : v[i] * f0;
          }
          if (c + 8 < end) fetch(c + 8, v, w);
        } else {  // a wait gave up: NaN instead of a wrong result
#pragma unroll
          for (int i = 0; i < 8; ++i) r[i] = __uint_as_float(0x7fc00000u);
        }
        store8<MODE>(a, plan, r, f0, f1, lane, n0 + c);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        for (int k = 0; k < (two ? 2 : 1); ++k) {
          const uint32_t bar = smem_addr(&d_empty[buf ^ k]);
          arrive_remote(map_to_rank(bar, 0));
        }
      }
      if (!two) buf ^= 1;
    }
  }

  // every MMA has completed (or its wait has given up) before shared and tensor memory go
  __syncthreads();
  const bool done = __all_sync(kFull, bx_begin >= bx_end || tc_wait(smem_addr(&drain), 0u, &s_abort)) && !s_abort;
  tc_fence_after();
  if constexpr (!PAIR) {
    // ---- the slices of the tile: partial sums to the CTA that finishes their columns ----------
    const int slices = a.slices, cols = a.n / slices;  // columns this CTA finishes
    const int quarter = warp & 3, part = warp >> 2;    // the warps of a quarter share the columns
    constexpr int kStride = 8 * (TcFormat<FMT>::kThreads / 128);
    const uint32_t ta = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    constexpr float kUnit = FMT == QZ_NVFP4 ? 256.0f : 1.0f;
    const float f0 = sum_factor<FMT>(a.tscale0) * kUnit, f1 = a.p.n_weights == 2 ? sum_factor<FMT>(a.tscale1) * kUnit : 0.0f;
    const bool has0 = MODE == kModeBackward ? bx_begin < min(bx_end, a.boxes_w) : bx_begin < bx_end;
    const bool has1 = MODE == kModeBackward && max(bx_begin, a.boxes_w) < bx_end;
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
      for (int c = 8 * part; c < a.n; c += kStride) {
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
    const int c_begin = static_cast<int>(rank) * cols;
    const StorePlan plan = store_plan<MODE>(a, m0, quarter, lane, n0 + c_begin, n0 + c_begin + cols);
    for (int c = 8 * part; c < cols && n0 + c_begin + c < a.p.tokens; c += kStride) {
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
      store8<MODE>(a, plan, v, f0, f1, lane, n0 + c_begin + c);
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
inline bool encode(CUtensorMap* m, int swizzle, const void* base, int64_t inner, int64_t outer, int64_t pitch, int box_in, int box_out) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_in), static_cast<cuuint32_t>(box_out)}, es[2] = {1, 1};
  return enc(m, swizzle < 128 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
             box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle == 32 ? CU_TENSOR_MAP_SWIZZLE_32B : swizzle == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
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
  cfg.blockDim = dim3(TcFormat<FMT>::kThreads);
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

template <int FMT>
qz_status launch_plan(TcArgs& a, const Plan& plan, cudaStream_t s) {
  const ProductArgs& p = a.p;
  const bool back = p.mode == kModeBackward;
  a.n = plan.n;
  a.tiles_n = plan.tiles_n;
  a.tiles = plan.tiles;
  a.m_base = static_cast<int>(plan.m_base);
  a.slices = plan.slices;
  a.slice_boxes = plan.slice_boxes;
  constexpr int kBoxK = TcFormat<FMT>::kBoxK, kGroups = TcFormat<FMT>::kGroups;
  constexpr uint32_t kBoxBytes = TcFormat<FMT>::kBoxBytes;
  const int b_rows = plan.pair ? plan.n / 2 : plan.n;
  // two rounds of code boxes, or one where that leaves the tokens fewer than three stages
  const uint32_t stage_b = static_cast<uint32_t>(b_rows) * kBoxK * 2;
  a.code_slots = kRingRoom<FMT> < 2 * kGroups * kBoxBytes + 3 * stage_b ? kGroups : 2 * kGroups;
  a.b_stages = static_cast<int>(std::min<uint32_t>(kMaxBStages, (kRingRoom<FMT> - a.code_slots * kBoxBytes) / stage_b));
  const int code_line = back ? 64 : kBoxK / 2;  // bytes, and the swizzle
  const int code_rows = back ? kBoxK : p.mode == kModeGated ? 16 : 128;
  bool ok = encode(&a.map_x0, 128, p.x0, a.nsum, p.tokens, p.ld_x * 2, kBK, b_rows) &&
            encode(&a.map_w0, code_line, p.w0.codes, p.cols / 2, p.rows, p.cols / 2, code_line, code_rows);
  if (p.n_weights == 2) ok = ok && encode(&a.map_w1, code_line, p.w1.codes, p.cols / 2, p.rows, p.cols / 2, code_line, code_rows);
  if (p.n_weights == 2 && back) ok = ok && encode(&a.map_x1, 128, p.x1, a.nsum, p.tokens, p.ld_x * 2, kBK, b_rows);
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
  a.boxes_w = boxes_of(p.format, a.nsum);
  a.boxes = back ? a.boxes_w * p.n_weights : a.boxes_w;
  const auto aligned_scales = [&](uintptr_t n) { return reinterpret_cast<uintptr_t>(a.scales0) % n == 0 && reinterpret_cast<uintptr_t>(a.scales1) % n == 0; };
  const int unit = p.format == QZ_MXFP4 ? 2 : 4;  // bytes of scales per 64 columns
  a.scales_vec = p.cols % 128 == 0 && aligned_scales(2 * unit) ? 2 : p.cols % 64 == 0 && aligned_scales(unit) ? 1 : 0;
  Plan plans[2];
  const int launches = plan_of(p, plans);
  if (launches == 0) return QZ_ERR_UNSUPPORTED;
  for (int i = 0; i < launches; ++i) {
    const qz_status st = launch_plan<FMT>(a, plans[i], s);
    if (st != QZ_OK) return st;
  }
  return QZ_OK;
}

}  // namespace
}  // namespace qz
