// qz_product_few.cuh -- products of a few tokens (decoding, small batches) with 4-bit weights
// (included once per weight format):
//   y[t][r] = sum_c W[r][c] x[t][c]        (one weight, or gate and up with the activation)
//
// Every weight is used once per token, so the weights' 4 bits (and scales) are the traffic and HBM
// the bound; what has to fit beside the traffic is the decoding: at HBM speed an SM has about 22
// issue slots for 8 weights a lane, one mma.sync m16n8k16 (16 weight rows, 8 tokens).
//   - E2M1 pairs become f16 by one conversion each, INT4 nibbles by the bits of f16 1024 + n.
//   - f16 holds E2M1 times an E4M3 block scale exactly (6 significant bits, 2^-10 .. 2688), so
//     NVFP4 weights are scaled before the product; E8M0 and fp32 scales take the fp32 sum of their
//     block or group (one FMA per output).
//   - The activations are f16 too: token t's values times a power of two 2^p that brings its
//     largest finite magnitude into [2^14, 2^15), and the sum is multiplied by 2^-p.  f16 holds the 8
//     bits of every value down to 2^-31 of that magnitude (2^-17, in units of 2^-24).  Where a token
//     spans more, or p is negative (sums times the smallest scales would leave fp32), all activations
//     of the call stay bf16 and the weights are turned into bf16, exactly: see `wide`.  (Logits below:
//     38 us, such activations 60.)
//
// A tile is 16 outputs (gated: 16 of gate and of up).  ks of a CTA's warps share a tile, each with a
// contiguous part of the sum, and join their partial sums in shared memory in warp order; CTAs
// (one per SM) are persistent over the tiles.  A warp streams 256 columns of its 16 rows a step
// (whole 128-byte lines) through a ring of its own by TMA and runs on into the next tile, so the
// copies never pause; a step's scales are loaded into registers one step ahead.
//
// Measured, on the GPU alone: 32768 x 8192 MXFP4, 4 tokens: 38 us, 3.8 TB/s (floor 21); 16384 x 4096
// NVFP4 gate and up, 1 token: 21 us, 3.6 TB/s (floor 11); 4096 x 4096 NVFP4, 1 token: 5.7 us (floor 1.4).
// No pipe is full: some 20 instructions per mma.sync, issued in 0.5 of the cycles by four warps a
// scheduler, wait for one another, and the start stages all activations in every CTA (0.48 us a token
// and 4096 columns) before the first product.  More warps leave each too few registers (31 -> 36 us
// for the gated token).
#pragma once

#include <cuda.h>  // CUtensorMap and its enumerators (types only; the encoder is looked up)
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "qz_device.cuh"
#include "qz_internal.h"
#include "qz_pipe.cuh"
#include "qz_product.h"
#include "qz_weight.cuh"

namespace qz {
namespace {

struct FewArgs {
  CUtensorMap map_w0, map_w1;  // codes [rows][cols / 2] bytes, box 128 x 16
  ProductArgs p;
  int tiles, ks, groups, steps;  // warps per tile, tiles a CTA works on at once, 256-wide steps of a row
  int depth;                     // ring slots
  int x_chunks;                  // 32-wide chunks of the activations' copy (whole steps)
  int64_t scale_pitch;           // bytes per weight row
};

constexpr uint64_t kFewWaitNs = 1000000000ull;  // 1 s: far beyond any copy's latency
// Bounded wait for a copy; after one has given up nothing is waited for, and the outputs are NaN.
__device__ __forceinline__ void few_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return;
    if (globaltimer_ns() - t0 > kFewWaitNs) *abort = 1;
  }
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ bool few_elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mulh(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// a word's 8 weights as four f16 pairs: E2M1 values (2 q, 2 q + 1), or INT4 integers (q, q + 4)
template <int FMT>
__device__ __forceinline__ void decode_word(uint32_t w, uint32_t (&v)[4]) {
  if constexpr (FMT == QZ_INT4) {
    // pairs (q, q + 4): f16 1024 + (n ^ 8), less 1032, is the two's complement value, exactly
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      const uint32_t h = q == 0 ? w : w >> 8;
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(v[q]) : "r"((h & 0x000F000Fu) ^ 0x64086408u), "r"(0x64086408u));
      // four bits further up: 1024 + 16 (n ^ 8), times 1 / 16, less 72
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(v[q + 1]) : "r"((h & 0x00F000F0u) ^ 0x64806480u), "r"(0x2C002C00u), "r"(0xD480D480u));
    }
  } else {
    asm("{\n\t.reg .b8 b<4>;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
        : "r"(w));
  }
}
__device__ __forceinline__ uint32_t min_abs_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b32 x, y;\n\tabs.f16x2 x, %1;\n\tabs.f16x2 y, %2;\n\tmin.f16x2 %0, x, y;\n\t}" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// an f16 pair of values of at most 8 significant bits as bf16, exactly
__device__ __forceinline__ uint32_t to_bf16(uint32_t h) {
  float lo, hi;
  f16x2_to_f32(h, lo, hi);
  return bf16x2_bits(lo, hi);
}
__device__ __forceinline__ float pow2(int e) {  // 2^e as fp32, e in [-149, 127]
  return e >= -126 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : __uint_as_float(1u << (e + 149));
}

// The scales of a weight row's 256 columns of a step, in the words they are stored in: eight E8M0
// bytes, sixteen E4M3 bytes, or eight, four or two fp32 (groups of 32, 64, 128: LOG = 5, 6, 7).
template <int FMT, int LOG>
struct StepScales {
  static constexpr int kWords = FMT == QZ_MXFP4 ? 2 : FMT == QZ_NVFP4 ? 4 : 256 >> LOG;
  uint32_t v[kWords];
};
// p: the row's scales
template <int FMT, int LOG>
__device__ __forceinline__ void load_step_scales(StepScales<FMT, LOG>& s, const uint8_t* p, int step) {
  constexpr int kWords = StepScales<FMT, LOG>::kWords;
  p += 4 * kWords * step;
  if constexpr (kWords == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    s.v[0] = v.x;
    s.v[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
      s.v[i] = v.x;
      s.v[i + 1] = v.y;
      s.v[i + 2] = v.z;
      s.v[i + 3] = v.w;
    }
  }
}

// One step's scales of weight rows g and g + 8 as this lane loads them ahead.  RAGGED: rows that are
// not whole steps have their scales at any alignment, so the quad's lanes share the narrow loads (past
// the row's end: a scale of 1 or 0, the codes there are 0) and exchange the words when they are used.
template <int FMT, int LOG, bool RAGGED>
struct AheadScales {
  StepScales<FMT, LOG> row[2];
  __device__ __forceinline__ void load(const uint8_t* const (&p)[2], int step, int, int) {
#pragma unroll
    for (int h = 0; h < 2; ++h) load_step_scales<FMT, LOG>(row[h], p[h], step);
  }
  __device__ __forceinline__ void words(StepScales<FMT, LOG> (&s)[2], int) const {
    s[0] = row[0];
    s[1] = row[1];
  }
};
template <int FMT, int LOG>
struct AheadScales<FMT, LOG, true> {
  static constexpr int kWords = StepScales<FMT, LOG>::kWords;
  uint32_t raw[FMT == QZ_INT4 ? 2 * kWords : 4];
  // blocks: scales of a row
  __device__ __forceinline__ void load(const uint8_t* const (&p)[2], int step, int t, int blocks) {
    if constexpr (FMT == QZ_MXFP4) {  // lane t: word t % 2 of row t / 2
      const uint8_t* q = t < 2 ? p[0] : p[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = 8 * step + 4 * (t & 1) + i;
        raw[i] = b < blocks ? __ldg(q + b) : 127u;
      }
    } else if constexpr (FMT == QZ_NVFP4) {  // lane t: word t of both rows; an even number of blocks
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = 16 * step + 4 * t + 2 * (i & 1);
        raw[i] = b < blocks ? __ldg(reinterpret_cast<const uint16_t*>(p[i >> 1] + b)) : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2 * kWords; ++i) {
        const int b = kWords * step + i % kWords;
        raw[i] = b < blocks ? __ldg(reinterpret_cast<const uint32_t*>(p[i / kWords]) + b) : 0u;
      }
    }
  }
  __device__ __forceinline__ void words(StepScales<FMT, LOG> (&s)[2], int lane) const {
    if constexpr (FMT == QZ_MXFP4) {
      const uint32_t w = __byte_perm(__byte_perm(raw[0], raw[1], 0x0040), __byte_perm(raw[2], raw[3], 0x0040), 0x5410);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i >> 1].v[i & 1] = __shfl_sync(kFull, w, (lane & 28) | i);
    } else if constexpr (FMT == QZ_NVFP4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w = raw[2 * h] | raw[2 * h + 1] << 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) s[h].v[i] = __shfl_sync(kFull, w, (lane & 28) | i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2 * kWords; ++i) s[i / kWords].v[i % kWords] = raw[i];
    }
  }
};

template <int FMT, int LOG, int NT, bool GATED, bool RAGGED>
__global__ void __launch_bounds__(32 * kFewWarps, 1) product_few_kernel(const __grid_constant__ FewArgs a) {
  extern __shared__ uint8_t few_raw[];
  __shared__ __align__(8) uint64_t s_full[kFewWarps][kMaxDepth];
  __shared__ uint32_t s_amax[8 * NT];
  __shared__ volatile int s_abort;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const ProductArgs& p = a.p;
  const int depth = a.depth;
  uint8_t* few_smem = few_raw + ((1024u - (smem_addr(few_raw) & 1023u)) & 1023u);  // swizzled boxes: 1 KiB
  const uint8_t* mine_ring = few_smem + warp * (depth * kSlot);
  const uint32_t ring = smem_addr(mine_ring);
  float* join = reinterpret_cast<float*>(few_smem + kFewWarps * depth * kSlot);
  uint8_t* xs = few_smem + kFewWarps * (depth * kSlot + kJoin * 4);
  // ks warps share a tile; gated: ks more have the same outputs of the second weight
  constexpr int kWeights = GATED ? 2 : 1;
  const int ks = a.ks, team = ks * kWeights, group = warp / team, member = warp % team, part = member % ks;
  const bool second = GATED && member >= ks;
  const bool busy = group < a.groups;
  const int tile0 = busy ? blockIdx.x * a.groups + group : a.tiles, tile_step = gridDim.x * a.groups;
  const int s_begin = part * a.steps / ks, s_end = (part + 1) * a.steps / ks;
  const int rows = static_cast<int>(p.rows), tokens = static_cast<int>(p.tokens);
  const uint32_t full = smem_addr(&s_full[warp][0]);

  if (lane == 0) {
    for (int i = 0; i < kMaxDepth; ++i) mbar_init(full + 8u * i, 1);
    mbar_init_fence();
  }
  if (threadIdx.x == 0) s_abort = 0;
  if (threadIdx.x < 8 * NT) s_amax[threadIdx.x] = 0u;
  __syncthreads();

  // ---- the copies, depth - 1 steps ahead of their use ----
  int ptile = tile0, ps = s_begin, pi = 0;
  const auto issue = [&]() {
    if (ptile < a.tiles) {
      if (few_elect()) {
        const uint32_t bar = full + 8u * pi, dst = ring + pi * kSlot;
        mbar_expect_tx(bar, kSlot);
        tma_box(dst, second ? &a.map_w1 : &a.map_w0, ps * 128, ptile * 16, bar);
      }
      __syncwarp();
      if (++ps == s_end) {
        ps = s_begin;
        ptile += tile_step;
      }
      if (++pi == depth) pi = 0;
    }
  };
  for (int i = 0; i < depth - 1; ++i) issue();

  // ---- the activations, times 2^p, as f16 (wide: as they are): [32-wide chunk][token][32], zero past the columns ----
  // wide: f16 does not hold them.  Every CTA sees the same activations and so decides the same.
  bool wide;
  {
    constexpr int kHeld = 8, kAll = 32 * kFewWarps;
    // a round holds up to eight pieces of 8 values a thread, each of them kAll consecutive pieces of one token
    const int per_token = a.x_chunks * 4, per_row = static_cast<int>(p.cols / 8), blocks = (per_token + kAll - 1) / kAll, n = blocks * tokens;
    uint4 v[kHeld];
    // the round's blocks one after the other: (tok, blk), uniform over the CTA
    const auto each = [&](int base_tok, int base_blk, auto&& f) {
      int tok = base_tok, blk = base_blk;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        if (tok >= tokens) break;
        f(i, tok, blk * kAll + static_cast<int>(threadIdx.x));
        if (++blk == blocks) {
          blk = 0;
          ++tok;
        }
      }
    };
    const auto load = [&](int i, int tok, int c) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (c < per_row) v[i] = __ldg(reinterpret_cast<const uint4*>(p.x0 + tok * p.ld_x) + c);
    };
    const auto magnitude = [&](int i, int tok, int) {
      const uint32_t w[4] = {v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu, v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu};
      const uint32_t m2 = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
      uint32_t m = max(m2 & 0xffffu, m2 >> 16);
      if (m >= 0x7f80u) {  // the largest finite magnitude
        m = 0u;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t lo = w[q] & 0xffffu, hi = w[q] >> 16;
          m = max(m, max(hi < 0x7f80u ? hi : 0u, lo < 0x7f80u ? lo : 0u));
        }
      }
      m = __reduce_max_sync(kFull, m);
      if (lane == 0) atomicMax(&s_amax[tok], m << 16);
    };
    const auto put = [&](int tok, int c, uint32_t (&o)[4]) {
      if constexpr (FMT == QZ_INT4) {  // values 0 .. 7 in the order of the weights' pairs
        const uint32_t e[4] = {o[0], o[1], o[2], o[3]};
        o[0] = __byte_perm(e[0], e[2], 0x5410);
        o[1] = __byte_perm(e[0], e[2], 0x7632);
        o[2] = __byte_perm(e[1], e[3], 0x5410);
        o[3] = __byte_perm(e[1], e[3], 0x7632);
      }
      if (c < per_token)
        *reinterpret_cast<uint4*>(xs + ((c >> 2) * tokens + tok) * 64 + (c & 3) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    };
    bool beyond = false;  // this thread has met a value that f16 does not hold
    const auto convert = [&](int i, int tok, int c) {
      const uint32_t m = s_amax[tok];
      // 2^p: 14 less the exponent of the largest magnitude, 120 at most
      const float f = pow2(m == 0u ? 0 : min(120, 14 + 127 - static_cast<int>(m >> 23)));
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[q]) : "f"(__uint_as_float(w[q] & 0xffff0000u) * f), "f"(__uint_as_float(w[q] << 16) * f));
      // The largest has exponent field E, p = 141 - E (120 at most: then f16 holds every bf16 value).
      // Values but 0 with a field below E - 31 are too small (subnormals have the spacing of field 1);
      // they are among those that came out below 2^-16.
      const uint32_t small = min_abs_f16x2(min_abs_f16x2(o[0], o[1]), min_abs_f16x2(o[2], o[3]));
      if ((small & 0xff00u) == 0u || (small & 0xff000000u) == 0u) {
        const int E = static_cast<int>(m >> 23), least = E > 32 ? (E - 31) << 7 : 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int lo = w[q] & 0x7fffu, hi = (w[q] >> 16) & 0x7fffu;
          beyond |= (lo != 0 && lo < least) || (hi != 0 && hi < least);
        }
      }
      if constexpr (FMT != QZ_NVFP4) beyond |= m >= 142u << 23;
      put(tok, c, o);
    };
    for (int base = 0, tok = 0, blk = 0; base < n; base += kHeld) {
      each(tok, blk, load);
      each(tok, blk, magnitude);
      tok = (base + kHeld) / blocks;
      blk = (base + kHeld) - tok * blocks;
    }
    __syncthreads();
    for (int base = 0, tok = 0, blk = 0; base < n; base += kHeld) {
      if (n > kHeld) each(tok, blk, load);  // else still in registers
      each(tok, blk, convert);
      tok = (base + kHeld) / blocks;
      blk = (base + kHeld) - tok * blocks;
    }
    wide = __syncthreads_or(beyond);
    if (wide) {  // again, in little code
#pragma unroll 1
      for (int i = threadIdx.x; i < per_token * tokens; i += kAll) {
        const int tok = i / per_token, c = i - tok * per_token;
        const uint4 w = c < per_row ? __ldg(reinterpret_cast<const uint4*>(p.x0 + tok * p.ld_x) + c) : make_uint4(0u, 0u, 0u, 0u);
        uint32_t o[4] = {w.x, w.y, w.z, w.w};
        put(tok, c, o);
      }
      __syncthreads();
    }
  }
  if (!busy) return;  // (fewer tiles than warps to share them; no barrier of the whole CTA follows)
  int ci = 0;
  uint32_t cph = 0;
  // The tiles, in code of its own for wide activations (tests inside one loop cost the other 1.5 us of 37).
  const auto run = [&](auto kind) {
    constexpr bool kWide = decltype(kind)::value;
    // this lane's B operand: token 8 nt + g (the last again past the end: its columns are not stored)
    const uint8_t* xa[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xa[nt] = xs + min(8 * nt + g, tokens - 1) * 64 + 16 * t;
    const uint32_t x_chunk = 64u * tokens;

    // 2^-p of a token, and the unit of the sums on bf16 operands
    const auto token_down = [&](int tok) {
      const uint32_t m = s_amax[min(tok, tokens - 1)];
      return pow2(m == 0u ? 0 : -min(120, 14 + 127 - static_cast<int>(m >> 23)));
    };
    constexpr float kWideUnit = FMT == QZ_NVFP4 ? 0x1p12f : FMT == QZ_INT4 ? 0x1p11f : 1.0f;

    // scales of rows g and g + 8, one step ahead
    AheadScales<FMT, LOG, RAGGED> next;
    const int row_blocks = static_cast<int>(p.cols >> p.log2_block);
    int ntile = tile0, ns = s_begin;
    const uint8_t* pr[2];
    const auto point = [&]() {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        pr[h] = static_cast<const uint8_t*>(second ? p.w1.scales : p.w0.scales) + min(ntile * 16 + g + 8 * h, rows - 1) * a.scale_pitch;
    };
    const auto load_next = [&]() {  // (past the last tile: its last row's again)
      next.load(pr, ns, t, row_blocks);
      if (++ns == s_end) {
        ns = s_begin;
        ntile += tile_step;
        point();
      }
    };
    point();
    load_next();

    const uint32_t word = 128u * g + 4u * t;  // word t of chunk c of row g: 16 (c ^ g) further (128-byte swizzle)
    for (int tile = tile0; tile < a.tiles; tile += tile_step) {
      float z[NT][4] = {};
      bool exact = false;  // not wide: this tile's sums have gone over to bf16 operands
#pragma unroll 1
      for (int s = s_begin; s < s_end; ++s) {
        StepScales<FMT, LOG> now[2];
        next.words(now, lane);
        load_next();
        few_wait(full + 8u * ci, cph, &s_abort);
        __syncwarp();  // the slot before is read by every lane
        issue();
        const uint8_t* slot = mine_ring + ci * kSlot + word;
        if (++ci == depth) {
          ci = 0;
          cph ^= 1u;
        }
        bool odd = false;
        if constexpr (FMT == QZ_NVFP4) {
          // this lane's block of chunk c is 2 c + t / 2: eight E4M3 bytes, then f16 (chunks 2 i, 2 i + 1)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sel = t < 2 ? 0x6420u : 0x7531u;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t b;
              asm("prmt.b32 %0, %1, %2, %3;" : "=r"(b) : "r"(now[h].v[2 * i]), "r"(now[h].v[2 * i + 1]), "r"(sel));
              asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
                  : "=r"(now[h].v[2 * i]), "=r"(now[h].v[2 * i + 1])
                  : "r"(b));
            }
          }
        } else if (!kWide) {
          // E8M0 bytes of 0 are not what an exponent field of 0 means.  Bytes above 191 and fp32 scales above
          // 2^73 could take the sum of a block times 2^p out of fp32: from there on this warp's part of the
          // tile is summed as in `wide` (a unit of its own for the large sums would lose the small ones).
          bool high = false;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < StepScales<FMT, LOG>::kWords; ++i) {
              if constexpr (FMT == QZ_MXFP4) {
                const uint32_t e = now[h].v[i];
                odd |= ((e - 0x01010101u) & ~e & 0x80808080u) != 0u;  // a byte 0 (and some bytes 1 above one)
                high |= ((e & 0x80808080u) & ((e << 1) & 0x80808080u)) != 0u;  // a byte above 191
              } else {
                high |= fabsf(__uint_as_float(now[h].v[i])) > 0x1p73f;
              }
            }
          if (!exact && __any_sync(kFull, high)) {
            exact = true;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) z[nt][i] *= token_down(8 * nt + 2 * t + (i & 1)) * (1.0f / kWideUnit);
          }
          odd = __any_sync(kFull, odd);
        }
        const uint32_t x0 = static_cast<uint32_t>(s) * 8u * x_chunk;
        [[maybe_unused]] float acc[FMT == QZ_NVFP4 ? 1 : NT][4];  // the sum of a block or group, before its scale
        [[maybe_unused]] constexpr int kPer = FMT == QZ_INT4 ? 1 << (LOG - 5) : 1;  // chunks of it
        const auto chunk = [&](int c, bool rare) {  // chunk c: 32 columns, lane t its word t
          uint4 xv[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) xv[nt] = *reinterpret_cast<const uint4*>(xa[nt] + x0 + c * x_chunk);
          uint32_t v[2][4];
          [[maybe_unused]] float f[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            decode_word<FMT>(*reinterpret_cast<const uint32_t*>(slot + 1024 * h + ((c ^ g) << 4)), v[h]);
            if constexpr (FMT == QZ_NVFP4) {
              const uint32_t both = __byte_perm(now[h].v[c >> 1], 0, (c & 1) ? 0x3232 : 0x1010);
#pragma unroll
              for (int q = 0; q < 4; ++q) v[h][q] = mulh(v[h][q], both);
            } else if constexpr (FMT == QZ_MXFP4) {
              const uint32_t E = now[h].v[c >> 2];
              f[h] = __uint_as_float(((c & 3) == 3 ? E >> 1 : E << (23 - 8 * (c & 3))) & 0x7f800000u);
              if (rare) f[h] = pow2(static_cast<int>((E >> (8 * (c & 3))) & 255u) - 127);
            } else {
              f[h] = __uint_as_float(now[h].v[c / kPer]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (FMT == QZ_NVFP4) {
              mma(z[nt], v[0][0], v[1][0], v[0][1], v[1][1], xv[nt].x, xv[nt].y);
              mma(z[nt], v[0][2], v[1][2], v[0][3], v[1][3], xv[nt].z, xv[nt].w);
            } else {  // the block's scale takes its sum
              if (c % kPer == 0) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
              mma(acc[nt], v[0][0], v[1][0], v[0][1], v[1][1], xv[nt].x, xv[nt].y);
              mma(acc[nt], v[0][2], v[1][2], v[0][3], v[1][3], xv[nt].z, xv[nt].w);
              if (c % kPer == kPer - 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[nt][i] = __fmaf_rn(f[i >> 1], acc[nt][i], z[nt][i]);
              }
            }
          }
        };
        // The same on bf16 operands, for any activations and scales.  MXFP4 and NVFP4 weights take their
        // scales before the product (6 significant bits); NVFP4 weights are 2^-12 and INT4 integers 2^-11
        // of their value, so that no product leaves fp32 before the tensor scale or the group's scale.
        const auto wide_chunk = [&](int c) {
          uint4 xv[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            xv[nt] = *reinterpret_cast<const uint4*>(xa[nt] + x0 + c * x_chunk);
            if constexpr (!kWide) {  // back from f16: the activations as they were
              const float d = token_down(8 * nt + g);
              for (uint32_t* q : {&xv[nt].x, &xv[nt].y, &xv[nt].z, &xv[nt].w}) {
                float lo, hi;
                f16x2_to_f32(*q, lo, hi);
                *q = bf16x2_bits(lo * d, hi * d);
              }
            }
          }
          uint32_t v[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            decode_word<FMT>(*reinterpret_cast<const uint32_t*>(slot + 1024 * h + ((c ^ g) << 4)), v[h]);
            uint32_t k = 0x10001000u;  // 2^-11
            if constexpr (FMT == QZ_NVFP4) {
              k = mulh(__byte_perm(now[h].v[c >> 1], 0, (c & 1) ? 0x3232 : 0x1010), 0x0C000C00u);
            } else if constexpr (FMT == QZ_MXFP4) {
              const uint32_t b = (now[h].v[c >> 2] >> (8 * (c & 3))) & 255u;
              k = (b == 255u ? 0x7FC0u : b == 0u ? 0x0040u : b << 7) * 0x00010001u;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) v[h][q] = FMT == QZ_MXFP4 ? mul_bf16x2(to_bf16(v[h][q]), k) : to_bf16(mulh(v[h][q], k));
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (FMT == QZ_INT4) {
              if (c % kPer == 0) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
              mma_bf16(acc[nt], v[0][0], v[1][0], v[0][1], v[1][1], xv[nt].x, xv[nt].y);
              mma_bf16(acc[nt], v[0][2], v[1][2], v[0][3], v[1][3], xv[nt].z, xv[nt].w);
              if (c % kPer == kPer - 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[nt][i] = __fmaf_rn(__uint_as_float(now[i >> 1].v[c / kPer]), acc[nt][i], z[nt][i]);
              }
            } else {
              mma_bf16(z[nt], v[0][0], v[1][0], v[0][1], v[1][1], xv[nt].x, xv[nt].y);
              mma_bf16(z[nt], v[0][2], v[1][2], v[0][3], v[1][3], xv[nt].z, xv[nt].w);
            }
          }
        };
        // (loops of their own: tests inside one cost its chunks their overlap)
        if (kWide || (FMT != QZ_NVFP4 && exact)) {
#pragma unroll
          for (int c = 0; c < 8; ++c) wide_chunk(c);
        } else if (FMT != QZ_MXFP4 || !odd) {
#pragma unroll
          for (int c = 0; c < 8; ++c) chunk(c, false);
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) chunk(c, true);
        }
      }
      // ---- join the parts, eight tokens at a time, and store ----
      [[maybe_unused]] const float f0 = sum_factor<FMT>(p.w0.tscale), f1 = GATED ? sum_factor<FMT>(p.w1.tscale) : 0.0f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float* mine = join + warp * kJoin;
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // tokens 8 nt + 2 t and + 1: 2^-p of each
          const float down = kWide || exact ? kWideUnit : token_down(8 * nt + 2 * t + i);
#pragma unroll
          for (int h = 0; h < 2; ++h) mine[(2 * t + i) * kTokenStride + g + 8 * h] = z[nt][2 * h + i] * down;
        }
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * team) : "memory");
        const float* from = join + group * team * kJoin;
        const int count = 16 * min(8, tokens - 8 * nt);
        for (int e = member * 32 + lane; e < count; e += 32 * team) {
          const int row = tile * 16 + (e & 15), tok = 8 * nt + (e >> 4);
          float sum[kWeights];
#pragma unroll
          for (int m = 0; m < kWeights; ++m) {
            const float* q = from + m * ks * kJoin + (e >> 4) * kTokenStride + (e & 15);
            sum[m] = q[0];
            for (int w = 1; w < ks; ++w) sum[m] += q[w * kJoin];
          }
          if (row >= rows) continue;
          const int64_t o = static_cast<int64_t>(tok) * p.ld_y + row;
          const float v = s_abort ? __uint_as_float(0x7fc00000u) : sum[0] * f0;
          if constexpr (GATED) {
            const float u = sum[kWeights - 1] * f1;
            static_cast<uint16_t*>(p.y)[o] = bf16_bits((p.act == QZ_ACT_SILU ? act_value<QZ_ACT_SILU>(v) : act_value<QZ_ACT_GELU_TANH>(v)) * u);
            if (p.g_out) {
              const int64_t q = static_cast<int64_t>(tok) * p.ld_gu + row;
              p.g_out[q] = bf16_bits(v);
              p.u_out[q] = bf16_bits(u);
            }
          } else if (p.out_f32) {
            static_cast<float*>(p.y)[o] = v;
          } else {
            static_cast<uint16_t*>(p.y)[o] = bf16_bits(v);
          }
        }
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * team) : "memory");
      }
    }
  };
  if (!wide) run(std::false_type{});
  else run(std::true_type{});
  // (every copy issued has been waited for by its step; after a wait that gave up they get a second more)
  if (s_abort)
    for (int i = 0; i < depth; ++i) {
      const uint64_t t0 = globaltimer_ns();
      const uint32_t ph = i < ci ? cph : cph ^ 1u;
      while (!mbar_try_wait(full + 8u * i, ph) && globaltimer_ns() - t0 < kFewWaitNs / 8) {
      }
    }
}

template <int FMT, int LOG, int NT, bool GATED, bool RAGGED>
qz_status run_few(const FewArgs& a, cudaStream_t s) {
  const void* k = reinterpret_cast<const void*>(&product_few_kernel<FMT, LOG, NT, GATED, RAGGED>);
  if (!set_dyn_smem(k, static_cast<int>(kFewSmem))) return QZ_ERR_CUDA;
  const int grid = std::min((a.tiles + a.groups - 1) / a.groups, sm_count());
  const size_t smem = few_fixed(a.depth) + static_cast<size_t>(a.p.tokens * few_steps(a.p) * 512);
  product_few_kernel<FMT, LOG, NT, GATED, RAGGED><<<grid, 32 * kFewWarps, smem, s>>>(a);
  return launch_status();
}
template <int FMT, int LOG, bool GATED, bool RAGGED>
qz_status run_few_nt(FewArgs& a, cudaStream_t s) {
  const ProductArgs& p = a.p;
  const int nt = static_cast<int>((p.tokens + 7) / 8), sms = sm_count();
  constexpr int kWeights = GATED ? 2 : 1;
  // Warps per tile: the fewest steps one after the other, a join and its barriers counted as half
  // a step; every warp has a step, and a CTA's teams have 15 named barriers.
  double best = 1e30;
  for (int ks = kFewWarps / kWeights; ks >= 1; ks /= 2) {
    if (ks > a.steps) continue;
    const int groups = std::max(1, std::min({kFewWarps / (ks * kWeights), (a.tiles + sms - 1) / sms, 15}));
    const int64_t rounds = (a.tiles + static_cast<int64_t>(groups) * sms - 1) / (static_cast<int64_t>(groups) * sms);
    const double cost = static_cast<double>(rounds) * ((a.steps + ks - 1) / ks + 0.5 * nt);
    if (cost < best) {
      best = cost;
      a.ks = ks;
      a.groups = groups;
    }
  }
  a.depth = few_depth(p);
  if (nt == 1) return run_few<FMT, LOG, 1, GATED, RAGGED>(a, s);
  if constexpr (few_tokens(FMT) > 16) {
    if (nt == 3) return run_few<FMT, LOG, 3, GATED, RAGGED>(a, s);
    if (nt == 4) return run_few<FMT, LOG, 4, GATED, RAGGED>(a, s);
  }
  return run_few<FMT, LOG, 2, GATED, RAGGED>(a, s);
}
bool encode_codes(CUtensorMap* m, const ProductArgs& p, const WeightView& w) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.cols / 2), static_cast<cuuint64_t>(p.rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.cols / 2)};
  const cuuint32_t box[2] = {128, 16}, es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(w.codes), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, bool RAGGED = false>
qz_status launch_few(const ProductArgs& p, cudaStream_t s) {
  FewArgs a{};
  a.p = p;
  if (!encode_codes(&a.map_w0, p, p.w0) || (p.n_weights == 2 && !encode_codes(&a.map_w1, p, p.w1))) return QZ_ERR_CUDA;
  a.tiles = static_cast<int>((p.rows + 15) / 16);
  a.steps = static_cast<int>(few_steps(p));
  a.x_chunks = 8 * a.steps;
  a.scale_pitch = (p.cols >> p.log2_block) * (FMT == QZ_INT4 ? 4 : 1);
  const bool two = p.mode == kModeGated;
  if constexpr (FMT == QZ_INT4) {
    if (p.log2_block == 5) return two ? run_few_nt<FMT, 5, true, RAGGED>(a, s) : run_few_nt<FMT, 5, false, RAGGED>(a, s);
    if (p.log2_block == 6) return two ? run_few_nt<FMT, 6, true, RAGGED>(a, s) : run_few_nt<FMT, 6, false, RAGGED>(a, s);
    return two ? run_few_nt<FMT, 7, true, RAGGED>(a, s) : run_few_nt<FMT, 7, false, RAGGED>(a, s);
  } else {
    return two ? run_few_nt<FMT, 0, true, RAGGED>(a, s) : run_few_nt<FMT, 0, false, RAGGED>(a, s);
  }
}

}  // namespace
}  // namespace qz
