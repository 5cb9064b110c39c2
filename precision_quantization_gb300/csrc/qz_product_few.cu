// qz_product_few.cu -- products of a few tokens (decoding, small batches) with 4-bit weights:
//   y[t][r] = sum_c W[r][c] x[t][c]        (one weight, or gate and up with the activation)
//
// Every weight is used once per token, so the weights' 4 bits (and scales) are the traffic and HBM
// the bound; the work to hide is the decoding, 8 weights per lane and mma.sync m16n8k16 (weights
// 16 rows, tokens the 8 columns: 32 tokens share one decoding in four of them).  The weights
// are exact in bf16 times their block scale (E2M1) or as integers (INT4, whose group scale takes
// the fp32 sum of its group), so the sums are those of include/qz.h.
//
// A tile is 16 outputs (gated: 16 of gate and of up).  KS of a CTA's eight warps share a tile, each
// with a contiguous part of the sum, and join their partial sums in shared memory in warp order;
// CTAs are persistent over the tiles.  A warp streams 128 columns of its 16 rows a step (64 bytes
// a row) through a ring of kDepth steps by cp.async, running on into the next tile, so the copies
// never pause; the activations come through L1, which they alone use.
#include <algorithm>
#include <cstdint>

#include "qz_device.cuh"
#include "qz_internal.h"
#include "qz_pipe.cuh"
#include "qz_product.h"
#include "qz_weight.cuh"

namespace qz {
namespace {

constexpr int kFewWarps = 8;
constexpr int kTokenStride = 20;  // floats of a token's 16 sums in the join (banks 8 t + g)

struct FewArgs {
  ProductArgs p;
  int tiles, ks, steps, scale_bytes;  // warps per tile, 128-wide steps of a row, bytes of scales a step
  int64_t code_pitch, scale_pitch;    // bytes per weight row
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mulb(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// byte q of a word as two 4-bit fields at bits 0 and 16
template <int Q>
__device__ __forceinline__ uint32_t nibbles(uint32_t t0, uint32_t t1) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(t0), "r"(t1), "n"(0x8080 | Q | ((4 + Q) << 8)));
  return d;
}
// E2M1 pairs as bf16 times 2^-126: sign to bit 15, exponent and mantissa to bits 6-8
__device__ __forceinline__ void word_pairs(uint32_t w, uint32_t (&d)[4]) {
  const uint32_t t0 = w & 0x0F0F0F0Fu, t1 = (w >> 4) & 0x0F0F0F0Fu;
  d[0] = nibbles<0>(t0, t1);
  d[1] = nibbles<1>(t0, t1);
  d[2] = nibbles<2>(t0, t1);
  d[3] = nibbles<3>(t0, t1);
}

// FMT; MT weights (gate and up: 2); NT groups of eight tokens; ring of D steps.
template <int FMT, int MT, int NT>
struct FewShape {
  static constexpr int kDepth = MT == 2 ? (NT >= 4 ? 3 : 4) : 8;
  static constexpr int kScale = FMT == QZ_MXFP4 ? 4 : FMT == QZ_NVFP4 ? 8 : 16;  // bytes of scales per row and step at most
  static constexpr uint32_t kSlot = MT * (1024 + 16 * kScale);
  static constexpr uint32_t kJoin = MT * NT * 8 * kTokenStride * 4;              // bytes per warp
  static constexpr uint32_t kSmem = kFewWarps * (kDepth * kSlot + kJoin);
};

template <int FMT, int MT, int NT>
__global__ void __launch_bounds__(32 * kFewWarps, 2) product_few_kernel(const __grid_constant__ FewArgs a) {
  using S = FewShape<FMT, MT, NT>;
  constexpr int kDepth = S::kDepth;
  extern __shared__ __align__(16) uint8_t few_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const ProductArgs& p = a.p;
  const uint32_t ring = smem_addr(few_smem) + warp * (kDepth * S::kSlot);
  const int ks = a.ks, group = warp / ks, part = warp % ks;
  const int tile0 = blockIdx.x * (kFewWarps / ks) + group, tile_step = gridDim.x * (kFewWarps / ks);
  const int s_begin = part * a.steps / ks, s_end = (part + 1) * a.steps / ks;
  const int rows = static_cast<int>(p.rows), tokens = static_cast<int>(p.tokens);

  // ---- the copies, kDepth - 1 steps ahead of the use ----
  int ptile = tile0, ps = s_begin, pslot = 0;
  const uint8_t* pc[MT][2];   // codes of rows g and g + 8 at this lane's 16 bytes of step 0
  const uint8_t* psc[MT];     // scales of row g (t = 0) or g + 8 (t = 1)
  const auto point = [&]() {
    const int r0 = min(ptile * 16 + g, rows - 1), r1 = min(ptile * 16 + g + 8, rows - 1);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const WeightView& w = m ? p.w1 : p.w0;
      pc[m][0] = w.codes + r0 * a.code_pitch + 16 * t;
      pc[m][1] = w.codes + r1 * a.code_pitch + 16 * t;
      psc[m] = static_cast<const uint8_t*>(w.scales) + (t == 0 ? r0 : r1) * a.scale_pitch;
    }
  };
  // INT4 reads word t of chunk c where FP4 reads its own chunk: chunk c of row g then sits at
  // c ^ (g / 2), which keeps the four-byte loads of a warp on 32 banks
  const uint32_t own = FMT == QZ_INT4 ? 64u * g + 16u * (t ^ (g >> 1)) : 16u * lane;
  const auto issue = [&]() {
    if (ptile < a.tiles) {
      const uint32_t slot = ring + pslot * S::kSlot;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        cp16(slot + m * 1024 + own, pc[m][0] + ps * 64);
        cp16(slot + m * 1024 + 512 + own, pc[m][1] + ps * 64);
        if (t < 2) {
          const uint32_t dst = slot + MT * 1024 + (m * 16 + g + 8 * t) * S::kScale;
          const uint8_t* src = psc[m] + static_cast<int64_t>(ps) * a.scale_bytes;
          if constexpr (FMT == QZ_MXFP4) {
            cp_small<4>(dst, src);
          } else if constexpr (FMT == QZ_NVFP4) {
            cp_small<8>(dst, src);
          } else {
            if (a.scale_bytes == 4) cp_small<4>(dst, src);
            else if (a.scale_bytes == 8) cp_small<8>(dst, src);
            else cp_small<16>(dst, src);
          }
        }
      }
      if (++ps == s_end) {
        ps = s_begin;
        ptile += tile_step;
        if (ptile < a.tiles) point();
      }
    }
    cp_commit();  // empty groups keep the count uniform
    pslot = pslot == kDepth - 1 ? 0 : pslot + 1;
  };
  if (ptile < a.tiles) point();
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) issue();

  // activations: token 8 nt + g (the last one again past the end: its columns are not stored)
  const uint16_t* px[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) px[nt] = p.x0 + static_cast<int64_t>(min(8 * nt + g, tokens - 1)) * p.ld_x + (FMT == QZ_INT4 ? 8 * t : 32 * t);

  float* join = reinterpret_cast<float*>(few_smem + kFewWarps * (kDepth * S::kSlot));
  constexpr int kJoin = S::kJoin / 4;
  int slot_i = 0;
  for (int tile = tile0; tile < a.tiles; tile += tile_step) {
    float z[MT][NT][4] = {};
#pragma unroll 1
    for (int s = s_begin; s < s_end; ++s) {
      cp_wait<kDepth - 2>();
      __syncwarp();  // every lane's copies of this slot are in; the slot before is read
      issue();
      const uint32_t slot = ring + slot_i * S::kSlot;
      slot_i = slot_i == kDepth - 1 ? 0 : slot_i + 1;
      if constexpr (FMT == QZ_INT4) {
        float acc[MT][NT][4] = {};
        const int per = a.scale_bytes == 4 ? 4 : a.scale_bytes == 8 ? 2 : 1;  // 32-wide chunks per group
        int gi = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // chunk c: 32 columns of one group, lane t its word t
          uint4 xv[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) xv[nt] = __ldg(reinterpret_cast<const uint4*>(px[nt] + s * 128 + 32 * c));
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint32_t at = slot + m * 1024 + 64u * g + 16u * (c ^ (g >> 1)) + 4u * t;
            uint32_t v[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              word_pairs(lds1(at + 512 * h), v[h]);
#pragma unroll
              for (int q = 0; q < 4; ++q)  // bf16 128 + (n ^ 8), less 136: the value, exactly
                asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(v[h][q]) : "r"((v[h][q] ^ 0x00080008u) | 0x43004300u), "r"(0xC308C308u));
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma(acc[m][nt], v[0][0], v[1][0], v[0][1], v[1][1], xv[nt].x, xv[nt].y);
              mma(acc[m][nt], v[0][2], v[1][2], v[0][3], v[1][3], xv[nt].z, xv[nt].w);
            }
          }
          if ((c + 1) % per == 0) {  // the group ends: its scale takes the sum
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const uint32_t sa = slot + MT * 1024 + (m * 16 + g) * S::kScale + 4u * gi;
              const float s0 = __uint_as_float(lds1(sa)), s1 = __uint_as_float(lds1(sa + 8 * S::kScale));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  z[m][nt][i] = __fmaf_rn(i < 2 ? s0 : s1, acc[m][nt][i], z[m][nt][i]);
                  acc[m][nt][i] = 0.0f;
                }
              }
            }
            ++gi;
          }
        }
      } else {
        uint32_t f[MT][2][2];   // bf16 factor pairs of rows g, g + 8; first and second 16 columns
        uint32_t extra[MT][2];
        bool big = false;
        uint4 cw[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            cw[m][h] = lds4(slot + m * 1024 + 512 * h + own);
            const uint32_t sa = slot + MT * 1024 + (m * 16 + g + 8 * h) * S::kScale;
            if constexpr (FMT == QZ_MXFP4) {
              // 2^(E - 127) 2^126; exponent fields above 254 take a second factor
              const uint32_t E = (lds1(sa) >> (8 * t)) & 255u;
              f[m][h][0] = f[m][h][1] = E == 255u ? 0x7FC07FC0u : (min(E + 126u, 254u) << 7) * 0x00010001u;
              extra[m][h] = E > 128u ? ((E - 1u) << 7) * 0x00010001u : 0x3F803F80u;
              big |= E > 128u;
            } else {
              // E4M3 bytes at bits 4-10 are 2^-120 of their value; times 2^127 2^111: 2^118 of it
              const uint32_t b = lds1(sa + 4u * (t >> 1)) >> (16 * (t & 1));
              const uint32_t c = mulb(mulb(((b & 255u) << 4) | ((b & 0xff00u) << 12), 0x7F007F00u), 0x77007700u);
              f[m][h][0] = __byte_perm(c, 0, 0x1010);
              f[m][h][1] = __byte_perm(c, 0, 0x3232);
            }
          }
        const bool any_big = FMT == QZ_MXFP4 && __any_sync(kFull, big);
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // word j: columns 32 t + 8 j .. + 7 of the step
          uint4 xv[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) xv[nt] = __ldg(reinterpret_cast<const uint4*>(px[nt] + s * 128 + 8 * j));
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint32_t v[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w = j == 0 ? cw[m][h].x : j == 1 ? cw[m][h].y : j == 2 ? cw[m][h].z : cw[m][h].w;
              word_pairs(w, v[h]);
#pragma unroll
              for (int q = 0; q < 4; ++q) v[h][q] = mulb((v[h][q] * 0x1040u) & 0x81C081C0u, f[m][h][j >> 1]);
              if (any_big) {
#pragma unroll
                for (int q = 0; q < 4; ++q) v[h][q] = mulb(v[h][q], extra[m][h]);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma(z[m][nt], v[0][0], v[1][0], v[0][1], v[1][1], xv[nt].x, xv[nt].y);
              mma(z[m][nt], v[0][2], v[1][2], v[0][3], v[1][3], xv[nt].z, xv[nt].w);
            }
          }
        }
      }
    }
    // ---- join the parts and store ----
    float* mine = join + warp * kJoin;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mine[((m * NT + nt) * 8 + 2 * t + (i & 1)) * kTokenStride + g + (i >= 2 ? 8 : 0)] = z[m][nt][i];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * ks) : "memory");
    const float* from = join + group * ks * kJoin;
    constexpr float kUnit = FMT == QZ_NVFP4 ? 256.0f : 1.0f;  // decoded NVFP4 weights are 2^-8 of their value
    const float f0 = sum_factor<FMT>(p.w0.tscale) * kUnit, f1 = MT == 2 ? sum_factor<FMT>(p.w1.tscale) * kUnit : 0.0f;
    for (int e = part * 32 + lane; e < 16 * tokens; e += 32 * ks) {
      const int row = tile * 16 + (e & 15), tok = e >> 4;
      float sum[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int at = (m * NT * 8 + tok) * kTokenStride + (e & 15);
        sum[m] = from[at];
        for (int w = 1; w < ks; ++w) sum[m] += from[w * kJoin + at];
      }
      if (row >= rows) continue;
      const int64_t o = static_cast<int64_t>(tok) * p.ld_y + row;
      const float v = sum[0] * f0;
      if constexpr (MT == 2) {
        const float u = sum[1] * f1;
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
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * ks) : "memory");
  }
  cp_wait<0>();
}

template <int FMT, int MT, int NT>
qz_status run_few(const FewArgs& a, cudaStream_t s) {
  using S = FewShape<FMT, MT, NT>;
  const void* k = reinterpret_cast<const void*>(&product_few_kernel<FMT, MT, NT>);
  if (!set_dyn_smem(k, static_cast<int>(S::kSmem))) return QZ_ERR_CUDA;
  const int per_cta = kFewWarps / a.ks;
  const int grid = std::min((a.tiles + per_cta - 1) / per_cta, 2 * sm_count());
  product_few_kernel<FMT, MT, NT><<<grid, 32 * kFewWarps, S::kSmem, s>>>(a);
  return launch_status();
}
template <int FMT, int MT>
qz_status run_few_nt(const FewArgs& a, cudaStream_t s) {
  switch ((a.p.tokens + 7) / 8) {
    case 1: return run_few<FMT, MT, 1>(a, s);
    case 2: return run_few<FMT, MT, 2>(a, s);
    case 3: return run_few<FMT, MT, 3>(a, s);
    default: return run_few<FMT, MT, 4>(a, s);
  }
}

}  // namespace

bool product_few_applicable(const ProductArgs& p) {
  // whole 128-wide steps; the scales of a step are one aligned copy; groups of 16 change inside
  // an INT4 mma
  if (p.mode == kModeBackward || p.tokens > kFewTokens || p.cols % 128 != 0 || p.cols == 0) return false;
  if (p.format == QZ_INT4 && p.log2_block < 5) return false;
  const uintptr_t n = p.format == QZ_MXFP4 ? 4 : p.format == QZ_NVFP4 ? 8 : (p.log2_block == 5 ? 16 : p.log2_block == 6 ? 8 : 4);
  const auto ok = [&](const void* q, uintptr_t a) { return reinterpret_cast<uintptr_t>(q) % a == 0; };
  return p.ld_x % 8 == 0 && ok(p.x0, 16) && ok(p.w0.codes, 16) && ok(p.w0.scales, n) &&
         (p.n_weights == 1 || (ok(p.w1.codes, 16) && ok(p.w1.scales, n)));
}

qz_status launch_product_few(const ProductArgs& p, cudaStream_t s) {
  FewArgs a{};
  a.p = p;
  a.tiles = static_cast<int>((p.rows + 15) / 16);
  a.steps = static_cast<int>(p.cols / 128);
  // all eight warps on a tile, while every warp has a step
  a.ks = 8;
  while (a.ks > a.steps) a.ks /= 2;
  a.scale_bytes = static_cast<int>((128 >> p.log2_block) * (p.format == QZ_INT4 ? 4 : 1));
  a.code_pitch = p.cols / 2;
  a.scale_pitch = static_cast<int64_t>(a.steps) * a.scale_bytes;
  const bool two = p.mode == kModeGated;
  if (p.format == QZ_MXFP4) return two ? run_few_nt<QZ_MXFP4, 2>(a, s) : run_few_nt<QZ_MXFP4, 1>(a, s);
  if (p.format == QZ_NVFP4) return two ? run_few_nt<QZ_NVFP4, 2>(a, s) : run_few_nt<QZ_NVFP4, 1>(a, s);
  return two ? run_few_nt<QZ_INT4, 2>(a, s) : run_few_nt<QZ_INT4, 1>(a, s);
}

}  // namespace qz
