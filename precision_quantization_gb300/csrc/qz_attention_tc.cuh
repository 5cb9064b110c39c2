// qz_attention_tc.cuh -- attention of many rows to the 8-bit cache (prompts) on the tcgen05 tensor cores,
// included once per format.  Heads of up to 128 elements.
//
//   x_j = (scale log2 e) ks_j (q . k_j),  p_j = 2^(x_j - m),  l = sum p_j,  out = sum p_j vs_j v_j / l
//
// A CTA holds two tiles of 128 rows (one where the sequences have fewer) of one sequence and kv head and
// walks the keys in tiles of 128 tokens.  Neither the tensor cores (41 %) nor the exponentials (21 %) are full: a row
// tile's own chain is the bound, scores - softmax - weights - P V - the next scores, which take the weights' place.  So
// each warp has one thing to do, and two row tiles take turns:
//   warps 0-7    softmax, one row of a tile a thread: x from tensor memory into registers, p back into its
//                place as f16
//   warps 8-15   decode: 16-byte pieces of codes become f16 in shared memory in the layout that the MMA
//                reads (keys K-major, values MN-major: the same bytes)
//   warp 16      issues the MMAs: x = Q K^T into 128 columns of tensor memory, out += P V with P as the
//                A operand from there
//   warps 17, 18 look up the pages and copy codes by TMA, keys and values, half a tile at a time
// in the order P0 V(j - 1), Q0 K(j), P1 V(j - 1), Q1 K(j): while one tile's softmax runs, the tensor cores work
// for the other.
// 8-bit codes are exact in f16, q is made f16 by a power of two of its row.  The maximum m is moved only
// when it is exceeded by more than 2^4, and the unit of the weights p vs (a power of two above every vs that the row
// has seen) by factors of four, so that the sums in tensor memory are rarely rescaled; p vs 2^11 / unit stays within
// f16, and keeps its 11 bits down to 2^-22 of the largest scale.
// Where the row tiles do not fill the GPU the keys are cut in `splits` parts, whose sums a second kernel joins.
//
// GPU times: 4096 new tokens of 8192, 32 / 8 heads x 128, E4M3: 471 us, 875 TFLOP/s (the operations at the library
// product's rate: 215); prompts of 5 sequences, 16 / 4 heads x 64, INT8: 108 us.  A step of 256 rows x 128 keys takes some
// 4400 cycles: 1330 of MMAs, and two softmaxes of 2900, a row tile's own chain of load, exponentials, conversion and
// store, which overlap with one another and with the MMAs only in part.  Sixteen softmax warps, two MMA warps, exponentials
// pipelined by hand and turns of the two tiles were slower.
#pragma once

#include "qz_attention.cuh"
#include "qz_internal.h"
#include "qz_tcgen05.cuh"

namespace qz {
namespace {

constexpr int kAttRows = 128, kAttKeys = 128;
constexpr int kAttSoftWarps = 8, kAttDecWarps = 8, kAttThreads = 32 * (kAttSoftWarps + kAttDecWarps + 4);
// registers a thread: launched with 96, 61440 in all = 256 x 176 + 256 x 40 + 128 x 48
constexpr int kAttSoftRegs = 176, kAttDecRegs = 40, kAttRestRegs = 48;
constexpr uint32_t kAttPanel = 128 * 128;            // 128 rows of 64 f16 values
constexpr uint32_t kAttTile = 2 * kAttPanel;
constexpr int kAttStages = 2, kAttScales = 4;
constexpr uint32_t kAttRaw = 128 * 128;              // a tile's codes
constexpr uint32_t kAttSmem = (2 + 2 * kAttStages) * kAttTile + 2 * kAttRaw + 1024;  // q, keys, values, codes of each
constexpr float kLazy = 4.0f, kPUnit = 0x1p11f;

struct AttTcArgs {
  AttentionArgs a;
  int32_t nq, splits, slots;   // row tiles of a CTA; parts of the keys; places for a kv head's CTAs
  int32_t box;                 // tokens of a copy: the largest of 16, 32, 64 that divides a page
  bool out_wide;               // 16-byte pieces of out are aligned
  CacheMaps maps;
};

// Bounded wait on phase `parity`.
__device__ __forceinline__ bool att_wait(uint64_t& bar, uint32_t parity, volatile int* abort) {
  const uint32_t at = smem_addr(&bar);
  if (held_try_wait(at, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!held_try_wait(at, parity)) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kTcWaitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// x (f16 pairs, tensor memory) as the A operand
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t at, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,"
      "%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]),
        "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]),
        "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]),
        "=f"(v[31])
      : "r"(at));
}
// every load before it has landed; the registers are handed on, so that nothing reads them earlier
__device__ __forceinline__ void tmem_wait32(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]),
                 "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]),
                 "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]),
                 "+f"(v[31]));
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
               "r"(v[14]), "r"(v[15])
               );
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint64_t add_pairs(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// fp32 accumulator, f16 operands; b_mn: B with its N index contiguous
__device__ __forceinline__ uint32_t idesc_f16(int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kAttRows >> 4) << 24);
}

struct AttBarriers {
  uint64_t k_full[kAttStages], k_empty[kAttStages], v_full[kAttStages], v_empty[kAttStages];
  uint64_t rk_full[2], rk_empty[2], rv_full[2], rv_empty[2];   // codes, by halves of a tile
  uint64_t s_full[2], p_full[2], scales[kAttScales], q_full, done;
};
struct AttScales {   // of a tile's 16-token groups; 0 for those past the end or without a page
  float ks[8], vs[8];
  float most;        // the largest finite |vs|
  uint32_t has;      // bit i: group i is there
  uint32_t odd;      // a scale is not finite
};

// The CTA's rows and keys.
struct AttWork {
  Span sp;
  int32_t seq, kvh, row0, rows;  // rows from row0 on, of `rows` in all
  int32_t t0, t1;                // tiles of keys
  int32_t seen0, seen1;          // the positions that every row sees
};

// ---- softmax ------------------------------------------------------------------------------------
// One row of tile q; a warp's 32 lanes of tensor memory.
__device__ __forceinline__ void softmax_role(const AttTcArgs& p, const AttWork& w, AttBarriers& bar, const AttScales* scales, uint32_t smem_q,
                                             uint32_t tmem, int q, volatile int* abort) {
  const AttentionArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, r = 32 * warp + lane;
  const int row = w.row0 + q * kAttRows + r, dim = a.c.dim;
  const bool mine = row < w.rows;
  const int i = row / a.group, head = w.kvh * a.group + row % a.group;
  const int64_t token = w.sp.row + i, pos = w.sp.p0 + i;
  // The warp's 32 rows of q as f16, K-major panels of 64 elements, 128-byte swizzle: a row at a time, four elements a
  // lane, all loads at once, eight rows' shuffles side by side.  Lane r keeps row r's factor.
  float fq = 0.0f;
  const int32_t left = w.rows - (w.row0 + q * kAttRows);  // of the tile's rows
  uint2 raw[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const bool in = 32 * warp + k < left && 4 * lane < dim;
    const int rr = w.row0 + q * kAttRows + 32 * warp + k, ri = rr / a.group;
    raw[k] = load_q4_raw(a, in, (w.sp.row + ri) * a.ld_q + (w.kvh * a.group + rr - ri * a.group) * a.hd_q + 4 * lane);
  }
#pragma unroll
  for (int rows = 0; rows < 32; rows += 8) {
    const int r0 = 32 * warp + rows;
    float x[8][4], top[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint2 b = raw[rows + k];
      x[k][0] = __uint_as_float(b.x << 16), x[k][1] = __uint_as_float(b.x & 0xffff0000u);
      x[k][2] = __uint_as_float(b.y << 16), x[k][3] = __uint_as_float(b.y & 0xffff0000u);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) top[k] = absmax_nan(absmax_nan(absmax_nan(fabsf(x[k][0]), x[k][1]), x[k][2]), x[k][3]);
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int k = 0; k < 8; ++k) top[k] = absmax_nan(top[k], __shfl_xor_sync(kFull, top[k], o));
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float down;
      const float up = q_unit(top[k], down);
      if (32 * warp + lane == r0 + k) fq = down * a.scale;
      if (4 * lane < dim) {
        const int line = r0 + k;
        const uint32_t at = smem_q + q * kAttTile + (lane >> 4) * kAttPanel + line * 128 + ((((lane >> 1) & 7) ^ (line & 7)) << 4) + (lane & 1) * 8;
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(f16x2_bits(x[k][0] * up, x[k][1] * up)),
                     "r"(f16x2_bits(x[k][2] * up, x[k][3] * up))
                     : "memory");
      }
    }
  }
  fence_proxy_async();
  __syncwarp();
  if (lane == 0) arrive_local(smem_addr(&bar.q_full));
  const int32_t end = mine ? static_cast<int32_t>(max(min(pos + 1, static_cast<int64_t>(w.sp.len)), static_cast<int64_t>(0))) : INT32_MAX;
  const int32_t begin = mine ? static_cast<int32_t>(max(pos + 1 - a.window, static_cast<int64_t>(0))) : 0;
  int32_t all_end = end, all_begin = begin;  // what every row of the warp sees
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    all_end = min(all_end, __shfl_xor_sync(kFull, all_end, o));
    all_begin = max(all_begin, __shfl_xor_sync(kFull, all_begin, o));
  }
  const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
  const uint32_t ts = tmem + q * kAttKeys + lanes, to = tmem + 2 * kAttKeys + q * kAttRows + lanes;
  float m = kNone, l = 0.0f, unit = 0x1p-100f;
  bool ok = true;
  for (int32_t t = w.t0; t < w.t1; ++t) {
    const int n = t - w.t0;
    const AttScales& sc = scales[n % kAttScales];
    ok = att_wait(bar.scales[n % kAttScales], (n / kAttScales) & 1, abort) && att_wait(bar.s_full[q], n & 1, abort);
    ok = __all_sync(kFull, ok);
    if (!ok) break;
    tc_fence_after();
    float v[4][32];
    tmem_load32(ts, v[0]);
    tmem_load32(ts + 32, v[1]);
    const int32_t j0 = t * kAttKeys;   // (keys lie below 2^31: so does the tile's last place but for the very last tile)
    const bool whole = all_end - j0 >= kAttKeys && j0 >= all_begin && sc.has == 255u, odd = sc.odd != 0;
    // 16 weights of group g from their scores: p = 2^(f x - from), their sum, and p fv as f16
    const auto weigh = [&](int g, float f, float fv, uint64_t minus, uint64_t (&sum)[2], uint32_t* y) {
      const float* s16 = &v[g >> 1][16 * (g & 1)];
      const uint64_t ff = pk(f, f), ffv = pk(fv, fv);
      uint64_t x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fma2(pk(s16[2 * e], s16[2 * e + 1]), ff, minus);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float x0, x1;
        upk(x[e], x0, x1);
        x[e] = pk(ex2(x0), ex2(x1));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e & 1] = add_pairs(sum[e & 1], x[e]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float x0, x1;
        upk(mul2(x[e], ffv), x0, x1);
        y[e] = f16x2_bits(x0, x1);
      }
    };
    const auto largest = [&](int g) {
      const float* x = &v[g >> 1][16 * (g & 1)];
      float y = x[0], z = x[1];
#pragma unroll
      for (int e = 2; e < 14; e += 4) y = max3(y, x[e], x[e + 1]), z = max3(z, x[e + 2], x[e + 3]);
      return fmaxf(max3(y, x[14], x[15]), z);
    };
    tmem_wait32(v[0]);
    tmem_wait32(v[1]);
    tmem_load32(ts + 64, v[2]);
    tmem_load32(ts + 96, v[3]);
    bool done = false;
    if (__all_sync(kFull, whole && !odd && m != kNone && sc.most <= unit)) {
      // the usual tile: the weights against the maximum so far while this tile's is still being found; taken back in the
      // rare case that it is exceeded
      const float inverse = kPUnit / unit;
      const uint64_t minus = pk(-m, -m);
      uint64_t sum[2] = {pk(0.0f, 0.0f), pk(0.0f, 0.0f)};
      float top = kNone;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c == 2) tmem_wait32(v[2]), tmem_wait32(v[3]);
        uint32_t y[16];
#pragma unroll
        for (int g = 2 * c; g < 2 * c + 2; ++g) {
          const float f = fq * sc.ks[g];
          weigh(g, f, sc.vs[g] * inverse, minus, sum, y + 8 * (g & 1));
          top = fmaxf(top, largest(g) * f);  // (a scale is not negative)
        }
        tmem_store16(ts + 16 * c, y);
      }
      if (!__any_sync(kFull, top > m + kLazy)) {
        float s0, s1;
        upk(add_pairs(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        done = true;
      }
    } else {
      tmem_wait32(v[2]);
      tmem_wait32(v[3]);
    }
    if (!done) {
      uint32_t off = 0;  // groups that the row sees nothing of: their scales may be anything, and change nothing that it keeps
      if (!whole) {
        const int hi = max(min(end - j0, kAttKeys), 0), lo = max(min(begin - j0, kAttKeys), 0);
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const bool none = 16 * g >= hi || 16 * g + 16 <= lo || !((sc.has >> g) & 1u);
          off |= (none ? 1u : 0u) << g;
          const int first = none ? 16 : lo - 16 * g, last = none ? 0 : hi - 16 * g;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float& x = v[g >> 1][16 * (g & 1) + e];
            if (e >= last || e < first) x = kNone;
          }
        }
      }
      const auto key_scale = [&](int g) {  // not 0, so that -inf stays -inf; NaN stays NaN
        float f;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(fq * sc.ks[g]), "f"(0x1p-126f));
        return odd && ((off >> g) & 1u) ? 0x1p-126f : f;
      };
      float top = kNone;
#pragma unroll
      for (int g = 0; g < 8; ++g) top = fmaxf(top, largest(g) * key_scale(g));
      const float was = m, unit_was = unit;
      if (top > m + kLazy || (m == kNone && top > m)) m = top;
      float most = sc.most;
      if (off) {
        most = 0.0f;
#pragma unroll
        for (int g = 0; g < 8; ++g) most = fmaxf(most, (off >> g) & 1u || !is_finite_f(sc.vs[g]) ? 0.0f : fabsf(sc.vs[g]));
      }
      if (most > unit)  // four times the next power of two
        unit = __uint_as_float((__float_as_uint(fminf(most, 0x1p120f)) & 0x7f800000u) + 3u * 0x00800000u);
      if (__any_sync(kFull, m != was || unit != unit_was)) {
        const float f = was == kNone ? 1.0f : ex2(was - m), fo = f * (unit_was / unit);
        l *= f;
        if (n > 0) {
#pragma unroll 1
          for (int c = 0; c < dim; c += 16) {
            float o8[8], o9[8];
            tmem_load8(to + c, o8);
            tmem_load8(to + c + 8, o9);
            tmem_wait8(o8);
            tmem_wait8(o9);
            uint32_t y[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(o8[e] * fo), y[8 + e] = __float_as_uint(o9[e] * fo);
            tmem_store16(to + c, y);
          }
        }
      }
      const float from = m == kNone ? 0.0f : m, inverse = kPUnit / unit;
      const uint64_t minus = pk(-from, -from);
      uint64_t sum[2] = {pk(0.0f, 0.0f), pk(0.0f, 0.0f)};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t y[16];
#pragma unroll
        for (int g = 2 * c; g < 2 * c + 2; ++g)
          weigh(g, key_scale(g), (off >> g) & 1u ? 0.0f : sc.vs[g] * inverse, minus, sum, y + 8 * (g & 1));
        tmem_store16(ts + 16 * c, y);
      }
      float s0, s1;
      upk(add_pairs(sum[0], sum[1]), s0, s1);
      l += s0 + s1;
    }
    tmem_stored();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_local(smem_addr(&bar.p_full[q]));
  }
  // ---- the result ----
  if (w.t0 < w.t1) ok = __all_sync(kFull, att_wait(bar.done, 0, abort)) && ok && !*abort;
  tc_fence_after();
  if (!ok) l = __uint_as_float(0x7fc00000u);
  const float back = unit * (1.0f / kPUnit);
  float *part = nullptr, *stat = nullptr;
  if (p.splits > 1) {
    const int64_t all = static_cast<int64_t>(a.b.tokens) * a.heads, split = blockIdx.x % p.splits, at = split * all + token * a.heads + head;
    part = static_cast<float*>(a.ws) + at * dim;
    stat = static_cast<float*>(a.ws) + p.splits * all * dim + at * 2;
    if (mine) stat[0] = m, stat[1] = l;
  }
  const bool wide = p.splits == 1 && p.out_wide;  // 16-byte stores
  const float scale = l == 0.0f ? 0.0f : __fdiv_rn(back, l);
  if (wide && mine && a.lse) a.lse[token * a.ld_lse + head] = l == 0.0f ? kNone : (m + log2f(l)) * 0.69314718055994531f;
#pragma unroll 1
  for (int c = 0; c < dim; c += 32) {  // (the accumulator has 128 columns whatever dim is)
    float o[32];
    __syncwarp();
    if (w.t0 < w.t1) {
      tmem_load32(to + c, o);
      tmem_wait32(o);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = 0.0f;
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int d = c + 8 * h;
      if (!mine || d >= dim) break;
      if (wide) {
        *reinterpret_cast<uint4*>(a.out + token * a.ld_out + head * a.hd_out + d) =
            make_uint4(bf16x2_bits(o[8 * h] * scale, o[8 * h + 1] * scale), bf16x2_bits(o[8 * h + 2] * scale, o[8 * h + 3] * scale),
                       bf16x2_bits(o[8 * h + 4] * scale, o[8 * h + 5] * scale), bf16x2_bits(o[8 * h + 6] * scale, o[8 * h + 7] * scale));
        continue;
      }
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float y[4] = {o[8 * h + 4 * z] * back, o[8 * h + 4 * z + 1] * back, o[8 * h + 4 * z + 2] * back, o[8 * h + 4 * z + 3] * back};
        if (part) *reinterpret_cast<float4*>(part + d + 4 * z) = make_float4(y[0], y[1], y[2], y[3]);
        else store_row(a, token, head, d + 4 * z, y, m, l);
      }
    }
  }
  tc_fence_before();
}

// ---- copies --------------------------------------------------------------------------------------
// KEYS: the keys' codes, and the scales of both; else the values' codes.  Lane i < 8 stands for the i-th 16
// tokens of a tile.  Pages are looked up two tiles ahead, scales one.
template <bool KEYS>
__device__ __forceinline__ void copy_role(const AttTcArgs& p, const AttWork& w, AttBarriers& bar, AttScales* scales, uint32_t raw, volatile int* abort) {
  const AttentionArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const uint32_t row = a.c.dim <= 64 ? 64u : 128u, bytes = static_cast<uint32_t>(p.box) * row, at = static_cast<uint32_t>(16 * lane) * row;
  uint64_t* full = KEYS ? bar.rk_full : bar.rv_full;
  uint64_t* empty = KEYS ? bar.rk_empty : bar.rv_empty;
  struct Place {
    int32_t page, in;
  };
  const auto look = [&](int32_t t) {
    const int64_t j = static_cast<int64_t>(t) * kAttKeys + 16 * lane;
    Place r{-1, 0};
    if (lane < 8 && t < w.t1 && j < w.sp.len) {
      const int32_t i = static_cast<int32_t>(j) / a.c.page;
      r.in = static_cast<int32_t>(j) - i * a.c.page;
      r.page = __ldg(a.b.table + w.seq * a.b.ld_table + i);
      if (r.page >= a.c.pages) r.page = -1;
    }
    return r;
  };
  const auto head_of = [&](const Place& r) { return max(r.page, 0) * a.c.heads + w.kvh; };
  float ks = 0.0f, vs = 0.0f;
  const auto fetch = [&](const Place& r) {
    ks = vs = 0.0f;
    if (KEYS && r.page >= 0) {
      const int64_t block = static_cast<int64_t>(head_of(r)) * (a.c.page >> a.c.log2_block) + (r.in >> a.c.log2_block);
      ks = __ldg(a.c.ks + block), vs = __ldg(a.c.vs + block);
    }
  };
  Place now = look(w.t0), next = look(w.t0 + 1);
  fetch(now);
  uint32_t parity = 0;
  bool ok = true;
  int32_t t = w.t0;
  for (; t < w.t1 && ok; ++t, parity ^= 1u) {
    const int n = t - w.t0;
    const bool starts = now.page >= 0 && lane % (p.box / 16) == 0;
    const uint32_t mask = __ballot_sync(kFull, starts);
    const int32_t head = head_of(now);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!(ok = __all_sync(kFull, att_wait(empty[h], parity ^ 1u, abort)))) break;
      if (KEYS && h == 0) {
        // (slot n % 4 is free: the keys of tile n - 1 are being decoded, so the scores of n - 3 are in, so the weights
        // of n - 4 were)
        float most = is_finite_f(vs) ? fabsf(vs) : 0.0f;
#pragma unroll
        for (int o = 4; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
        const uint32_t has = __ballot_sync(kFull, now.page >= 0);
        const uint32_t odd = __any_sync(kFull, !is_finite_f(ks) || !is_finite_f(vs)) ? 1u : 0u;
        AttScales& sc = scales[n % kAttScales];
        if (lane < 8) sc.ks[lane] = ks, sc.vs[lane] = vs;
        if (lane == 0) sc.has = has, sc.most = most, sc.odd = odd;
        __syncwarp();
        if (lane == 0) arrive_local(smem_addr(&bar.scales[n % kAttScales]));
      }
      if (lane == 0) mbar_expect_tx(smem_addr(&full[h]), __popc(mask & (h ? 0xf0u : 0x0fu)) * bytes);
      __syncwarp();
      if (starts && lane >> 2 == h) box_load(raw + at, KEYS ? &p.maps.k : &p.maps.v, 0, now.in, head, smem_addr(&full[h]));
    }
    now = next;
    next = look(t + 2);
    fetch(now);
  }
  if (*abort) {  // copies in flight land before the memory is released
    for (int i = 0; i < 4; ++i) mbar_wait(smem_addr(&full[i >> 1]), i & 1, kTcWaitNs / 4);
  }
}

// ---- decoding -----------------------------------------------------------------------------------
// A thread's pieces of half a tile: eight lanes take eight rows, so that both the reads (TMA's swizzle) and
// the writes (the MMA's) touch every bank once.
template <int FMT>
__device__ __forceinline__ void decode_role(const AttTcArgs& p, const AttWork& w, AttBarriers& bar, const AttScales* scales, uint32_t raw_k,
                                            uint32_t raw_v, uint32_t smem_k, uint32_t smem_v, volatile int* abort) {
  const int lane = threadIdx.x & 31, dw = static_cast<int>(threadIdx.x >> 5) - kAttSoftWarps, dim = p.a.c.dim, pieces = dim / 16;
  const int line = 8 * dw + (lane & 7);   // of 64
  const uint32_t row_bytes = dim <= 64 ? 64u : 128u;
  uint32_t from[2], to[2];                // pieces lane / 8 and lane / 8 + 4
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int ch = (lane >> 3) + 4 * i;
    from[i] = dim <= 64 ? line * 64 + ((ch ^ ((line >> 1) & 3)) << 4) : line * 128 + ((ch ^ (line & 7)) << 4);
    to[i] = i * kAttPanel + line * 128 + (((2 * (ch & 3)) ^ (line & 7)) << 4);
  }
  const bool first = (lane >> 3) < pieces, second = (lane >> 3) + 4 < pieces;
  const auto decode = [&](uint32_t raw, uint32_t tile, bool there) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!(i ? second : first)) continue;
      uint32_t cw[4], h[8];
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(cw[0]), "=r"(cw[1]), "=r"(cw[2]), "=r"(cw[3]) : "r"(raw + from[i]));
      if (!there) cw[0] = cw[1] = cw[2] = cw[3] = 0u;  // what is past the end, or not there, may be anything
#pragma unroll
      for (int k = 0; k < 4; ++k) pairs_in_word<FMT>(prepare_word<FMT>(cw[k]), h[2 * k], h[2 * k + 1]);
      const uint32_t x0[4] = {h[0], h[1], h[2], h[3]}, x1[4] = {h[4], h[5], h[6], h[7]};
      sts16(tile + to[i], x0);
      sts16((tile + to[i]) ^ 16u, x1);
    }
  };
  for (int32_t t = w.t0; t < w.t1; ++t) {
    const int n = t - w.t0, s = n % kAttStages;
    const uint32_t ph = (n / kAttStages) & 1, raw = n & 1;
    const int64_t rows = w.sp.len - static_cast<int64_t>(t) * kAttKeys;
    bool ok = true, there[2];
    // Where not every row sees the whole tile, a token whose values are not finite numbers gets zeros for them and NaN for
    // its key: its scores are masked for the rows that do not see it, and spoil the others.  (A warp's own lines.)
    if (FMT != QZ_INT8 && (t * static_cast<int64_t>(kAttKeys) < w.seen0 || t * static_cast<int64_t>(kAttKeys) + kAttKeys > w.seen1)) {
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (!(ok = __all_sync(kFull, att_wait(bar.rv_full[h], raw, abort) && att_wait(bar.rk_full[h], raw, abort)))) break;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t cw[4] = {0u, 0u, 0u, 0u};
          if (i ? second : first)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(cw[0]), "=r"(cw[1]), "=r"(cw[2]), "=r"(cw[3]) : "r"(raw_v + 64 * h * row_bytes + from[i]));
          odd = odd || has_nonfinite<FMT>(cw[0], cw[1], cw[2], cw[3]);
        }
        const uint32_t lines = __ballot_sync(kFull, odd);  // a line's pieces are those of lanes 8 apart
        if (lines & (0x01010101u << (lane & 7))) {
          const uint32_t zeros[4] = {0u, 0u, 0u, 0u}, nans[4] = {0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!(i ? second : first)) continue;
            sts16(raw_v + 64 * h * row_bytes + from[i], zeros);
            sts16(raw_k + 64 * h * row_bytes + from[i], nans);
          }
          fence_proxy_async();  // (before the next copies there)
        }
        __syncwarp();
      }
    }
    if (!ok) break;
#pragma unroll
    for (int z = 0; z < 2; ++z) {  // keys, values
      uint64_t* full = z ? bar.rv_full : bar.rk_full;
      uint64_t* empty = z ? bar.rv_empty : bar.rk_empty;
      ok = att_wait(z ? bar.v_empty[s] : bar.k_empty[s], ph ^ 1u, abort);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!(ok = __all_sync(kFull, ok && att_wait(full[h], raw, abort)))) break;
        if (z == 0) there[h] = 64 * h + line < rows && ((scales[n % kAttScales].has >> ((64 * h + line) >> 4)) & 1u);
        decode((z ? raw_v : raw_k) + 64 * h * row_bytes, (z ? smem_v : smem_k) + s * kAttTile + 64 * h * 128, there[h]);
        if (h == 1) fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive_local(smem_addr(&empty[h]));
      }
      if (!ok) break;
      if (lane == 0) arrive_local(smem_addr(z ? &bar.v_full[s] : &bar.k_full[s]));
    }
    if (!ok) break;
  }
}

// ---- the tensor cores ----------------------------------------------------------------------------
__device__ __forceinline__ void mma_role(const AttTcArgs& p, const AttWork& w, AttBarriers& bar, uint32_t smem_q, uint32_t smem_k, uint32_t smem_v,
                                         uint32_t tmem, volatile int* abort) {
  const int steps = p.a.c.dim / 16;
  const uint32_t id_s = idesc_f16(kAttKeys, false), id_o = idesc_f16(p.a.c.dim, true);
  bool ok = att_wait(bar.q_full, 0, abort);
  const auto scores = [&](int q, int s) {
    const uint64_t qd = desc_sw128(smem_q + q * kAttTile, 16u, 1024u), kd = desc_sw128(smem_k + s * kAttTile, 16u, 1024u);
    for (int k = 0; k < steps; ++k) {
      const uint32_t at = (k >> 2) * (kAttPanel >> 4) + 2u * (k & 3);
      tc_mma<1>(tmem + q * kAttKeys, qd + at, kd + at, id_s, k > 0);
    }
    tc_commit<1>(smem_addr(&bar.s_full[q]));
  };
  const auto sums = [&](int q, int s, bool first) {
    const uint64_t vd = desc_sw128(smem_v + s * kAttTile, kAttPanel, 1024u);
#pragma unroll
    for (int k = 0; k < kAttKeys / 16; ++k)
      mma_ts(tmem + 2 * kAttKeys + q * kAttRows, tmem + q * kAttKeys + 8 * k, vd + 128u * k, id_o, !(first && k == 0));
  };
  for (int32_t t = w.t0; t <= w.t1 && ok; ++t) {   // scores of tile t, sums of the one before
    const int n = t - w.t0, s = n % kAttStages, before = (n + kAttStages - 1) % kAttStages;
    if (t < w.t1 && !(ok = att_wait(bar.k_full[s], (n / kAttStages) & 1, abort))) break;
    if (n > 0 && !(ok = att_wait(bar.v_full[before], ((n - 1) / kAttStages) & 1, abort))) break;
    for (int q = 0; q < p.nq && ok; ++q) {
      if (n > 0) {
        if (!(ok = att_wait(bar.p_full[q], (n - 1) & 1, abort))) break;
        tc_fence_after();
        sums(q, before, n == 1);
        if (q == p.nq - 1) tc_commit<1>(smem_addr(&bar.v_empty[before]));
      }
      tc_fence_after();
      if (t < w.t1) scores(q, s);
    }
    if (ok && t < w.t1) tc_commit<1>(smem_addr(&bar.k_empty[s]));
  }
  tc_commit<1>(smem_addr(&bar.done));  // every MMA issued has completed before tensor and shared memory are released
}

template <int FMT>
__global__ void __launch_bounds__(kAttThreads, 1) attention_tc_kernel(const __grid_constant__ AttTcArgs p) {
  extern __shared__ uint8_t att_raw[];
  __shared__ __align__(8) AttBarriers bar;
  __shared__ AttScales scales[kAttScales];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int s_abort;
  const AttentionArgs& a = p.a;
  const int warp = static_cast<int>(threadIdx.x) >> 5;
  const uint32_t base = (smem_addr(att_raw) + 1023u) & ~1023u;
  const uint32_t smem_q = base, smem_k = base + 2 * kAttTile, smem_v = smem_k + kAttStages * kAttTile, raw_k = smem_v + kAttStages * kAttTile, raw_v = raw_k + kAttRaw;

  // the longest work first: the last rows of the last sequences see the most
  const int64_t at = blockIdx.x / p.splits;
  const int split = static_cast<int>(blockIdx.x % p.splits);
  const int64_t slot = p.slots - 1 - at / a.c.heads;
  AttWork w;
  w.kvh = static_cast<int32_t>(at % a.c.heads);
  const int tile_rows = p.nq * kAttRows;
  const auto first_slot = [&](int32_t s) { return tc_first_slot(start_of(a.b, s), s, a.group, tile_rows); };
  w.seq = count_upto(a.b.seqs, first_slot, slot) - 1;
  if (w.seq < 0) return;
  w.sp = span_of(a.b, w.seq, a.c.page);
  const int64_t all_rows = static_cast<int64_t>(w.sp.n) * a.group, row0 = tc_tile_row(slot, first_slot(w.seq), all_rows, tile_rows);
  if (row0 < 0) return;
  w.row0 = static_cast<int32_t>(row0);
  w.rows = static_cast<int32_t>(all_rows);
  {
    const int64_t last = min(row0 + tile_rows, all_rows) - 1;
    const int64_t lo = max(w.sp.p0 + row0 / a.group + 1 - a.window, static_cast<int64_t>(0));
    const int64_t hi = min(w.sp.p0 + last / a.group + 1, static_cast<int64_t>(w.sp.len));
    const int64_t t0 = lo / kAttKeys, count = max((hi + kAttKeys - 1) / kAttKeys - t0, static_cast<int64_t>(0));
    w.t0 = static_cast<int32_t>(t0 + count * split / p.splits);
    w.t1 = static_cast<int32_t>(t0 + count * (split + 1) / p.splits);
    w.seen0 = static_cast<int32_t>(max(w.sp.p0 + last / a.group + 1 - a.window, static_cast<int64_t>(0)));
    w.seen1 = static_cast<int32_t>(max(min(w.sp.p0 + row0 / a.group + 1, static_cast<int64_t>(w.sp.len)), static_cast<int64_t>(0)));
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kAttStages; ++s) {
      mbar_init(smem_addr(&bar.k_full[s]), kAttDecWarps);
      mbar_init(smem_addr(&bar.v_full[s]), kAttDecWarps);
      mbar_init(smem_addr(&bar.k_empty[s]), 1);
      mbar_init(smem_addr(&bar.v_empty[s]), 1);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(smem_addr(&bar.s_full[q]), 1);
      mbar_init(smem_addr(&bar.p_full[q]), 4);
    }
    for (int s = 0; s < kAttScales; ++s) mbar_init(smem_addr(&bar.scales[s]), 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(smem_addr(&bar.rk_full[h]), 1);
      mbar_init(smem_addr(&bar.rv_full[h]), 1);
      mbar_init(smem_addr(&bar.rk_empty[h]), kAttDecWarps);
      mbar_init(smem_addr(&bar.rv_empty[h]), kAttDecWarps);
    }
    mbar_init(smem_addr(&bar.q_full), 4 * p.nq);
    mbar_init(smem_addr(&bar.done), 1);
    mbar_init_fence();
    s_abort = 0;
  }
  if (warp == kAttSoftWarps + kAttDecWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (warp < kAttSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAttSoftRegs));
    if (warp / 4 < p.nq) softmax_role(p, w, bar, scales, smem_q, tmem, warp / 4, &s_abort);
  } else if (warp < kAttSoftWarps + kAttDecWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAttDecRegs));
    decode_role<FMT>(p, w, bar, scales, raw_k, raw_v, smem_k, smem_v, &s_abort);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAttRestRegs));
    if (warp == kAttSoftWarps + kAttDecWarps) {
      if (w.t0 < w.t1 && elect_one()) mma_role(p, w, bar, smem_q, smem_k, smem_v, tmem, &s_abort);
      __syncwarp();
      // (after a wait has given up the others may come here before the last MMA has completed)
      if (w.t0 < w.t1) att_wait(bar.done, 0, &s_abort);
      if (s_abort) mbar_wait(smem_addr(&bar.done), 0, kTcWaitNs);
    } else if (warp == kAttSoftWarps + kAttDecWarps + 1) {
      copy_role<true>(p, w, bar, scales, raw_k, &s_abort);
    } else if (warp == kAttSoftWarps + kAttDecWarps + 2) {
      copy_role<false>(p, w, bar, scales, raw_v, &s_abort);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kAttSoftWarps + kAttDecWarps) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// The parts' sums, four elements a thread.
__global__ void __launch_bounds__(256) attention_tc_join_kernel(const __grid_constant__ AttTcArgs p) {
  const AttentionArgs& a = p.a;
  const int dim = a.c.dim, quads = dim / 4;
  const int64_t all = static_cast<int64_t>(a.b.tokens) * a.heads;
  const int64_t first = static_cast<int64_t>(start_of(a.b, 0)) * a.heads, end = static_cast<int64_t>(start_of(a.b, a.b.seqs)) * a.heads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float* parts = static_cast<const float*>(a.ws);
  const float2* stats = reinterpret_cast<const float2*>(parts + p.splits * all * dim);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < all * quads; i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i / quads;
    const int d = 4 * static_cast<int>(i - row * quads);
    if (row < first || row >= end) continue;  // no sequence's
    float top = kNone;
#pragma unroll 4
    for (int k = 0; k < p.splits; ++k) top = fmaxf(top, stats[k * all + row].x);
    const float from = top == kNone ? 0.0f : top;
    float v[4] = {}, l = 0.0f;
#pragma unroll 4
    for (int k = 0; k < p.splits; ++k) {
      const float2 st = stats[k * all + row];
      const float f = ex2(st.x - from);
      const float4 y = *reinterpret_cast<const float4*>(parts + (k * all + row) * dim + d);
      l = __fmaf_rn(st.y, f, l);
      v[0] = __fmaf_rn(y.x, f, v[0]), v[1] = __fmaf_rn(y.y, f, v[1]);
      v[2] = __fmaf_rn(y.z, f, v[2]), v[3] = __fmaf_rn(y.w, f, v[3]);
    }
    store_row(a, row / a.heads, static_cast<int>(row % a.heads), d, v, top, l);
  }
}

template <int FMT>
qz_status launch_tc(const AttentionArgs& a, const TcAttPlan& plan, cudaStream_t s) {
  AttTcArgs p{};
  p.a = a;
  p.nq = plan.nq, p.splits = plan.splits, p.slots = plan.slots;
  p.out_wide = is_aligned(a.out, 16) && (a.b.tokens <= 1 || a.ld_out % 8 == 0) && (a.heads <= 1 || a.hd_out % 8 == 0);
  p.box = a.c.page % 64 == 0 ? 64 : a.c.page % 32 == 0 ? 32 : 16;
  if (a.c.pages > 0 && !encode_maps(&p.maps, a, p.box)) return QZ_ERR_CUDA;
  const auto k = &attention_tc_kernel<FMT>;
  if (!set_dyn_smem(reinterpret_cast<const void*>(k), kAttSmem)) return QZ_ERR_CUDA;
  k<<<static_cast<unsigned>(plan.grid), kAttThreads, kAttSmem, s>>>(p);
  if (launch_status() != QZ_OK) return QZ_ERR_CUDA;
  if (plan.splits == 1) return QZ_OK;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  const int64_t blocks = (static_cast<int64_t>(a.b.tokens) * a.heads * (a.c.dim / 4) + 255) / 256;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attention_tc_join_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return QZ_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace
}  // namespace qz
