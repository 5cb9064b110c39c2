// qz_cache.cu -- appending keys and values to a paged 8-bit cache, the keys (and the queries) rotated on
// the way (include/qz.h, qz_cache_append).
//
//   s = max(s_held, fl32(A / qmax)) per block of tokens and head, A = max |x| over its new values;
//   new codes RNE(fl32(x / s)), held codes RNE(fl32(decode(q) fl32(s_held / s))) where s has grown.
//
// A CTA takes one block of one kv head of one sequence: its new keys and values are read once and held in
// registers, 16 a thread and piece, from the amax to the codes.  Which blocks get tokens is known
// on the GPU only (lengths and starts lie there), so the grid covers the most that there can be: n tokens
// touch at most (n - 1) / block + 2 blocks, and with floor(start / block) + 2 s as sequence s's first slot
// no two sequences' slots meet.  (One token each: a warp does.)  Further CTAs rotate the queries.
//
// By its bytes bound by HBM; what takes the time is the chain length - page - amax - scale - codes, which a CTA goes
// through once, and some 20 instructions a value.  GPU times:
//   1 token, 8 kv heads x 128, E4M3         3.2 us, launch and the chain
//   128 sequences x 1 token, INT8           3.9 us (append_one_kernel)
//   prompts of 11400 tokens, E4M3, bf16     71 us for 263 MB: queries 39 (187 MB, 4.8 TB/s), keys and values 32
#include "qz_cache.h"

#include <climits>
#include <cstdint>

#include "qz_internal.h"
#include "qz_pipe.cuh"
#include "qz_rotary.cuh"

namespace qz {
namespace {

constexpr int kAppThreads = 256;
constexpr int kAppWarps = kAppThreads / 32;
// Tokens from which the queries have a launch of their own: beside keys and values they run with the 99 registers of
// append_kernel, 64 here (11400 tokens: 80 us in one launch, 72 in two); below, the launch itself (2 us) is more than that.
constexpr int64_t kApart = 256;

struct AppendArgs {
  CacheView c;
  BatchView b;
  RotaryView r;
  const void *k, *v, *q;
  void* q_out;
  int64_t ld_k, hd_k, ld_v, hd_v, ld_q, hd_q, ld_qo, hd_qo;
  int32_t q_heads, q_units;  // threads of a query vector
  uint32_t kv_ctas;          // for keys and values; the CTAs behind them rotate queries
};

template <int FMT>
__device__ __forceinline__ void encode16(const float (&x)[16], float s, uint32_t (&w)[4]) {
  float v[16];
  if (fast_div_ok(s)) {
    const float r = __frcp_rn(s);
    const uint64_t r2 = pk(r, r), ns2 = pk(-s, -s);
#pragma unroll
    for (int i = 0; i < 8; ++i) upk(div2(pk(x[2 * i], x[2 * i + 1]), r2, ns2), v[2 * i], v[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fdiv_rn(x[i], s);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = cvt8x2<FMT>(v[4 * i], v[4 * i + 1]) | (cvt8x2<FMT>(v[4 * i + 2], v[4 * i + 3]) << 16);
}
template <int FMT>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
  float v[4];
  dec8x2<FMT>(w & 0xffffu, v[0], v[1]);
  dec8x2<FMT>(w >> 16, v[2], v[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(v[i], r);
  return cvt8x2<FMT>(v[0], v[1]) | (cvt8x2<FMT>(v[2], v[3]) << 16);
}

// The queries of kQTokens of the call's tokens, rotated: their positions are found once, then a thread takes 16
// elements of kQHeads heads (VEC), or a pair or an element past the pairs of one.  (A search by every thread: prompts
// of 11400 tokens in all 87 us, 64 of them here.)
constexpr int kQTokens = 2, kQHeads = 2;
template <int DT, bool VEC>
__device__ __forceinline__ void rotate_queries(const AppendArgs& a, int64_t cta) {
  __shared__ int64_t s_pos[kQTokens];
  constexpr int64_t kNone = INT64_MIN;
  const int64_t t0 = cta * kQTokens;
  const uint32_t units = static_cast<uint32_t>(a.q_units), groups = static_cast<uint32_t>(VEC ? (a.q_heads + kQHeads - 1) / kQHeads : a.q_heads);
  const uint32_t per_token = groups * units, last = static_cast<uint32_t>(min(static_cast<int64_t>(kQTokens), a.b.tokens - t0)) * per_token;
  float v[kQHeads][16];
  int o0 = 0, o1 = 0;
  const auto load = [&](uint32_t i) {  // item i: the rows are there whether or not they belong to a sequence
    const uint32_t k = i / per_token, j = i - k * per_token;
    unit_offsets<true>(a.r, static_cast<int>(j % units), o0, o1);
#pragma unroll
    for (int z = 0; z < kQHeads; ++z) {  // heads h, h + groups
      const int64_t from = (t0 + k) * a.ld_q + min(static_cast<int>(j / units + z * groups), a.q_heads - 1) * a.hd_q;
      load8<DT>(a.q, from + o0, v[z]);
      load8<DT>(a.q, from + o1, v[z] + 8);
    }
  };
  if (VEC && threadIdx.x < last) load(threadIdx.x);  // (on its way while the positions are found)
  if (threadIdx.x < kQTokens) s_pos[threadIdx.x] = kNone;
  __syncthreads();
  if (!a.b.starts) {
    if (threadIdx.x < kQTokens && t0 + threadIdx.x < a.b.tokens) s_pos[threadIdx.x] = static_cast<int64_t>(max(__ldg(a.b.lengths + t0 + threadIdx.x), 0)) - 1;
  } else {
    // every sequence is looked at by some thread, all at once: shorter than a search, whose loads wait for one another
    for (int32_t s = static_cast<int32_t>(threadIdx.x); s < a.b.seqs; s += kAppThreads) {
      const Span sp = span_of(a.b, s, a.c.page);
#pragma unroll
      for (int k = 0; k < kQTokens; ++k)
        if (t0 + k >= sp.row && t0 + k < static_cast<int64_t>(sp.row) + sp.n) s_pos[k] = sp.p0 + (t0 + k - sp.row);
    }
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < last; i += kAppThreads) {
    const uint32_t k = i / per_token, j = i - k * per_token;
    const int u = static_cast<int>(j % units), h0 = static_cast<int>(j / units);
    const int64_t pos = s_pos[k], t = t0 + k;
    if constexpr (VEC) {
      if (i >= kAppThreads) load(i);
      if (pos == kNone) continue;
      if (16 * u < 2 * a.r.pairs) {
        Turns turns;
        load_turns(a.r, u, pos, 1.0f, turns);
#pragma unroll
        for (int z = 0; z < kQHeads; ++z) turn_unit(a.r, turns, v[z]);
      }
#pragma unroll
      for (int z = 0; z < kQHeads; ++z) {
        const int h = h0 + z * static_cast<int>(groups);
        if (h >= a.q_heads) break;
        const int64_t to = t * a.ld_qo + h * a.hd_qo;
        store8v<DT>(a.q_out, to + o0, v[z]);
        store8v<DT>(a.q_out, to + o1, v[z] + 8);
      }
    } else {
      if (pos == kNone) continue;
      const int64_t from = t * a.ld_q + h0 * a.hd_q, to = t * a.ld_qo + h0 * a.hd_qo;
      if (u >= a.r.pairs) {
        store_elem<DT>(a.q_out, to + u + a.r.pairs, load_elem<DT>(a.q, from + u + a.r.pairs));
        continue;
      }
      const int d0 = a.r.interleaved ? 2 * u : u, d1 = a.r.interleaved ? d0 + 1 : u + a.r.pairs;
      float v0 = load_elem<DT>(a.q, from + d0), v1 = load_elem<DT>(a.q, from + d1);
      if (pos < 0 || pos >= a.r.positions) v0 = v1 = __uint_as_float(0x7fc00000u);
      else turn(v0, v1, __ldg(a.r.cos + pos * a.r.pairs + u), __ldg(a.r.sin + pos * a.r.pairs + u));
      store_elem<DT>(a.q_out, to + d0, v0);
      store_elem<DT>(a.q_out, to + d1, v1);
    }
  }
}

// Where a block's codes and scale lie: keys or values of kv head h, the block that begins at position b0.
struct BlockPlace {
  uint8_t* codes;
  float* scale;
};
__device__ __forceinline__ BlockPlace block_place(const AppendArgs& a, bool is_k, int64_t page, int h, int64_t b0) {
  const int in_page = static_cast<int>(b0 % a.c.page);
  const int64_t head = page * a.c.heads + h;
  return BlockPlace{(is_k ? a.c.k : a.c.v) + (head * a.c.page + in_page) * a.c.dim,
                    (is_k ? a.c.ks : a.c.vs) + head * (a.c.page >> a.c.log2_block) + (in_page >> a.c.log2_block)};
}
// 16 values of a token's vector (the piece of unit_offsets), the keys' rotated
template <int DT, bool VEC>
__device__ __forceinline__ void load_piece(const RotaryView& r, const void* src, int64_t base, int u, int64_t pos, float (&x)[16]) {
  if constexpr (VEC) {
    int o0, o1;
    unit_offsets<true>(r, u, o0, o1);
    load8<DT>(src, base + o0, x);
    load8<DT>(src, base + o1, x + 8);
    if (r.cos && 16 * u < 2 * r.pairs) {
      Turns turns;
      load_turns(r, u, pos, 1.0f, turns);
      turn_unit(r, turns, x);
    }
  } else {
#pragma unroll 1
    for (int j = 0; j < 16; ++j) {
      const float v = turned<DT>(r, src, base, 16 * u + j, pos, 1.0f);
#pragma unroll
      for (int q = 0; q < 16; ++q) x[q] = q == j ? v : x[q];
    }
  }
}
template <int FMT>
__device__ __forceinline__ uint4 rescale16(uint4 w, float ratio, bool bad) {
  w.x = rescale4<FMT>(w.x, ratio);
  w.y = rescale4<FMT>(w.y, ratio);
  w.z = rescale4<FMT>(w.z, ratio);
  w.w = rescale4<FMT>(w.w, ratio);
  return bad ? make_uint4(0u, 0u, 0u, 0u) : w;
}

// One new token a sequence: a warp for its keys or values of one head.  (By the kernel below, 128 sequences of 8 heads:
// 12.4 us, four rounds of CTAs with little to do.)
template <int FMT, int DT, bool VEC>
__global__ void __launch_bounds__(kAppThreads) append_one_kernel(const AppendArgs a) {
  if (blockIdx.x >= a.kv_ctas) {
    rotate_queries<DT, VEC>(a, blockIdx.x - a.kv_ctas);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kAppWarps + (threadIdx.x >> 5);
  const bool is_k = !(item & 1);
  const int h = static_cast<int>((item >> 1) % a.c.heads);
  const int64_t s = (item >> 1) / a.c.heads;
  if (s >= a.b.seqs) return;
  const Span sp = span_of(a.b, static_cast<int32_t>(s), a.c.page);
  const int64_t pos = sp.p0;
  if (pos < 0 || pos >= sp.len || (a.r.cos && pos >= a.r.positions)) return;
  const int64_t b0 = pos >> a.c.log2_block << a.c.log2_block;
  RotaryView r = a.r;
  if (!is_k) r.cos = nullptr;
  const int units = a.c.dim / 16;  // 16 at most
  float x[16], amax = 0.0f;
  if (lane < units) load_piece<DT, VEC>(r, is_k ? a.k : a.v, s * (is_k ? a.ld_k : a.ld_v) + h * (is_k ? a.hd_k : a.hd_v), lane, pos, x);
  const int64_t page = page_of(a.b, a.c, static_cast<int32_t>(s), static_cast<int32_t>(b0));
  if (page < 0) return;
  const BlockPlace p = block_place(a, is_k, page, h, b0);
  const float old = pos > b0 ? *p.scale : 0.0f;
  if (lane < units) {
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = absmax_nan(amax, x[j]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = absmax_nan(amax, __shfl_xor_sync(kFull, amax, o));
  const float now = absmax_nan(__fdiv_rn(amax, Fmt8<FMT>::kMax), old);
  const bool bad = !is_finite_f(now), zero = now == 0.0f;
  if (lane == 0) *p.scale = now;
  if (lane < units) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (!bad && !zero) encode16<FMT>(x, now, w);
    int o0, o1;
    unit_offsets<VEC>(r, lane, o0, o1);
    uint8_t* row = p.codes + (pos - b0) * a.c.dim;
    *reinterpret_cast<uint2*>(row + o0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(row + o1) = make_uint2(w[2], w[3]);
  }
  if (pos > b0 && (bad || now > old)) {
    const float ratio = bad || zero ? 0.0f : __fdiv_rn(old, now);
    uint4* held = reinterpret_cast<uint4*>(p.codes);
#pragma unroll 4
    for (int i = lane; i < (pos - b0) * units; i += 32) held[i] = rescale16<FMT>(held[i], ratio, bad);
  }
}

// The two 8-value pieces of unit u as they lie in memory, and as rotated fp32 values.
template <int DT>
struct RawPiece {
  uint4 w[DT == QZ_BF16 ? 2 : 4];
};
template <int DT>
__device__ __forceinline__ RawPiece<DT> load_raw(const RotaryView& r, const void* src, int64_t base, int u) {
  int o0, o1;
  unit_offsets<true>(r, u, o0, o1);
  RawPiece<DT> p;
  if constexpr (DT == QZ_BF16) {
    const uint16_t* x = static_cast<const uint16_t*>(src) + base;
    p.w[0] = ld16B(x + o0), p.w[1] = ld16B(x + o1);
  } else {
    const float* x = static_cast<const float*>(src) + base;
    p.w[0] = ld16B(x + o0), p.w[1] = ld16B(x + o0 + 4), p.w[2] = ld16B(x + o1), p.w[3] = ld16B(x + o1 + 4);
  }
  return p;
}
template <int DT>
__device__ __forceinline__ void open_raw(const RotaryView& r, const RawPiece<DT>& p, int u, int64_t pos, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < (DT == QZ_BF16 ? 2 : 4); ++i) {
    const uint32_t w[4] = {p.w[i].x, p.w[i].y, p.w[i].z, p.w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == QZ_BF16) {
        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      } else {
        x[4 * i + j] = __uint_as_float(w[j]);
      }
    }
  }
  if (r.cos && 16 * u < 2 * r.pairs) {
    Turns turns;
    load_turns(r, u, pos, 1.0f, turns);
    turn_unit(r, turns, x);
  }
}

// Keys and values of one block of one kv head.  R: pieces of 16 values a thread.  The values are held as they were
// loaded and rotated twice, for the amax and for the codes: the registers go to loads in flight.  (Held rotated, keys and
// values by a CTA each: 39 us for 11400 tokens of 8 heads, without the queries.)  Where they would not fit, and where they
// take single loads, they are loaded again instead.
template <int FMT, int DT, int R, bool VEC>
__global__ void __launch_bounds__(kAppThreads) append_kernel(const AppendArgs a) {
  constexpr bool kHold = VEC && R * (DT == QZ_BF16 ? 1 : 2) <= 4;
  __shared__ float warp_amax[2][kAppWarps];
  if (blockIdx.x >= a.kv_ctas) {
    rotate_queries<DT, VEC>(a, blockIdx.x - a.kv_ctas);
    return;
  }
  const int h = static_cast<int>(blockIdx.x % static_cast<uint32_t>(a.c.heads));
  const int64_t slot = blockIdx.x / static_cast<uint32_t>(a.c.heads);
  const int block = a.c.block, lb = a.c.log2_block;
  const auto first_slot = [&](int32_t s) { return static_cast<int64_t>(start_of(a.b, s) >> lb) + 2 * static_cast<int64_t>(s); };
  const int32_t s = count_upto(a.b.seqs, first_slot, slot) - 1;
  if (s < 0) return;
  const Span sp = span_of(a.b, s, a.c.page);
  const int64_t first_new = sp.p0 > 0 ? sp.p0 : 0;
  const int64_t b0 = ((first_new >> lb) + slot - first_slot(s)) << lb;  // the block's first position
  const int64_t new0 = first_new > b0 ? first_new : b0;
  int64_t end = b0 + block < sp.len ? b0 + block : sp.len;
  if (a.r.cos && end > a.r.positions) end = a.r.positions;
  if (new0 >= end) return;
  // unit i: token i / units of the block, elements of unit i % units
  const int units = a.c.dim / 16, total = block * units;
  const int from = static_cast<int>(new0 - b0), to = static_cast<int>(end - b0);  // the new tokens' places
  const auto base = [&](int z, int t) { return (sp.row + (b0 + t - sp.p0)) * (z ? a.ld_v : a.ld_k) + h * (z ? a.hd_v : a.hd_k); };
  RotaryView none = a.r;
  none.cos = nullptr;
  int token[R], unit[R];
  RawPiece<DT> raw[kHold ? 2 : 1][kHold ? R : 1];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int i = static_cast<int>(threadIdx.x) + k * kAppThreads;
    token[k] = i / units, unit[k] = i - token[k] * units;
    if (i >= total) token[k] = -1;
    if constexpr (kHold) {
      if (token[k] >= from && token[k] < to) {
        raw[0][k] = load_raw<DT>(a.r, a.k, base(0, token[k]), unit[k]);
        raw[1][k] = load_raw<DT>(none, a.v, base(1, token[k]), unit[k]);
      }
    }
  }
  const int64_t page = page_of(a.b, a.c, s, static_cast<int32_t>(b0));
  if (page < 0) return;
  const auto values = [&](int z, int k, float (&x)[16]) {
    const RotaryView& r = z ? none : a.r;
    if constexpr (kHold) open_raw<DT>(r, raw[z][k], unit[k], b0 + token[k], x);
    else load_piece<DT, VEC>(r, z ? a.v : a.k, base(z, token[k]), unit[k], b0 + token[k], x);
  };
  float amax[2] = {0.0f, 0.0f}, old[2];
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const BlockPlace place = block_place(a, z == 0, page, h, b0);
    old[z] = from > 0 ? *place.scale : 0.0f;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (token[k] < from || token[k] >= to) continue;
      float x[16];
      values(z, k, x);
#pragma unroll
      for (int j = 0; j < 16; ++j) amax[z] = absmax_nan(amax[z], x[j]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax[z] = absmax_nan(amax[z], __shfl_xor_sync(kFull, amax[z], o));
    if ((threadIdx.x & 31u) == 0) warp_amax[z][threadIdx.x >> 5] = amax[z];
  }
  __syncthreads();  // (every thread has read the old scales by now, too)
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const BlockPlace place = block_place(a, z == 0, page, h, b0);
#pragma unroll
    for (int w = 0; w < kAppWarps; ++w) amax[z] = absmax_nan(amax[z], warp_amax[z][w]);
    const float now = absmax_nan(__fdiv_rn(amax[z], Fmt8<FMT>::kMax), old[z]);
    if (threadIdx.x == 0) *place.scale = now;
    const bool bad = !is_finite_f(now), zero = now == 0.0f, grown = from > 0 && (bad || now > old[z]);
    const float ratio = bad || zero ? 0.0f : __fdiv_rn(old[z], now);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (token[k] < 0) break;
      uint8_t* row = place.codes + static_cast<int64_t>(token[k]) * a.c.dim;
      if (token[k] >= from && token[k] < to) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (!bad && !zero) {
          float x[16];
          values(z, k, x);
          encode16<FMT>(x, now, w);
        }
        int o0, o1;
        unit_offsets<VEC>(z ? none : a.r, unit[k], o0, o1);
        *reinterpret_cast<uint2*>(row + o0) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(row + o1) = make_uint2(w[2], w[3]);
      } else if (token[k] < from && grown) {
        uint4* p = reinterpret_cast<uint4*>(row + 16 * unit[k]);
        *p = rescale16<FMT>(*p, ratio, bad);
      }
    }
  }
}

// The queries alone, beside prompts: their kernel takes half the registers.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kAppThreads) append_queries_kernel(const AppendArgs a) { rotate_queries<DT, VEC>(a, blockIdx.x); }

template <int FMT, int DT, bool VEC>
void run_append(const AppendArgs& a, unsigned grid, unsigned q_grid, cudaStream_t s) {
  if (q_grid) append_queries_kernel<DT, VEC><<<q_grid, kAppThreads, 0, s>>>(a);
  if (grid == 0) return;
  const int pieces = a.c.block * (a.c.dim / 16);
  if (!a.b.starts) append_one_kernel<FMT, DT, VEC><<<grid, kAppThreads, 0, s>>>(a);
  else if (pieces <= kAppThreads) append_kernel<FMT, DT, 1, VEC><<<grid, kAppThreads, 0, s>>>(a);
  else if (pieces <= 2 * kAppThreads) append_kernel<FMT, DT, 2, VEC><<<grid, kAppThreads, 0, s>>>(a);
  else if (pieces <= 4 * kAppThreads) append_kernel<FMT, DT, 4, VEC><<<grid, kAppThreads, 0, s>>>(a);
  else append_kernel<FMT, DT, 8, VEC><<<grid, kAppThreads, 0, s>>>(a);
}
template <int FMT>
void run_append(const AppendArgs& a, int dtype, bool vec, unsigned grid, unsigned q_grid, cudaStream_t s) {
  if (dtype == QZ_BF16) vec ? run_append<FMT, QZ_BF16, true>(a, grid, q_grid, s) : run_append<FMT, QZ_BF16, false>(a, grid, q_grid, s);
  else vec ? run_append<FMT, QZ_F32, true>(a, grid, q_grid, s) : run_append<FMT, QZ_F32, false>(a, grid, q_grid, s);
}

}  // namespace

qz_status check_cache(const qz_cache* c) {
  if (!c) return QZ_ERR_NULL;
  if (c->format != QZ_INT8 && c->format != QZ_FP8_E4M3 && c->format != QZ_FP8_E5M2) return QZ_ERR_ENUM;
  if (c->pages < 0 || c->kv_heads <= 0 || c->page <= 0 || c->dim <= 0) return QZ_ERR_SHAPE;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return QZ_ERR_UNSUPPORTED;
  if (c->page > 1024 || c->dim > 256 || c->dim % 16) return QZ_ERR_UNSUPPORTED;
  if (c->page % c->block) return QZ_ERR_SHAPE;
  if (c->kv_heads > 65535 || c->pages > INT32_MAX / c->kv_heads) return QZ_ERR_UNSUPPORTED;
  if (c->pages > 0 && (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales)) return QZ_ERR_NULL;
  if (!is_aligned(c->k_codes, 16) || !is_aligned(c->v_codes, 16) || !is_aligned(c->k_scales, 4) || !is_aligned(c->v_scales, 4))
    return QZ_ERR_ALIGN;
  return QZ_OK;
}

qz_status check_batch(const qz_batch* b, int64_t tokens) {
  if (!b) return QZ_ERR_NULL;
  if (b->sequences < 0 || b->table_pages < 0 || b->ld_table < b->table_pages) return QZ_ERR_SHAPE;
  if (b->sequences > (1 << 24) || b->table_pages > (1 << 24) || tokens > (1 << 30)) return QZ_ERR_UNSUPPORTED;
  if (b->sequences > 0 && b->ld_table > INT64_MAX / 8 / b->sequences) return QZ_ERR_SHAPE;
  if (!b->starts && tokens != b->sequences) return QZ_ERR_SHAPE;
  if (b->sequences > 0 && tokens > 0 && (!b->lengths || (!b->table && b->table_pages > 0))) return QZ_ERR_NULL;
  if (!is_aligned(b->table, 4) || !is_aligned(b->lengths, 4) || !is_aligned(b->starts, 4)) return QZ_ERR_ALIGN;
  return QZ_OK;
}

CacheView view_of(const qz_cache& c) {
  CacheView v{};
  v.k = static_cast<uint8_t*>(c.k_codes), v.v = static_cast<uint8_t*>(c.v_codes);
  v.ks = c.k_scales, v.vs = c.v_scales;
  v.pages = c.pages;
  v.heads = c.kv_heads, v.page = c.page, v.block = c.block, v.dim = c.dim;
  v.log2_block = c.block == 16 ? 4 : c.block == 32 ? 5 : c.block == 64 ? 6 : 7;
  return v;
}
BatchView view_of(const qz_batch& b, int64_t tokens) {
  BatchView v{};
  v.table = b.table, v.lengths = b.lengths, v.starts = b.starts;
  v.ld_table = b.ld_table;
  v.seqs = static_cast<int32_t>(b.sequences), v.table_pages = static_cast<int32_t>(b.table_pages);
  v.tokens = static_cast<int32_t>(tokens);
  return v;
}

}  // namespace qz

using namespace qz;

extern "C" qz_status qz_cache_append(const qz_cache* cache, const qz_batch* batch, int32_t dtype, const void* k, int64_t ld_k,
                                     int64_t hd_k, const void* v, int64_t ld_v, int64_t hd_v, int64_t tokens,
                                     const qz_rotary_table* table, const void* q, int64_t ld_q, int64_t hd_q, int64_t heads,
                                     void* q_out, int64_t ld_qo, int64_t hd_qo, qz_stream_t stream) {
  qz_status st;
  if ((st = check_cache(cache)) != QZ_OK) return st;
  if (dtype != QZ_BF16 && dtype != QZ_F32) return QZ_ERR_ENUM;
  const int64_t kv = cache->kv_heads, dim = cache->dim;
  if ((st = check_vectors(tokens, kv, dim, ld_k, hd_k)) != QZ_OK || (st = check_vectors(tokens, kv, dim, ld_v, hd_v)) != QZ_OK ||
      (st = check_batch(batch, tokens)) != QZ_OK)
    return st;
  if (table && (st = check_rotary_table(table, dim)) != QZ_OK) return st;
  if ((q == nullptr) != (q_out == nullptr) || (q && !table)) return QZ_ERR_NULL;
  if (q && ((st = check_vectors(tokens, heads, dim, ld_q, hd_q)) != QZ_OK || (st = check_vectors(tokens, heads, dim, ld_qo, hd_qo)) != QZ_OK))
    return st;
  if (q && (heads % kv || moves_in_place(q, ld_q, hd_q, q_out, ld_qo, hd_qo, tokens, heads))) return QZ_ERR_SHAPE;
  if (tokens == 0 || batch->sequences == 0) return QZ_OK;
  if (!k || !v) return QZ_ERR_NULL;
  const int64_t e = dtype == QZ_BF16 ? 2 : 4;
  if (!is_aligned(k, e) || !is_aligned(v, e) || !is_aligned(q, e) || !is_aligned(q_out, e)) return QZ_ERR_ALIGN;
  AppendArgs a{};
  a.c = view_of(*cache);
  a.b = view_of(*batch, tokens);
  a.r = view_of(table);
  a.k = k, a.v = v, a.q = q, a.q_out = q_out;
  a.ld_k = ld_k, a.hd_k = hd_k, a.ld_v = ld_v, a.hd_v = hd_v;
  a.ld_q = ld_q, a.hd_q = hd_q, a.ld_qo = ld_qo, a.hd_qo = hd_qo;
  const bool vec = (!a.r.cos || rotary_vec(a.r, dim)) && rows_vec(k, e, tokens, ld_k, kv, hd_k) && rows_vec(v, e, tokens, ld_v, kv, hd_v) &&
                   (!q || (rows_vec(q, e, tokens, ld_q, heads, hd_q) && rows_vec(q_out, e, tokens, ld_qo, heads, hd_qo)));
  const int64_t slots = cache->pages == 0 ? 0 : batch->starts ? tokens / cache->block + 2 * batch->sequences : batch->sequences;
  a.q_heads = static_cast<int32_t>(heads);
  a.q_units = static_cast<int32_t>(vec ? dim / 16 : dim - a.r.pairs);
  const int64_t q_ctas = q && heads ? (tokens + kQTokens - 1) / kQTokens : 0;
  if (slots > INT32_MAX / kv / 2) return QZ_ERR_UNSUPPORTED;
  const int64_t kv_ctas = batch->starts ? slots * kv : (2 * slots * kv + kAppWarps - 1) / kAppWarps, ctas = kv_ctas + q_ctas;
  if (ctas > INT32_MAX) return QZ_ERR_UNSUPPORTED;
  if (ctas == 0) return QZ_OK;
  a.kv_ctas = static_cast<uint32_t>(kv_ctas);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool apart = batch->starts && tokens >= kApart;
  const unsigned grid = static_cast<unsigned>(apart ? kv_ctas : ctas), q_grid = static_cast<unsigned>(apart ? q_ctas : 0);
  if (cache->format == QZ_INT8) run_append<QZ_INT8>(a, dtype, vec, grid, q_grid, s);
  else if (cache->format == QZ_FP8_E4M3) run_append<QZ_FP8_E4M3>(a, dtype, vec, grid, q_grid, s);
  else run_append<QZ_FP8_E5M2>(a, dtype, vec, grid, q_grid, s);
  return launch_status();
}
