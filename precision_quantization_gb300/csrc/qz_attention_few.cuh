// qz_attention_few.cuh -- attention of a few rows to the 8-bit cache (decoding), included once per format.
//
//   x_j = (scale log2 e) ks_j (q . k_j),  m = max x_j,  p_j = 2^(x_j - m),  l = sum p_j,
//   out = sum p_j vs_j v_j / l        (k_j, v_j the codes, ks_j, vs_j their block's scales)
//
// Bound by HBM: every code is read once and meets up to 32 rows.  So the codes stream and everything else
// has to fit beside them: a warp has a ring of its own that TMA fills, a step of 32 tokens (of more than 128
// elements: 16) a stage, in the hardware's swizzle.  Keys and values are the products' A operands,
//   x^T [tokens][rows] = K q^T,   out^T [elements][rows] += V^T p^T,
// so that eight rows, what a kv head's group often has, fill the operand of eight columns, and what was
// decoded for one column tile serves them all.  The summation index of K q^T and the rows of V^T may be
// permuted; with lane (g, c) = (lane / 4, lane % 4)
//   keys    rows g and g + 8 of 16, bytes 64 h + 16 c .. + 15: four 16-wide products,
//   values  rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9, bytes w g .. w g + w - 1 (w = dim / 8): w / 2 products
// are whole 16-byte pieces, read from different banks.  8-bit codes are exact in f16, q is made f16 by a
// power of two of its row.  The weights p vs are made f16 times 2^15 / unit, unit a power of two of the row's, above
// every vs that it has seen so far, so that a weight far below the largest scale keeps its 11 bits (down to 2^-28 of
// it); a transpose of 8 x 8 (movmatrix) makes them operands.
//
// The work is cut in equal shares of steps over a persistent grid, whatever the lengths are (they lie on
// the GPU): item after item (sequence, kv head, row tile), a CTA's share begins and ends anywhere.  A share
// that holds part of an item leaves its sums in the workspace, and the CTAs of the second kernel join them.
//
// GPU times (in brackets the bytes of the visible keys and values at the copy rate, 6.7 TB/s):
//   64 sequences x 1 token, up to 8192 long, 32 / 8 heads x 128, INT8    158 us (123), 5.2 TB/s
//   1 token of 131072, 64 / 8 heads x 128, E4M3                          58 us (40), 4.6 TB/s
//   24 sequences x 3 tokens, window 4096, 40 / 8 heads x 64, E5M2        57 us (15)
//   1 token of 517                                                       9.4 us
// Between 60 and 80 % of HBM no pipe is full (the decoding ALU 58 %, issue 0.5 to 0.6 a cycle): three warps a
// scheduler wait for fixed latencies.  With 15 rows of 64 elements (the third) a code meets twice the softmax and half
// the products; its warps wait most of the time too (issue 0.47, HBM 24 %), with the joins at the ends of items.  Codes
// as the B operand, rows as A, took 226 and 80 us; rings filled by cp.async 240 and 84.  Units by what a row sees, and
// the look for codes that are no finite numbers, cost 1 % of the first two and 5 us of the third.
#pragma once

#include <type_traits>

#include "qz_attention.cuh"
#include "qz_internal.h"
#include "qz_tcgen05.cuh"

namespace qz {
namespace {

constexpr uint64_t kFewWaitNs = 1000000000ull;  // 1 s: far beyond any copy's latency

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the transpose of an 8 x 8 matrix of 16-bit values, row g's columns 2 c and 2 c + 1 in lane (g, c)
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
// one 4-byte value, announced on the barrier like the lane's own arrival
__device__ __forceinline__ void copy_scale(uint32_t dst, const float* src, uint32_t bar) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Bounded wait for a step.  After one of the CTA's warps has given up no other waits long: the CTA's results are NaN.
// (The flag is looked at where a wait is long already; a test before each wait costs registers, and 64 x 1 token 2 to 4 us.)
__device__ __forceinline__ bool step_wait(uint32_t bar, uint32_t parity, volatile int& gave_up) {
  if (held_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!held_try_wait(bar, parity)) {
    if (gave_up || globaltimer_ns() - t0 > kFewWaitNs) {
      gave_up = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void arrive_on(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void lds16(uint32_t (&w)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}

// ---- sizes --------------------------------------------------------------------------------------
// DP: dim rounded up to 64, 128 or 256; NT: tiles of 8 rows.
template <int DP, int NT>
struct FewSizes {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStep = few_att_step(DP), kHalves = kStep / 16;   // tokens of a step, in 16s
  // the sums take NT DP / 4 registers a thread: twelve warps where they leave room for the rest
  static constexpr int kWarps = NT == 1 || NT * DP == 128 ? 12 : 8, kThreads = 32 * kWarps;
  static constexpr uint32_t kHalf = 16 * DP;                             // bytes of 16 tokens' keys or values
  static constexpr uint32_t kStage = 2 * kHalves * kHalf;                // keys, then values
  static constexpr uint32_t kQ = NT * (DP / 16) * 256;                   // q as B operands
  static constexpr int kJoinCols = NT == 1 ? 64 : 32;                    // columns joined at a time
  static constexpr uint32_t kJoin = kWarps * kRows * kJoinCols * 4;
  static constexpr int kRoom = 226 * 1024 - 1024 - 4096 - static_cast<int>(kQ + kJoin);  // 4 KiB: static
  static constexpr int kStages = kRoom / static_cast<int>(kWarps * kStage) < 4 ? kRoom / static_cast<int>(kWarps * kStage) : 4;
  static_assert(kStages >= 2);
  static constexpr uint32_t kRing = kWarps * kStages * kStage;
  static constexpr uint32_t kSmem = kRing + kQ + kJoin + 1024;           // (the ring starts on a 1024-byte boundary)
  static constexpr int kSlot = kRows * (DP + 2);                         // floats of a partial result: sums, m, l
};
struct FewMeta {     // an item that begins in a CTA's share and does not end there
  int32_t seq, head, row0, last;   // last: the CTA whose share holds its end; seq < 0: none
};

// ---- the work -----------------------------------------------------------------------------------
struct SeqWork {
  Span sp;
  int32_t tiles;       // row tiles
  int32_t step0, steps;  // the steps that any of its rows may see (whole items: 1 unit an item)
};
__device__ __forceinline__ SeqWork seq_work(const AttentionArgs& a, int32_t s, int rows, int step) {
  SeqWork w;
  w.sp = span_of(a.b, s, a.c.page);
  w.tiles = static_cast<int32_t>((static_cast<int64_t>(w.sp.n) * a.group + rows - 1) / rows);
  const int64_t lo = w.sp.p0 + 1 - a.window;
  w.step0 = lo > 0 ? static_cast<int32_t>(lo / step) : 0;
  w.steps = max(static_cast<int32_t>((static_cast<int64_t>(w.sp.len) + step - 1) / step) - w.step0, 1);
  return w;
}
__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// A segment: the part of an item that lies in this CTA's share.
struct Segment {
  SeqWork w;
  int32_t seq, kvh, row0, rows;
  int32_t t0, t1;        // its steps
  int64_t item_u0;       // the item's first unit
};

template <int FMT, int DP, int NT, bool WHOLE>
__global__ void __launch_bounds__(FewSizes<DP, NT>::kThreads, 1)
    attention_few_kernel(const AttentionArgs a, const __grid_constant__ CacheMaps maps, int grid, int min_chunk) {
  using Z = FewSizes<DP, NT>;
  constexpr int kRows = Z::kRows, kStages = Z::kStages, kStep = Z::kStep, kHalves = Z::kHalves, kWarps = Z::kWarps;
  constexpr int kSteps16 = DP / 16, kCols = DP / 8, kTiles = DP / 16;  // products of a sum, columns of a lane, tiles of 16 elements
  constexpr int kPieces = DP == 256 ? 2 : 1;    // 16-byte pieces of a lane's columns; 4-element ones of its part of a row of q
  constexpr bool kHeld = NT * DP <= 128;        // q in registers, else read from shared memory for each step
  constexpr uint32_t kRowBytes = DP < 128 ? 64 : 128, kSlab = kStep * kRowBytes;  // a box's row, and a step's boxes of one x
  extern __shared__ uint8_t few_raw[];
  __shared__ int64_t s_scan[kWarps + 1], s_found[2];
  __shared__ float s_fq[kRows], s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ float s_unit[kWarps][kRows], s_shrink[kWarps][kRows];  // (in registers: spills with four row tiles)
  __shared__ int32_t s_end[kRows], s_begin[kRows];
  __shared__ float s_top[kRows], s_sum[kRows];
  __shared__ __align__(16) float s_scale[kWarps][kStages][4];  // ks, vs of the first 16 tokens, of the second
  __shared__ int32_t s_has[kWarps][kStages];                   // bit i: the i-th 16 tokens have a page
  __shared__ __align__(8) uint64_t s_full[kWarps][kStages];
  __shared__ uint32_t s_spoiled[kWarps];  // tokens of a step, seen by some rows alone, whose values are not finite numbers
  __shared__ volatile int s_gave_up;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const uint32_t base = (smem_addr(few_raw) + 1023u) & ~1023u;
  uint8_t* smem = few_raw + (base - smem_addr(few_raw));
  const uint32_t ring = base + warp * (kStages * Z::kStage);
  const uint32_t q_smem = base + Z::kRing;
  float* join = reinterpret_cast<float*>(smem + Z::kRing + Z::kQ);
  if (tid == 0) s_gave_up = 0;
  // 0 at a segment's start; NaN where a row sees a value that is no finite number
  for (int r = lane; r < kRows; r += 32) s_l[warp][r] = 0.0f;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(smem_addr(&s_full[warp][i]), 1 + 2 * kHalves);  // the codes, the scales
    mbar_init_fence();
  }

  // ---- this CTA's share: units [u0, u1) of the sequences' work one after the other ---------------
  const auto work_of = [&](const SeqWork& w) { return static_cast<int64_t>(w.tiles) * a.c.heads * (WHOLE ? 1 : w.steps); };
  const auto units_of = [&](int32_t s) { return s < a.b.seqs ? work_of(seq_work(a, s, kRows, kStep)) : 0; };
  int64_t u0, u1, chunk = 1, before = 0;
  const bool few = a.b.seqs <= Z::kThreads;  // one look at the lengths does
  int64_t mine = few || !WHOLE ? units_of(tid) : 0;
  if (!WHOLE) {
    int64_t sum = mine;
    for (int32_t s = tid + Z::kThreads; s < a.b.seqs; s += Z::kThreads) sum += units_of(s);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0) s_scan[warp] = sum;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += s_scan[w];
    __syncthreads();
    chunk = max((total + grid - 1) / grid, static_cast<int64_t>(min_chunk));
    u0 = blockIdx.x * chunk;
    u1 = min(u0 + chunk, total);
    if (tid == 0) static_cast<FewMeta*>(a.ws)[blockIdx.x].seq = -1;
  } else {
    u0 = blockIdx.x;
    u1 = u0 + 1;
  }
  if (u0 >= u1) return;
  bool found = false;  // the sequence that holds unit u0
  for (int32_t s0 = 0; s0 < a.b.seqs && !found; s0 += Z::kThreads) {
    if (!few) mine = units_of(s0 + tid);
    const int64_t in_warp = warp_scan(mine, lane);
    if (lane == 31) s_scan[warp] = in_warp;
    __syncthreads();
    int64_t at = before + in_warp, all = before;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += s_scan[w];
      all += s_scan[w];
    }
    if (u0 < at && u0 >= at - mine) {
      s_found[0] = s0 + tid;
      s_found[1] = at - mine;
    }
    found = u0 < all;
    before = all;
    __syncthreads();
  }
  if (!found) return;  // (whole items: the grid covers the most that there can be)
  before = s_found[1];
  float* slots = reinterpret_cast<float*>(static_cast<char*>(a.ws) + static_cast<size_t>(grid) * sizeof(FewMeta));

  int64_t u = u0;
  Segment n;  // the next segment
  n.seq = static_cast<int32_t>(s_found[0]);
  n.w = seq_work(a, n.seq, kRows, kStep);
  const auto advance = [&]() -> bool {
    if (u >= u1) return false;
    while (u >= before + work_of(n.w)) {
      before += work_of(n.w);
      if (++n.seq >= a.b.seqs) return false;  // (not reached while the lengths stay as they are)
      n.w = seq_work(a, n.seq, kRows, kStep);
    }
    const int64_t in_seq = u - before, item = WHOLE ? in_seq : in_seq / n.w.steps;
    n.t0 = WHOLE ? 0 : static_cast<int32_t>(in_seq - item * n.w.steps);
    n.t1 = WHOLE ? n.w.steps : static_cast<int32_t>(min(static_cast<int64_t>(n.w.steps), n.t0 + (u1 - u)));
    n.kvh = static_cast<int32_t>(item / n.w.tiles);
    n.row0 = static_cast<int32_t>(item % n.w.tiles) * kRows;
    n.rows = static_cast<int32_t>(min(static_cast<int64_t>(kRows), static_cast<int64_t>(n.w.sp.n) * a.group - n.row0));
    n.item_u0 = u - n.t0;
    u += WHOLE ? 1 : n.t1 - n.t0;
    return true;
  };

  // ---- the copies of this warp's steps, a ring ahead ---------------------------------------------
  // the next step and the end; the next 16 tokens' position, their page's place in the table and first row there
  int32_t ct = 0, c_end = 0, c_index = 0, c_in = 0, c_page = -1, c_stage = 0, c_len = 0, c_kvh = 0;
  int64_t c_pos = 0;
  const int32_t* c_row = nullptr;
  const auto entry = [&]() { return c_pos < c_len ? __ldg(c_row + c_index) : -1; };
  const auto aim = [&](const Segment& s) {  // at a segment's steps: a run of them for each warp
    const int32_t count = s.t1 - s.t0;
    ct = s.t0 + static_cast<int32_t>(static_cast<int64_t>(count) * warp / kWarps);
    c_end = s.t0 + static_cast<int32_t>(static_cast<int64_t>(count) * (warp + 1) / kWarps);
    c_pos = (static_cast<int64_t>(s.w.step0) + ct) * kStep;
    c_index = static_cast<int32_t>(c_pos / a.c.page);
    c_in = static_cast<int32_t>(c_pos - static_cast<int64_t>(c_index) * a.c.page);
    c_row = a.b.table + s.seq * a.b.ld_table;
    c_len = s.w.sp.len;
    c_kvh = s.kvh;
    c_page = ct < c_end ? entry() : -1;
  };
  const auto copy = [&]() {  // one step, into c_stage
    if (ct >= c_end) return;
    ++ct;
    const uint32_t bar = smem_addr(&s_full[warp][c_stage]), to = ring + c_stage * Z::kStage;
    int32_t page[kHalves], in[kHalves];
#pragma unroll
    for (int i = 0; i < kHalves; ++i) {
      page[i] = static_cast<uint32_t>(c_page) < static_cast<uint32_t>(a.c.pages) ? c_page : -1;
      if (c_pos >= c_len) page[i] = -1;
      in[i] = c_in;
      c_pos += 16;
      c_in += 16;
      if (c_in == a.c.page) {
        c_in = 0;
        ++c_index;
        c_page = entry();
      }
    }
    if (lane < 2 * kHalves) {
      const int i = kHalves == 2 ? lane >> 1 : 0;
      const int32_t pg = kHalves == 2 && i ? page[kHalves - 1] : page[0], at = kHalves == 2 && i ? in[kHalves - 1] : in[0];
      if (pg >= 0) {
        const int64_t block = (static_cast<int64_t>(pg) * a.c.heads + c_kvh) * (a.c.page >> a.c.log2_block) + (at >> a.c.log2_block);
        copy_scale(smem_addr(&s_scale[warp][c_stage][lane]), ((lane & 1) ? a.c.vs : a.c.ks) + block, bar);
      } else {
        arrive_on(bar);
      }
    }
    if (lane == 0) {
      int32_t has = 0;
#pragma unroll
      for (int i = 0; i < kHalves; ++i) has |= (page[i] >= 0 ? 1 : 0) << i;
      s_has[warp][c_stage] = has;
      if (has) {
        mbar_expect_tx(bar, (kHalves == 2 && has == 3 ? 2u : 1u) * 2u * Z::kHalf);
#pragma unroll
        for (int i = 0; i < kHalves; ++i) {
          if (page[i] < 0) continue;
          const int32_t head = page[i] * a.c.heads + c_kvh;
#pragma unroll
          for (int h = 0; h < kPieces; ++h) {
            box_load(to + h * kSlab + i * (16 * kRowBytes), &maps.k, 128 * h, in[i], head, bar);
            box_load(to + kHalves * Z::kHalf + h * kSlab + i * (16 * kRowBytes), &maps.v, 128 * h, in[i], head, bar);
          }
        }
      } else {
        arrive_on(bar);
      }
    }
    c_stage = c_stage + 1 == kStages ? 0 : c_stage + 1;
  };
  // this warp's rows of the next segment's q, on their way before its codes are asked for (behind those they take
  // four times as long)
  constexpr int kQRows = (kRows + kWarps - 1) / kWarps;
  uint2 q_next[kQRows][kPieces];
  const auto ask_q = [&](const Segment& s) {
#pragma unroll
    for (int j = 0; j < kQRows; ++j) {
      const int r = warp + j * kWarps, i = (s.row0 + r) / a.group, head = s.kvh * a.group + (s.row0 + r) - i * a.group;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int d = 4 * (lane + 32 * k);
        q_next[j][k] = load_q4_raw(a, r < s.rows && d < a.c.dim, (s.w.sp.row + i) * a.ld_q + head * a.hd_q + d);
      }
    }
  };
  int stage = 0;
  uint32_t phase = 0;
  bool failed = false;   // a wait has given up: this CTA's results are NaN
  __syncwarp();
  bool more = advance();
  if (more) {
    ask_q(n);
    aim(n);
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) copy();
  }

  while (more) {
    const Segment s = n;
    // ---- q as f16 B operands, row by row; what each row sees ------------------------------------
#pragma unroll
    for (int j = 0; j < kQRows; ++j) {
      const int r = warp + j * kWarps, i = (s.row0 + r) / a.group;
      if (r >= kRows) break;
      float x[kPieces][4];
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const uint2 b = q_next[j][k];
        x[k][0] = __uint_as_float(b.x << 16), x[k][1] = __uint_as_float(b.x & 0xffff0000u);
        x[k][2] = __uint_as_float(b.y << 16), x[k][3] = __uint_as_float(b.y & 0xffff0000u);
#pragma unroll
        for (int e = 0; e < 4; ++e) top = absmax_nan(top, x[k][e]);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) top = absmax_nan(top, __shfl_xor_sync(kFull, top, o));
      float down;
      const float up = q_unit(top, down);
      if (lane == 0) {
        const int64_t pos = s.w.sp.p0 + (s.row0 + min(r, s.rows - 1)) / a.group;  // (rows past the item's see what its last one sees)
        s_fq[r] = down * a.scale;
        s_end[r] = static_cast<int32_t>(max(min(pos + 1, static_cast<int64_t>(s.w.sp.len)), static_cast<int64_t>(0)));
        s_begin[r] = static_cast<int32_t>(max(pos + 1 - a.window, static_cast<int64_t>(0)));
      }
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int d = 4 * (lane + 32 * k);
        if (d < DP) {
          const uint32_t at = q_smem + (((r >> 3) * kSteps16 + d / 64 * 4 + (d >> 2) % 4) * 32 + (r & 7) * 4 + (d >> 4) % 4) * 8;
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(f16x2_bits(x[k][0] * up, x[k][1] * up)),
                       "r"(f16x2_bits(x[k][2] * up, x[k][3] * up))
                       : "memory");
        }
      }
    }
    __syncthreads();
    const auto load_q = [&](int t, int k, uint32_t (&b)[2]) {
      asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(b[0]), "=r"(b[1]) : "r"(q_smem + ((t * kSteps16 + k) * 32 + lane) * 8));
    };
    uint32_t qf[kHeld ? NT * kSteps16 : 1][2];
    if constexpr (kHeld) {
#pragma unroll
      for (int k = 0; k < NT * kSteps16; ++k) load_q(k / kSteps16, k % kSteps16, qf[k]);
    }
    // this lane's rows: 8 t + 2 c + e
    float fq[NT][2];
    int32_t end[NT][2], begin[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * t + 2 * c + e;
        fq[t][e] = s_fq[r];
        end[t][e] = s_end[r];
        begin[t][e] = s_begin[r];
      }
    // what every row sees (their positions do not decrease)
    const int32_t all_end = s_end[0], all_begin = s_begin[s.rows - 1], len = s.w.sp.len;

    float o[NT][kTiles][4], mx[NT][2], sum[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      mx[t][0] = mx[t][1] = kNone;
      sum[t][0] = sum[t][1] = 0.0f;
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][j][e] = 0.0f;
    }
    float least = 0x1p-100f;   // the smallest of the rows' units,
    bool mixed = false;        // and whether there are others (all in s_unit then): rows that do not see a block of large values keep theirs
    const int32_t count = s.t1 - s.t0;
    const int32_t w0 = s.t0 + static_cast<int32_t>(static_cast<int64_t>(count) * warp / kWarps);
    const int32_t w1 = s.t0 + static_cast<int32_t>(static_cast<int64_t>(count) * (warp + 1) / kWarps);
    for (int32_t st = w0; st < w1; ++st) {
      failed = !__all_sync(kFull, step_wait(smem_addr(&s_full[warp][stage]), phase, s_gave_up)) || failed;
      if (failed) break;
      const uint32_t from = ring + stage * Z::kStage;
      const int32_t has = s_has[warp][stage];
      const float4 scales = *reinterpret_cast<const float4*>(s_scale[warp][stage]);
      const float ks[2] = {scales.x, scales.z}, vs[2] = {scales.y, scales.w};
      const int64_t p64 = (static_cast<int64_t>(s.w.step0) + st) * kStep;
      const int32_t p = static_cast<int32_t>(p64);
      if (has) {
        // ---- x^T = K q^T ------------------------------------------------------------------------
        float x[NT][kHalves][4] = {};
#pragma unroll
        for (int h = 0; h < DP / 64; ++h) {
          uint32_t k0[kHalves][4], k1[kHalves][4];
#pragma unroll
          for (int i = 0; i < kHalves; ++i) {
            if constexpr (DP == 64) {  // 64-byte rows: 16-byte piece i of row r lies at i ^ (r / 2 % 4)
              const uint32_t at = from + i * 1024 + g * 64 + ((c ^ ((g >> 1) & 3)) << 4);
              lds16(k0[i], at);
              lds16(k1[i], at + 8 * 64);
            } else {                   // 128-byte rows: at i ^ (r % 8)
              const uint32_t at = from + (h >> 1) * kSlab + i * 2048 + g * 128 + (((4 * (h & 1) + c) ^ g) << 4);
              lds16(k0[i], at);
              lds16(k1[i], at + 8 * 128);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t qb[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if constexpr (kHeld) qb[t][0] = qf[t * kSteps16 + 4 * h + k][0], qb[t][1] = qf[t * kSteps16 + 4 * h + k][1];
              else load_q(t, 4 * h + k, qb[t]);
            }
#pragma unroll
            for (int i = 0; i < kHalves; ++i) {
              const uint32_t y0 = prepare_word<FMT>(k0[i][k]), y1 = prepare_word<FMT>(k1[i][k]);
              uint32_t ka[4];
              pairs_in_word<FMT>(y0, ka[0], ka[2]);
              pairs_in_word<FMT>(y1, ka[1], ka[3]);
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16816(x[t][i], ka, qb[t][0], qb[t][1]);
            }
          }
        }
        const bool whole = p64 + kStep <= all_end && p >= all_begin && has == (1 << kHalves) - 1;
        // ---- softmax: value 2 z + e of half i is token 16 i + 8 z + g, row 8 t + 2 c + e ------------
        bool moved = false;
        float was[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = kNone;
#pragma unroll
            for (int i = 0; i < kHalves; ++i) {
              const float f = fq[t][e] * ks[i];
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                float& v = x[t][i][2 * z + e];
                v *= f;
                if (!whole) {
                  const int64_t j = p64 + 16 * i + 8 * z + g;
                  if (j >= end[t][e] || j < begin[t][e] || !((has >> i) & 1)) v = kNone;
                }
                top = fmaxf(top, v);
              }
            }
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 4));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 8));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
            was[t][e] = mx[t][e];
            if (top > mx[t][e]) {
              mx[t][e] = top;
              moved = true;
            }
          }
        const float most = fmaxf(has & 1 ? vs[0] : 0.0f, has & 2 ? vs[kHalves - 1] : 0.0f);
        // (what is rare lies behind the one branch that there is anyway)
        if (__any_sync(kFull, moved || most > least || (FMT != QZ_INT8 && !whole))) {
          float unit_was = least;
          const auto unit_for = [](float unit, float most) {  // the next power of two above `most`
            return most > unit ? __uint_as_float((__float_as_uint(fminf(most, 0x1p125f)) & 0x7f800000u) + 0x00800000u) : unit;
          };
          if (most > least) {  // (the same for every lane)
            bool shared = !mixed;    // every row sees something of what there is
#pragma unroll
            for (int i = 0; i < kHalves; ++i) shared = shared && (!((has >> i) & 1) || (p64 + 16 * i < all_end && p64 + 16 * i + 15 >= all_begin));
            if (__builtin_expect(shared, 1)) {
              least = unit_for(least, most);
            } else {           // no block changes what a row that sees nothing of it keeps
              float lowest = 0x1p127f, highest = 0.0f;
#pragma unroll 1
              for (int r = 2 * c; r < kRows; r += r & 1 ? 7 : 1) {  // this lane's rows
                float seen = 0.0f;
#pragma unroll
                for (int i = 0; i < kHalves; ++i)
                  if (((has >> i) & 1) && p64 + 16 * i < s_end[r] && p64 + 16 * i + 15 >= s_begin[r]) seen = fmaxf(seen, vs[i]);
                const float unit = mixed ? s_unit[warp][r] : least, to = unit_for(unit, seen);
                lowest = fminf(lowest, to), highest = fmaxf(highest, to);
                __syncwarp();  // every lane of the row has read it
                if (g == 0) s_unit[warp][r] = to, s_shrink[warp][r] = unit / to;
              }
              __syncwarp();
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float shrink = s_shrink[warp][8 * t + 2 * c + e];
#pragma unroll
                  for (int j = 0; j < kTiles; ++j) {
                    o[t][j][e] *= shrink;
                    o[t][j][2 + e] *= shrink;
                  }
                }
#pragma unroll
              for (int d = 1; d < 4; d <<= 1) {
                lowest = fminf(lowest, __shfl_xor_sync(kFull, lowest, d));
                highest = fmaxf(highest, __shfl_xor_sync(kFull, highest, d));
              }
              least = unit_was = lowest;
              mixed = lowest != highest;
            }
          }
          if (FMT != QZ_INT8 && !whole && (p < all_begin || (p64 + kStep > all_end && all_end < len))) {
            // Positions that not every row sees: values there that are not finite numbers become zeros, and NaN the sums of the
            // rows that see them.
            const uint32_t at = from + kHalves * Z::kHalf + 16 * lane;
            const auto odd_at = [&](uint32_t d) {
              uint32_t w[4];
              lds16(w, at + d);
              return has_nonfinite<FMT>(w[0], w[1], w[2], w[3]);
            };
            bool odd = false;
#pragma unroll 4
            for (uint32_t d = 0; d < kHalves * Z::kHalf; d += 512) odd = odd_at(d) || odd;
            if (__any_sync(kFull, odd)) {
              if (lane == 0) s_spoiled[warp] = 0u;
              __syncwarp();
#pragma unroll 1
              for (uint32_t d = 0; d < kHalves * Z::kHalf; d += 512) {
                if (!odd_at(d)) continue;
                atomicOr(&s_spoiled[warp], 1u << ((16 * lane + d) / kRowBytes % kStep));
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + d), "r"(0u) : "memory");
                fence_proxy_async();  // (before the next copy to this stage)
              }
              __syncwarp();
              const uint32_t spoiled = s_spoiled[warp] & ((has & 1 ? 0xffffu : 0u) | (has & 2 ? 0xffff0000u : 0u));
#pragma unroll 1
              for (int r = lane; r < kRows; r += 32) {
                const int64_t lo = max(s_begin[r] - p64, static_cast<int64_t>(0)), hi = min(s_end[r] - p64, static_cast<int64_t>(kStep));
                const uint32_t seen = hi > lo ? (0xffffffffu >> (32 - static_cast<int>(hi - lo))) << lo : 0u;
                if (spoiled & seen) s_l[warp][r] = __uint_as_float(0x7fc00000u);
              }
            }
          }
          const float shrink = unit_was / least;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float f = mx[t][e] == kNone ? 1.0f : ex2(was[t][e] - mx[t][e]), fo = f * shrink;
              sum[t][e] *= f;
#pragma unroll
              for (int j = 0; j < kTiles; ++j) {
                o[t][j][e] *= fo;
                o[t][j][2 + e] *= fo;
              }
            }
        }
        uint32_t pb[NT][kHalves][2];
        const auto weigh = [&](auto each) {  // each: every row its own unit
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float y[kHalves][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float top = mx[t][e] == kNone ? 0.0f : mx[t][e];
              const float unit = decltype(each)::value ? s_unit[warp][8 * t + 2 * c + e] : least;
              const float inverse = __uint_as_float((269u << 23) - __float_as_uint(unit));  // 2^15 / unit
#pragma unroll
              for (int i = 0; i < kHalves; ++i)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const float v = x[t][i][2 * z + e], w = ex2(v - top);
                  sum[t][e] += w;
                  y[i][2 * z + e] = w * (vs[i] * inverse);
                  if (!whole && v == kNone) y[i][2 * z + e] = 0.0f;  // (the scale of what is not seen may be anything)
                }
            }
#pragma unroll
            for (int i = 0; i < kHalves; ++i)
#pragma unroll
              for (int z = 0; z < 2; ++z) pb[t][i][z] = transposed(f16x2_bits(y[i][2 * z], y[i][2 * z + 1]));
          }
        };
        if (__builtin_expect(mixed, 0)) weigh(std::true_type{});
        else weigh(std::false_type{});
        // ---- out^T += V^T p^T ---------------------------------------------------------------------
#pragma unroll
        for (int i = 0; i < kHalves; ++i)
#pragma unroll
          for (int h = 0; h < kPieces; ++h) {
            uint32_t vw[4][4];
            const uint32_t vfrom = from + kHalves * Z::kHalf + i * (16 * kRowBytes);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = 2 * c + (k & 1) + 8 * (k >> 1);
              if constexpr (DP == 64) {
                const uint32_t at = vfrom + r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8;
                asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(vw[k][0]), "=r"(vw[k][1]) : "r"(at));
              } else {  // DP = 256: pieces 2 g and 2 g + 1 of 16, eight a box
                const int piece = DP == 128 ? g : 2 * g + h;
                lds16(vw[k], vfrom + (piece >> 3) * kSlab + r * 128 + (((piece & 7) ^ (r & 7)) << 4));
              }
              // memory past the end, or of a page that is not there, may hold anything
              if (!whole && (p64 + 16 * i + r >= len || !((has >> i) & 1))) vw[k][0] = vw[k][1] = vw[k][2] = vw[k][3] = 0u;
            }
#pragma unroll
            for (int j = 0; j < kTiles / kPieces; ++j) {
              const int q = j >> 1;
              uint32_t va[4];
              if (j & 1) {
                pairs_of_words<FMT, 2>(vw[0][q], vw[1][q], va[0], va[1]);
                pairs_of_words<FMT, 2>(vw[2][q], vw[3][q], va[2], va[3]);
              } else {
                pairs_of_words<FMT, 0>(vw[0][q], vw[1][q], va[0], va[1]);
                pairs_of_words<FMT, 0>(vw[2][q], vw[3][q], va[2], va[3]);
              }
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16816(o[t][8 * h + j], va, pb[t][i][0], pb[t][i][1]);
            }
          }
      }
      __syncwarp();  // every lane has read the stage
      copy();
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (failed) {
#pragma unroll
      for (int t = 0; t < NT; ++t) sum[t][0] = sum[t][1] = __uint_as_float(0x7fc00000u);
    }
    more = advance();
    if (more && !failed) {  // the next segment's first steps are on their way while the sums are joined
      ask_q(n);
      aim(n);
#pragma unroll 1
      for (int i = 0; i < kStages; ++i) copy();
    }

    // ---- the warps' sums, joined some columns at a time ------------------------------------------
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) sum[t][e] += __shfl_xor_sync(kFull, sum[t][e], w);
        if (g == 0) {
          s_m[warp][8 * t + 2 * c + e] = mx[t][e];
          s_l[warp][8 * t + 2 * c + e] += sum[t][e];
          if (!mixed) s_unit[warp][8 * t + 2 * c + e] = least;
        }
      }
    const bool first = s.t0 == 0, last = s.t1 == s.w.steps;
    float* slot = WHOLE || (first && last) ? nullptr : slots + (2 * static_cast<size_t>(blockIdx.x) + (first ? 1 : 0)) * Z::kSlot;
    constexpr int kQuads = Z::kJoinCols / 32;    // float4s of each of the eight column groups at a time
#pragma unroll
    for (int q = 0; q < kCols / 4; q += kQuads) {
#pragma unroll
      for (int z = 0; z < kQuads; ++z)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e)  // [warp][row][z][column group]
            *reinterpret_cast<float4*>(join + (((warp * kRows + 8 * t + 2 * c + e) * kQuads + z) * 8 + g) * 4) =
                make_float4(o[t][2 * (q + z)][e], o[t][2 * (q + z)][2 + e], o[t][2 * (q + z) + 1][e], o[t][2 * (q + z) + 1][2 + e]);
      __syncthreads();
      if (q == 0) {  // each warp's factor for the row's sums, in place of its maximum; the row's own m and l
        for (int r = warp; r < kRows; r += kWarps) {  // lane k: warp k's
          const float m = lane < kWarps ? s_m[lane < kWarps ? lane : 0][r] : kNone;
          float top = m;
#pragma unroll
          for (int w = 8; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, w));
          const float f = ex2(m - (top == kNone ? 0.0f : top));
          float l = lane < kWarps ? f * s_l[lane < kWarps ? lane : 0][r] : 0.0f;
          if (lane < kWarps) s_l[lane][r] = 0.0f;  // for the next segment
#pragma unroll
          for (int w = 8; w; w >>= 1) l += __shfl_xor_sync(kFull, l, w);
          if (lane < kWarps) s_m[lane][r] = f * s_unit[lane][r] * 0x1p-15f;
          if (lane == 0) s_top[r] = top, s_sum[r] = l;
        }
        __syncthreads();
      }
      for (int i = tid; i < kRows * 8 * kQuads; i += Z::kThreads) {
        const int r = i / (8 * kQuads), d = kCols * (i & 7) + 4 * (q + (i >> 3) % kQuads);
        if (r >= s.rows) break;
        float v[4] = {};
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float f = s_m[k][r];
          const float4 y = *reinterpret_cast<const float4*>(join + (k * kRows * kQuads * 8 + i) * 4);
          v[0] = __fmaf_rn(y.x, f, v[0]), v[1] = __fmaf_rn(y.y, f, v[1]);
          v[2] = __fmaf_rn(y.z, f, v[2]), v[3] = __fmaf_rn(y.w, f, v[3]);
        }
        if (slot) {
          *reinterpret_cast<float4*>(slot + r * DP + d) = make_float4(v[0], v[1], v[2], v[3]);
          if (d == 0) {
            slot[kRows * DP + r] = s_top[r];
            slot[kRows * (DP + 1) + r] = s_sum[r];
          }
        } else {
          const int i0 = (s.row0 + r) / a.group;
          store_row(a, s.w.sp.row + i0, s.kvh * a.group + (s.row0 + r) - i0 * a.group, d, v, s_top[r], s_sum[r]);
        }
      }
      __syncthreads();
    }
    if (!WHOLE && first && !last && tid == 0) {
      FewMeta meta;
      meta.seq = s.seq;
      meta.head = s.kvh;
      meta.row0 = s.row0;
      meta.last = static_cast<int32_t>((s.item_u0 + s.w.steps - 1) / chunk);
      static_cast<FewMeta*>(a.ws)[blockIdx.x] = meta;
    }
  }
  if (failed) {  // copies still in flight land before the memory is released
    for (int i = 0; i < kStages; ++i) {
      held_wait(smem_addr(&s_full[warp][stage]), phase, kFewWaitNs);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
}

// Joins the partial results of the items that more than one share holds: CTA (i, y) the y-th part of the
// rows of the item that begins in share i.
template <int DP, int NT>
__global__ void __launch_bounds__(128) attention_join_kernel(const AttentionArgs a, int grid) {
  using Z = FewSizes<DP, NT>;
  constexpr int kRows = Z::kRows;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const FewMeta meta = static_cast<const FewMeta*>(a.ws)[blockIdx.x];
  if (meta.seq < 0) return;
  const float* slots = reinterpret_cast<const float*>(static_cast<const char*>(a.ws) + static_cast<size_t>(grid) * sizeof(FewMeta));
  const Span sp = span_of(a.b, meta.seq, a.c.page);
  const int rows = static_cast<int>(min(static_cast<int64_t>(kRows), static_cast<int64_t>(sp.n) * a.group - meta.row0));
  const int parts = meta.last - static_cast<int>(blockIdx.x) + 1;
  const auto part = [&](int k) { return slots + (2 * (static_cast<size_t>(blockIdx.x) + k) + (k == 0 ? 1 : 0)) * Z::kSlot; };
  for (int i = static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x); i < rows * (DP / 4); i += static_cast<int>(gridDim.y * blockDim.x)) {
    const int r = i / (DP / 4), d = 4 * (i % (DP / 4));
    if (d >= a.c.dim) continue;
    float top = kNone;
#pragma unroll 4
    for (int k = 0; k < parts; ++k) top = fmaxf(top, part(k)[kRows * DP + r]);
    const float from = top == kNone ? 0.0f : top;
    float v[4] = {}, l = 0.0f;
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const float* p = part(k);
      const float f = ex2(p[kRows * DP + r] - from);
      const float4 y = *reinterpret_cast<const float4*>(p + r * DP + d);
      l = __fmaf_rn(p[kRows * (DP + 1) + r], f, l);
      v[0] = __fmaf_rn(y.x, f, v[0]), v[1] = __fmaf_rn(y.y, f, v[1]);
      v[2] = __fmaf_rn(y.z, f, v[2]), v[3] = __fmaf_rn(y.w, f, v[3]);
    }
    store_row(a, sp.row + (meta.row0 + r) / a.group, meta.head * a.group + (meta.row0 + r) % a.group, d, v, top, l);
  }
}

// ---- host side ----------------------------------------------------------------------------------
template <int FMT, int DP, int NT>
qz_status run_few(const AttentionArgs& a, const FewPlan& p, cudaStream_t s) {
  using Z = FewSizes<DP, NT>;
  CacheMaps maps{};
  if (a.c.pages > 0 && !encode_maps(&maps, a, 16)) return QZ_ERR_CUDA;
  if (p.whole) {
    const auto k = &attention_few_kernel<FMT, DP, NT, true>;
    if (!set_dyn_smem(reinterpret_cast<const void*>(k), Z::kSmem)) return QZ_ERR_CUDA;
    k<<<static_cast<unsigned>(p.grid), Z::kThreads, Z::kSmem, s>>>(a, maps, p.grid, p.min_chunk);
    return launch_status();
  }
  const auto k = &attention_few_kernel<FMT, DP, NT, false>;
  if (!set_dyn_smem(reinterpret_cast<const void*>(k), Z::kSmem)) return QZ_ERR_CUDA;
  k<<<static_cast<unsigned>(p.grid), Z::kThreads, Z::kSmem, s>>>(a, maps, p.grid, p.min_chunk);
  if (launch_status() != QZ_OK) return QZ_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.grid), 4);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attention_join_kernel<DP, NT>, a, p.grid) != cudaSuccess) {
    cudaGetLastError();
    return QZ_ERR_CUDA;
  }
  return launch_status();
}
template <int FMT>
qz_status launch_few(const AttentionArgs& a, const FewPlan& p, cudaStream_t s) {
  switch (few_att_dim(a.c.dim)) {
    case 64: return p.row_tiles == 1 ? run_few<FMT, 64, 1>(a, p, s) : p.row_tiles == 2 ? run_few<FMT, 64, 2>(a, p, s) : run_few<FMT, 64, 4>(a, p, s);
    case 128: return p.row_tiles == 1 ? run_few<FMT, 128, 1>(a, p, s) : p.row_tiles == 2 ? run_few<FMT, 128, 2>(a, p, s) : run_few<FMT, 128, 4>(a, p, s);
    default: return p.row_tiles == 1 ? run_few<FMT, 256, 1>(a, p, s) : run_few<FMT, 256, 2>(a, p, s);
  }
}

}  // namespace
}  // namespace qz
