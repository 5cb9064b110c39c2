// qz_product_plan.h -- how the tcgen05 products (qz_product_tc.cuh) divide a call, and what each kind
// of kernel is estimated to take.
#pragma once

#include <algorithm>
#include <cstdint>

#include "qz_internal.h"
#include "qz_product.h"

namespace qz {

constexpr int kBM = 128;  // outputs per CTA (MMA rows, tensor-memory lanes)
constexpr int box_of(int format) { return format == QZ_INT4 ? 64 : 128; }  // summands of a box: eight MMAs
inline int boxes_of(int format, int64_t sum) { return static_cast<int>((sum + box_of(format) - 1) / box_of(format)); }

// The form and its tiles for outputs [m_base, m_base + nout).  Estimated in SM cycles: a box's eight
// MMAs take 4 cycles a token column (128 x n x 16 each at 8192 FLOP a cycle); its hand-over takes
// some 750 cycles in a pair, whose decoders share the tokens' copies, and 950 alone; a tile of the
// second form starts with an empty pipeline and ends with the exchange.
struct Plan {
  bool pair;
  int n, tiles_n, tiles, slices, slice_boxes, grid;
  int64_t m_base;
  double cost;
};
inline void tokens_per_tile(int64_t tokens, int most, int unit, int* n, int64_t* tiles_n) {
  const int64_t t = (tokens + most - 1) / most;
  *n = static_cast<int>(((tokens + t - 1) / t + unit - 1) / unit * unit);
  *tiles_n = (tokens + *n - 1) / *n;
}
inline Plan plan_pairs(int64_t m_base, int64_t nout, int out_per_cta, int64_t tokens, int boxes, double least) {
  Plan best{};
  best.cost = 1e30;
  const int64_t pairs = std::max(1, sm_count() / 2);
  for (int most = 256; most >= 64; most -= 32) {  // narrower tiles where they fill the last round better
    int n;
    int64_t tiles_n;
    tokens_per_tile(tokens, most, 32, &n, &tiles_n);
    const int64_t tiles = (nout + 2 * out_per_cta - 1) / (2 * out_per_cta) * tiles_n;
    const double cost = static_cast<double>((tiles + pairs - 1) / pairs) * boxes * std::max(4.0 * n + 40, least) + 6000;
    if (tiles < (int64_t{1} << 30) && cost < best.cost)
      best = Plan{true, n, static_cast<int>(tiles_n), static_cast<int>(tiles), 1, boxes, static_cast<int>(2 * std::min(tiles, pairs)), m_base, cost};
  }
  return best;
}
inline Plan plan_alone(int64_t m_base, int64_t nout, int out_per_cta, int64_t tokens, int boxes) {
  Plan best{};
  best.cost = 1e30;
  const int sms = sm_count();
  for (int s = 1; s <= 8; s *= 2)
    for (int most : {192, 128}) {
      int n;
      int64_t tiles_n;
      tokens_per_tile(tokens, most, std::max(32, 8 * s), &n, &tiles_n);  // the columns divide into eights per slice
      const int64_t tiles = (nout + out_per_cta - 1) / out_per_cta * tiles_n;
      const int per = (boxes + s - 1) / s;
      const int64_t clusters = std::max(1, s == 1 ? sms : (s == 2 ? sms * 9 / 10 : sms * 5 / 6) / s);
      // above 128 tokens the copies have two stages only
      const double box = std::max(4.0 * n, n > 128 ? 1200.0 : 950.0);
      const double cost = static_cast<double>((tiles + clusters - 1) / clusters) * (per * box + 6000 + (s > 1 ? 2000 + 16.0 * n : 0));
      if (tiles * s < (int64_t{1} << 30) && cost < best.cost)
        best = Plan{false, n, static_cast<int>(tiles_n), static_cast<int>(tiles), s, per, static_cast<int>(tiles * s), m_base, cost};
    }
  return best;
}
// One launch, or two: where a few tiles of the pairs would make a round of their own, the last
// outputs' tiles go to a second launch that splits their sums over the whole GPU.
inline int plan_of(const ProductArgs& p, Plan (&plan)[2]) {
  const bool back = p.mode == kModeBackward;
  const int64_t nout = back ? p.cols : p.rows, tokens = p.tokens;
  const int out_per_cta = p.mode == kModeGated ? kBM / 2 : kBM;
  const int boxes = boxes_of(p.format, back ? p.rows : p.cols) * (back ? p.n_weights : 1);
  const double least = p.format == QZ_INT4 ? 1060.0 : 750.0;
  const Plan pairs = plan_pairs(0, nout, out_per_cta, tokens, boxes, least), alone = plan_alone(0, nout, out_per_cta, tokens, boxes);
  plan[0] = alone.cost < pairs.cost ? alone : pairs;
  if (plan[0].cost > 1e29) return 0;
  const int64_t per_round = std::max(1, sm_count() / 2) / pairs.tiles_n;  // rows of pairs' tiles a round takes
  const int64_t rows_m = (nout + 2 * out_per_cta - 1) / (2 * out_per_cta);
  if (per_round < 1 || rows_m <= per_round || rows_m % per_round == 0) return 1;
  const int64_t first = rows_m / per_round * per_round * 2 * out_per_cta;
  const Plan a = plan_pairs(0, first, out_per_cta, tokens, boxes, least), b = plan_alone(first, nout - first, out_per_cta, tokens, boxes);
  if (a.cost + b.cost + 4000 >= plan[0].cost) return 1;
  plan[0] = a;
  plan[1] = b;
  return 2;
}

// Microseconds of the tiles and of the streaming kernel on the GPU, fitted to forward products of 1 to 32 tokens,
// 256 to 32768 outputs and 1024 to 16384 columns, gated and not, timed on both (512 pairs): 96 per cent of the
// estimates are within a quarter, and the kernel chosen took 1.18 times the other's time at worst.
//   tiles      the plan's cycles.
//   streaming  the start; the activations' staging in every CTA, 0.48 a token and 4096 columns; the weights,
//              0.11 a million E2M1 (INT4 0.14) for up to 8 tokens, 0.15 (0.18) for up to 16, 0.23 above.
// 16 tokens, NVFP4: 512 x 2048 12.1 us streaming and 7.7 on the tiles, 32768 x 4096 31.4 and 34.5; 32 tokens,
// INT4 groups of 32: 512 x 2048 23.5 and 9.7, 32768 x 2048 43.5 and 49.
inline double tiles_us(const ProductArgs& p) {
  Plan plan[2];
  const int n = plan_of(p, plan);
  if (n == 0) return 1e30;
  return 1.4 + (plan[0].cost + (n == 2 ? plan[1].cost + 4000 : 0.0)) / 1700;
}
inline double few_us(const ProductArgs& p) {
  const bool int4 = p.format == QZ_INT4;
  const double rate = p.tokens <= 8 ? (int4 ? 0.14 : 0.11) : p.tokens <= 16 ? (int4 ? 0.18 : 0.15) : 0.23;
  const double staged = static_cast<double>(p.tokens) * static_cast<double>((p.cols + 4095) / 4096);
  return 4.5 + 0.48 * staged + rate * 1e-6 * p.n_weights * static_cast<double>(p.rows) * static_cast<double>(p.cols);
}

}  // namespace qz
