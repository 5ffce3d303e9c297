// product_plan.hpp -- which tiles a product of 16-bit operands is made of, and over how many workgroups its K is split.
#pragma once
#include <stdint.h>

#include <cmath>

namespace fp8dp {

// Tiles of a product of m x n outputs over `stages` of K, and over how many workgroups K is split.
enum TileShape { kTile256, kTile192, kTile128, kTileAny };   // 256 x 256, 256 x 192, 128 x 128, the same at any alignment
struct ProductPlan {
  TileShape shape;
  int splits;
};
inline int64_t tiles_of(TileShape t, int64_t m, int64_t n) {
  const int64_t bm = t == kTile256 || t == kTile192 ? 256 : 128;
  const int64_t bn = t == kTile256 ? 256 : t == kTile192 ? 192 : 128;
  return ((m + bm - 1) / bm) * ((n + bn - 1) / bn);
}
// The plan of the least estimate, in us: a workgroup's stages of 64 of K and, for each tile, its ends (the first copies,
// the outputs).  The stages' times were measured, as the difference of K = 4096 and 1024 over 48, with every compute unit busy
// with one tile or two: 256 x 256 1.40 .. 1.72 (4096 x 4096), 256 x 192 1.02 .. 1.04, 128 x 128 0.44 .. 0.49 where it has a
// compute unit to itself, 0.80 .. 0.85 for two, at any alignment 1.04 .. 1.30 and 1.35 .. 1.56.  A K that is
// shared costs a join.  With estimates that favoured shares by a third more, gradients of 1025 x 1023 x 1001 took 50.5 us
// for 45.9 (dx from three shares, now one), 8192 x 2048 x 768 169 for 161, one forward of 100 x 1024 x 1024 14.1 for 11.6;
// 1000 x 8192 x 4096 is the worst loss that was found (302, now 312).  256 x 192 was measured with operands that the caches
// hold: dx of 16384 x 2048 x 768, whose [dg | du] comes from memory, takes 1.57 a stage.  There is no term for bytes, so that of
// plans for few tokens and wide weights, which memory bounds, the estimates cannot tell the faster.
inline ProductPlan plan_product(int64_t m, int64_t n, int64_t stages, bool dual, bool direct, double cus) {
  ProductPlan best = {direct ? kTile256 : kTileAny, 1};
  double least = 1e30;
  auto offer = [&](TileShape t, double per_stage, double alone, int per_cu, double ends) {
    const double tiles = (double)tiles_of(t, m, n);
    for (int s = 1; s <= 8 && (s == 1 || stages / s >= 4); ++s) {
      const double groups = tiles * s, turns = std::ceil(groups / (cus * per_cu));
      const double each = (double)((stages + s - 1) / s) * (groups <= cus ? alone : per_stage) + ends;
      const double join = s == 1 ? 0.0 : 4.0 + s * (double)m * (double)n * 8.0 / 4e6;
      const double us = turns * each + join;
      if (us < least) {
        least = us;
        best = {t, s};
      }
    }
  };
  if (direct) {
    offer(kTile256, 1.45, 1.45, 1, 5.0);
    if (!dual) offer(kTile192, 1.05, 1.05, 1, 4.5);
    offer(kTile128, 0.82, 0.45, 2, 3.5);
  } else {
    offer(kTileAny, 1.45, 1.15, 2, 3.5);
  }
  return best;
}

}  // namespace fp8dp
