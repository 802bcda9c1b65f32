// ffn_plan.h -- which tile a product of the gated feed-forward projections takes, and
// whether its k is cut.  Host only.
#pragma once

#include <stdint.h>

namespace m3 {

constexpr int kPlanRowBytes = 128;  // of k in a tile's row

// The tile, and the parts that k is cut into: of the tiles below the one whose rounds
// over the 256 CUs take the least, by its area and the share of the largest tile's
// rate that it reaches by itself (8192 x 2048 x 4096, both products, in one tile size
// each: bfloat16 243, 285, 412 and 547 us; float, whose products take longer than what
// feeds them, 1.88, 1.86, 1.94 and 2.06 ms).  With 512 rows of those the largest tile
// would take 42 us where the second takes 23, with 100 rows 41 where the third takes 9,
// all on inputs that do not change (others come from memory: 31 and 12).  Where a product has few tiles and a long k, its parts fill the CUs
// instead, of eight tiles of k at least (the backward pass of 256 x 2048 x 4096,
// bfloat16: 61 to 48 us, of 20000 x 64 x 300 120 to 44, float 291 to 75);
// joining them takes some 6 us and the parts' way through memory, in the unit of the
// rest: a chip of largest tiles takes 128 bytes of k in 1.6 us, float in 7.4.  No tile
// takes them in less than 0.3 us, which its loads and barriers need.  The two smallest
// tiles' workgroups, a wave a SIMD, wait less where two share a CU: in float a tile by
// itself takes 1.3 times its share, and k is cut until there are two (the backward pass
// of 256 x 2048 x 4096: 167 to 151 us, of 16384 x 256 x 1024: 354 to 331); bfloat16, whose
// parts take longer to join than their products, gains nothing.
struct Plan {
  int tile, parts, each;
};
inline Plan plan_gemm(int64_t M, int64_t cols, int64_t K, int esize, bool cut) {
  const struct {
    int m, n;
    double bf16, f32;
  } tiles[] = {{256, 256, 1.0, 1.0}, {128, 128, 0.85, 1.0}, {64, 64, 0.6, 0.96}, {32, 64, 0.45, 0.9}};
  const int64_t step = kPlanRowBytes / esize, steps = (K + step - 1) / step;
  Plan best = {};
  double least = 0;
  const int first = esize == 2 ? 0 : 1;  // (the largest gains nothing in float)
  for (int i = first; i < 4; ++i) {
    const int64_t count = (M + tiles[i].m - 1) / tiles[i].m * ((cols + tiles[i].n - 1) / tiles[i].n);
    const bool pairs = esize == 4 && i >= 2;
    int64_t parts = cut ? (pairs ? 512 : 256) / count : 1;
    if (parts > steps / 8) parts = steps / 8;
    if (parts < 1) parts = 1;
    const int64_t each = (steps + parts - 1) / parts;
    parts = (steps + each - 1) / each;
    const double rate = esize == 2 ? tiles[i].bf16 : tiles[i].f32;
    const int64_t rounds = (count * parts + 255) / 256;
    double cost = (pairs && rounds == 1 ? 1.3 : (double)rounds) * tiles[i].m * tiles[i].n / rate;
    const double alone = esize == 2 ? 12000.0 : 2700.0;
    cost = (cost < alone ? alone : cost) * (double)each;
    if (parts > 1) cost += (6.0 + (double)parts * (double)M * (double)cols * 8.0 / 5.0e6) * (esize == 2 ? 41500.0 : 8900.0);
    if (i == first || cost < least) {
      least = cost;
      best = Plan{i, (int)parts, (int)(each * step)};
    }
  }
  return best;
}

}  // namespace m3
