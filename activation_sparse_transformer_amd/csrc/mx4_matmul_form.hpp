// Which kernel form multiplies T tokens in 4 bits with nb blocks of 16 weight rows by kb blocks of 128
// columns.  By itself, so that a host test can check the rule and the forms it selects.
#pragma once

#include <stdint.h>

namespace sffn {

enum Mx4MatmulForm {
  // eight waves split the columns: tokens x blocks of rows of a workgroup
  MX4_FEW_16x1,
  MX4_FEW_16x2,
  MX4_FEW_16x4,
  MX4_FEW_32x1,
  MX4_FEW_32x2,
  MX4_FEW_64x2,
  // stages in LDS: rows x tokens of a workgroup
  MX4_TILE_64x64,
  MX4_TILE_128x64,
  MX4_TILE_128x128,
  MX4_TILE_128x256,
  MX4_FORMS
};

struct Mx4TileCost {
  int rows, tokens;   // of a workgroup
  int per_cu;         // workgroups of a CU at a time
  int alone, shared;  // ns a stage of 128 columns takes: a CU's only workgroup, and each of many
  int ends[2];        // ns of the first loads and of the results: bf16, fp32
};
// From kernel times at 2304 to 65536 rows, 1024 to 16384 columns and 64 to 2048 tokens.
constexpr Mx4TileCost MX4_TILE_COST[] = {{64, 64, 5, 200, 118, {3500, 3900}},
                                         {128, 64, 4, 250, 200, {3800, 4700}},
                                         {128, 128, 3, 310, 285, {4700, 6300}},
                                         {128, 256, 2, 470, 480, {7200, 10500}}};

// Estimated ns of a tile form.
inline double mx4_tile_ns(int f, int32_t nb, int32_t kb, int32_t T, bool y_f32) {
  const Mx4TileCost& c = MX4_TILE_COST[f - MX4_TILE_64x64];
  const int64_t groups = ((int64_t)nb * 16 + c.rows - 1) / c.rows * ((T + c.tokens - 1) / c.tokens);
  const int64_t each = (groups + 255) / 256, rounds = (each + c.per_cu - 1) / c.per_cu;  // of a CU
  const int64_t apart = c.alone * rounds, together = c.shared * each;
  return (double)kb * (double)(apart > together ? apart : together) + (double)c.ends[y_f32] * (double)rounds;
}
// And of MX4_FEW_64x2: a wave takes one block of columns in about 650 ns, later with more than one
// workgroup a CU.
inline double mx4_few_ns(int32_t nb, int32_t kb, int32_t T) {
  const double groups = (double)((nb + 1) / 2) * ((T + 63) / 64), load = 1.25 * groups / 256;
  return 3000 + (double)((kb + 7) / 8) * 650 * (load > 1 ? load : 1);
}

// rounding: the kernel rounds its (at most 16) tokens itself, once for all blocks of a wave.  (Kernel us at
// 16 x 1, 2, 4: 2304 x 9216 9.7, 10.9, 12.9; 8192 x 2048 5.6, 4.8, 5.4; 32768 x 4096 23, 17, 14; of tokens
// in 4 bits 4.5, 5.4, -; 3.3, 3.3, -; 11.5, 11.8, -; 65536 x 8192 55, 43, -.)
// 17 to 32 tokens take two blocks (32 x 16384 x 4096 9.3 us with one, 7.9 with two) where there are enough
// (32 x 2304 x 9216 6.0 and 6.8), and so do up to 64 then (6.8; 8.9 at once).  Above that the estimates
// choose (100 x 8192 x 2048: 64 x 2 6.3 us, tiles of 64 x 64 6.7, 128 x 128 9.7; 128 x 2304 x 9216 9.2 and 16;
// 64 x 32768 x 4096 16.2 and 13.9; 1024 x 8192 x 2048: tiles of 64 x 64 23, 128 x 128 16.3, 128 x 256 17.4;
// 16384 x 9216 x 2304: 400, 245, 212; fp32 results of 333 x 9999 x 1504: 128 x 64 11.4, 128 x 128 12.3).
inline int mx4_matmul_form(int32_t nb, int32_t kb, int32_t T, bool rounding, bool y_f32) {
  if (T <= 16) {
    if (rounding) return nb < 512 ? MX4_FEW_16x1 : nb < 1024 ? MX4_FEW_16x2 : MX4_FEW_16x4;
    return nb < 4096 ? MX4_FEW_16x1 : MX4_FEW_16x2;
  }
  if (T <= 32) return nb < 256 ? MX4_FEW_32x1 : MX4_FEW_32x2;
  if (T <= 64 && nb < 256) return MX4_FEW_32x2;
  int best = MX4_FEW_64x2;
  double best_ns = mx4_few_ns(nb, kb, T);
  for (int f = MX4_TILE_64x64; f < MX4_FORMS; ++f) {
    const double ns = mx4_tile_ns(f, nb, kb, T, y_f32);
    if (ns < best_ns) {
      best = f;
      best_ns = ns;
    }
  }
  return best;
}

}  // namespace sffn
