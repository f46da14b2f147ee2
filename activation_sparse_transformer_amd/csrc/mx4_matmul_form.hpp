// Which kernel form multiplies T tokens in 4 bits with nb blocks of 16 weight rows by kb blocks of 128
// columns.  By itself, so that a host test can check the rule and the forms it selects.
#pragma once

#include <stdint.h>

namespace sffn {

constexpr int FEW_WAVES = 8;  // of a workgroup of the forms for few tokens

enum Mx4MatmulForm {
  MX4_FEW_1,         // 16 tokens, 1 block of rows a workgroup, 8 parts of the columns
  MX4_FEW_4,         // 16 tokens, 2 x 4 blocks, 4 parts
  MX4_FEW_32,        // 32 tokens, 1 block, 8 parts
  MX4_FEW_64,        // 64 tokens, 2 blocks, 8 parts
  MX4_TILE_64x64,    // rows x tokens of a workgroup
  MX4_TILE_128x64,
  MX4_TILE_128x128,
  MX4_TILE_128x256,
  MX4_FORMS
};

struct Mx4TileCost {
  int rows, tokens;   // of a workgroup
  int per_cu;         // workgroups of a CU at a time
  int alone, shared;  // ns a stage of 128 columns takes: a CU's only workgroup, and each of many
  int epilogue;       // ns of the results of one
};
// Measured at 8192 x 2048 to 16384 weights and 128 to 2048 tokens.
constexpr Mx4TileCost MX4_TILE_COST[] = {
    {64, 64, 5, 240, 118, 500}, {128, 64, 4, 300, 215, 1000}, {128, 128, 3, 345, 285, 2000}, {128, 256, 2, 470, 480, 4000}};

inline int mx4_matmul_form(int32_t nb, int32_t kb, int32_t T) {
  if (T <= 16) return nb < 2048 ? MX4_FEW_1 : MX4_FEW_4;
  if (T <= 32 && nb < 2048) return MX4_FEW_32;
  if (T <= 64 && nb < 2048) return MX4_FEW_64;
  int best = MX4_TILE_64x64;
  double best_ns = 0;
  for (int f = MX4_TILE_64x64; f < MX4_FORMS; ++f) {
    const Mx4TileCost& c = MX4_TILE_COST[f - MX4_TILE_64x64];
    const double groups = (double)(((int64_t)nb * 16 + c.rows - 1) / c.rows) * ((T + c.tokens - 1) / c.tokens);
    const double each = (double)(int64_t)((groups + 255) / 256);  // workgroups of a CU
    const double rounds = (double)(int64_t)((each + c.per_cu - 1) / c.per_cu);
    const double stage = c.alone * rounds > c.shared * each ? c.alone * rounds : c.shared * each;
    const double ns = kb * stage + c.epilogue * rounds;
    if (f == MX4_TILE_64x64 || ns < best_ns) {
      best = f;
      best_ns = ns;
    }
  }
  return best;
}

}  // namespace sffn
