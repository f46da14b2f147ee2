// The kernel form that a product with 4-bit weights takes: token tiles (of 16 tokens) and row blocks
// (of 16 rows) of a wave, and the waves of a workgroup that split k.  Host code without HIP.
#pragma once

#include <cstdint>

#include "../../include/ffn_ops.h"

namespace sffn {

constexpr int MX4_WAVES = 8;  // of a workgroup
struct Mx4Shape {
  int tt, rb, ks;  // token tiles 1..4, row blocks 1..4, k parts 2, 4, 8
};

// Whether two workgroups fit a CU: 128 registers and half of the LDS do without spilling.
constexpr bool mx4_pairs(int x_dtype, int tt, int rb) {
  return tt == 1 || (x_dtype == SFFN_E4M3 && rb * tt <= (tt == 2 ? 6 : 8)) ||
         (x_dtype == SFFN_BF16 && rb * tt <= 4 && tt == 2);
}

// The forms that mx4_shape can choose, for any sizes; no other kernel is built.  One or two row
// blocks go with few workgroups, whose waves all split k.  Three take four and two k parts from
// 3072 and 6144 (more than 16 tokens: 1536 and 3072) blocks of rows times token groups on, where four
// row blocks have the lower estimate but for the token types that load the least.  More than two
// tiles of fp32 tokens would not fit the LDS; of the others, three or four with few row blocks never
// have a lower estimate than two with twice as many.
constexpr bool mx4_built(int x_dtype, int tt, int rb, int ks) {
  const bool fp32 = x_dtype == SFFN_F32, fp8 = x_dtype == SFFN_E4M3;
  if (tt > 2 && (fp32 || rb < (tt == 4 ? 3 : fp8 ? 1 : 2))) return false;
  if (rb < 3) return ks == 8;
  if (rb == 3) return ks == 8 || (ks == 4 && !(fp32 && tt == 1)) || (fp8 && tt > 1);
  return true;
}

inline int64_t mx4_token_groups(int64_t T, int tt) { return (T + tt * 16 - 1) / (tt * 16); }

// Estimated time of a form, in units of a wave's work on one block of 16 rows, 128 columns and up to
// 32 tokens: per block of columns that on the tokens (loads, conversions) and on rb blocks of
// weights, for as many workgroups as a CU gets, and for every workgroup (for every two where two fit
// at once) the 10 units, 2 us, that its loads and its join take to pass.  Three and four tiles of
// tokens cost 1.35 and 1.7 times two (the weights are expanded once), and 13 and 16 units.  Fitted to
// sweeps of rb and tt over N 2048 .. 65536, K 256 .. 8192.
inline double mx4_cost(int x_dtype, int tt, int rb, int64_t nb, int64_t kb, int64_t T) {
  const double tokens = x_dtype == SFFN_F32 ? 4.0
                        : tt == 1           ? 2.2
                        : x_dtype == SFFN_BF16 ? 3.0
                                               : 1.5;
  const int64_t groups = (nb * mx4_token_groups(T, tt) + rb - 1) / rb, n = (groups + 255) / 256;
  const int64_t turns = mx4_pairs(x_dtype, tt, rb) ? (n + 1) / 2 : n;
  const double blocks = kb > MX4_WAVES ? (double)kb / MX4_WAVES : 1.0;
  const double more = tt > 2 ? tt - 2 : 0;
  return (10.0 + 3.0 * more) * (double)turns +
         (double)n * blocks * (tokens + rb) * (1.0 + 0.35 * more);
}

// The row blocks with the least estimate.  Measured, 1 / 2 / 4: one token, K 2048: N 2048 3.0 / 3.4 /
// 4.2 us, 8192 4.0 / 3.6 / 4.3; 64 tokens in 8 bits (two tiles), 1 / 2 / 3 / 4: N 8192 8.0 / 6.3 /
// 7.9 / 6.1, 9216 (K 2304) 10.6 / 10.3 / 8.0 / 10.7.
inline double mx4_best(int x_dtype, int tt, int64_t nb, int64_t kb, int64_t T, int* rb) {
  double best = mx4_cost(x_dtype, tt, *rb = 1, nb, kb, T);
  for (int i = 2; i <= 4; ++i) {
    const double c = mx4_cost(x_dtype, tt, i, nb, kb, T);
    if (c < best) {
      best = c;
      *rb = i;
    }
  }
  return best;
}

// For nb blocks of 16 rows, kb blocks of 128 columns and T tokens.
inline Mx4Shape mx4_shape(int x_dtype, int64_t nb, int64_t kb, int64_t T) {
  Mx4Shape s{1, 1, MX4_WAVES};
  if (T <= 16) {
    mx4_best(x_dtype, 1, nb, kb, T, &s.rb);
  } else {
    const double two = mx4_best(x_dtype, s.tt = 2, nb, kb, T, &s.rb);
    // All tokens at once read and expand the weights once: 32768 x 2048 with 64 in 8 bits 16 us, 18 in
    // two halves; the halves fill the GPU better for fewer rows: 9216 x 2304 8.7 and 8.0.
    const int all = T > 48 ? 4 : 3;
    int rb = 1;
    if (x_dtype != SFFN_F32 && T > 32 && mx4_best(x_dtype, all, nb, kb, T, &rb) < two) {
      s.tt = all;
      s.rb = rb;
    }
  }
  // Waves that split k cost a join, and idle beyond the blocks of columns; they take rows instead
  // while that leaves enough workgroups (65536 x 256, one token: 3.9 against 5.3 us; 65536 x 2048, 64
  // tokens in 8 bits: 28 against 33).
  const int64_t blocks = nb * mx4_token_groups(T, s.tt), enough = s.tt > 1 ? 256 : 512;
  while (s.ks > 2 && blocks * s.ks / (2 * s.rb * MX4_WAVES) >= enough) s.ks /= 2;
  return s;
}

}  // namespace sffn
