// How the layer norm's kernels share a row among lanes, and which of its gradient's forms take which sizes.
// By itself, so that a host test can check the rules and the sizes that the GPU tests run.
#pragma once

#include <stdint.h>

namespace sffn {

// How a layer norm's kernels share a row of d elements: L lanes (16, 32, 64; several rows a
// workgroup), or L = 0: `waves` whole waves, as many as the row's vectors of 8 need at nv a lane.
struct RowShape {
  int lanes, waves, nv;
};
constexpr int rows_of(int lanes) { return lanes == 0 ? 1 : 256 / (lanes + (lanes == 0)); }  // of 4 waves
// wide: 16 elements a lane also where 8 would do (bf16 rows of the forward: 16384 x 2304 takes 51.8 us
// and 45.9 with 8 bits out, 54.9 and 54.9 with 8; fp32 rows, with as many bytes in 8, lose 2%).
inline RowShape row_shape(int32_t d, bool wide) {
  if (d <= 128) return {16, 4, 1};
  if (d <= 256) return {32, 4, 1};
  if (d <= 512) return {64, 4, 1};
  const int units = (d + 511) / 512;
  int nv = (units + 15) / 16;
  if (wide && nv < 2) nv = 2;
  return {0, (units + nv - 1) / nv, nv};
}

namespace ln_grad {
// Where the row groups sum the columns in registers: not above 16384 columns (they would spill), and
// not for few rows, for which reading dy and h once more is less than a second launch.  (us, bf16, read again
// and in registers: 512 x 2048 4.8 and 10.5, 1024 x 1024 5.4 and 9.0; past the border 1024 x 2048 10.6 and 11.8,
// 2048 x 512 6.2 and 7.0, but 2048 x 1024 13.7 and 10.1, 4096 x 128 8.0 and 6.2; fp32: 1024 x 1024 9.5 and 9.6,
// 1024 x 2048 13.2 and 13.2, 2048 x 512 8.4 and 7.5.)
inline bool few_rows(int64_t rows, int32_t d) { return rows <= 1024 && rows * d <= 1 << 20; }
inline bool sums_in_rows(int64_t rows, int32_t d) { return d <= 16384 && !few_rows(rows, d); }
// Rows of a workgroup: as few as make 8 waves.  (With 256 workgroups, 16384 x 2304 bf16 in 2 x 5 waves
// takes 56.4 us, in 5 69, in 3 x 5 57.4; 8192 x 4096 in 8 44.9, in 16 49.1.)
struct GradShape {
  RowShape row;
  int rows;
  int threads() const { return rows * (row.lanes > 0 ? row.lanes : 64 * row.waves); }
};
inline GradShape grad_shape(int32_t d) {
  const RowShape r = row_shape(d, false);
  if (r.nv > 1) return {{1024, 16, r.nv}, 1};  // (registers: a fixed number of lanes takes fewer)
  return {r, r.lanes > 0 ? 512 / r.lanes : (8 + r.waves - 1) / r.waves};
}
// Workgroups of the rows: one for a CU, with equal numbers of rows.  More would write and read more
// partial rows (16384 x 2304: 512 take 63.4 us, 384 unequally spread over the CUs 77).
inline int row_groups(int64_t rows, int32_t d) {
  const int rpb = grad_shape(d).rows;
  const int64_t need = (rows + rpb - 1) / rpb;
  const int64_t most = sums_in_rows(rows, d) ? 256 : 1 << 20;
  const int64_t turns = (need + most - 1) / most;
  return (int)((need + turns - 1) / turns);
}
// Parts of the rows whose columns other workgroups sum: one where that needs no second launch.
inline int sum_parts(int64_t rows, int32_t d) {
  if (few_rows(rows, d)) return 1;
  const int64_t parts = (rows + 1023) / 1024;
  return (int)(parts < 64 ? parts : 64);
}
}  // namespace ln_grad

}  // namespace sffn
