// Gradient of the layer norm.  With xh = (h - mean) rstd and t = dy gain:
//
//   dx = rstd (t - mean(t) - xh mean(t xh)) + dres
//   dgain[c] = sum over rows of dy[., c] xh[., c],   dbias[c] = sum over rows of dy[., c]
//
// One pass over dy, h and dres: the L lanes of a row keep its elements in registers between the
// row's two sums (reduced together) and dx.  A lane sees the same columns in every row its group
// takes, so it sums dgain and dbias in registers too; a workgroup joins its row groups in LDS in a
// fixed order and writes one partial row of each, and a second kernel adds the partial rows in
// order (no atomics: the result depends on the sizes alone).  Where registers do not hold the
// column sums (above 16384 columns), or where the second launch would take longer than reading a
// few rows twice, further workgroups of the first launch sum the columns from dy and h themselves.
// Bound by memory: 16384 x 2304 bf16 with dres moves 302 MB in 55.5 us (5.4 TB/s, both launches, replays of
// calls one after another; in a trace their medians are 60.5 and 4.8; about 5 more without the next row's loads
// in flight), 8192 x 4096 268 MB in 45.6; fp32 604 MB in 115 and 537 MB in 102 (5.3 TB/s).  Above 8192
// columns a lane has two vectors and no registers for the next row (2048 x 16384: 59 us, 4.5 TB/s; fp32, which
// spills 40 registers, 128 us, 4.2 TB/s).  Above 16384 dy and h are read twice, the second time in strips of
// 16 columns, which in bf16 are a quarter of a line (1024 x 32768: 134 us; fp32 233).
#include "ops_common.hpp"

namespace sffn {
namespace {

using namespace ln_grad;

// Column sums of GRAD_COLUMNS columns over the rows of one of a.sum_parts parts, by a workgroup of any
// number of waves: every 4 lanes take a row, 4 columns each; the 16 rows of a wave are joined by lane
// rotations, the waves in LDS, in order.
constexpr int GRAD_COLUMNS = 16;
template <typename T>
__device__ __forceinline__ void sum_columns(const LayerNormGradArgs& a, int blk) {
  __shared__ float join[2][16][GRAD_COLUMNS];
  const int groups = (int)blockDim.x / 4, waves = (int)blockDim.x / 64;
  const int blocks = (a.d + GRAD_COLUMNS - 1) / GRAD_COLUMNS;
  const int part = blk / blocks, col0 = blk % blocks * GRAD_COLUMNS;
  const int c4 = (int)(threadIdx.x & 3) * 4, g = (int)(threadIdx.x >> 2);
  const int col = col0 + c4, n = a.d - col;
  const int64_t per = (a.rows + a.sum_parts - 1) / a.sum_parts, first = part * per;
  const int64_t last = first + per < a.rows ? first + per : a.rows;
  float s[2][4] = {};
#pragma unroll 4
  for (int64_t row = first + g; row < last; row += groups) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride + col;
    const T* h = static_cast<const T*>(a.h) + row * a.h_stride + col;
    const float rstd = a.rstd[row], mean = a.mean[row];
    float y[4], x[4];
    load4<false>(dy, n, y);
    load4<false>(h, n, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[0][i] += y[i] * ((x[i] - mean) * rstd);
      s[1][i] += y[i];
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v = s[k][i];
      v += dpp<0x128>(v);  // rotations of a row's 16 lanes by 8 and by 4
      v += dpp<0x124>(v);
      v = rows_reduce(v, Add());
      if ((threadIdx.x & 63) < 4) join[k][threadIdx.x >> 6][c4 + i] = v;
    }
  __syncthreads();
  const int c = (int)threadIdx.x % GRAD_COLUMNS, which = (int)threadIdx.x / GRAD_COLUMNS;
  if (which < 2 && col0 + c < a.d) {
    float t = join[which][0][c];
    for (int i = 1; i < waves; ++i) t += join[which][i][c];
    float* out = a.part ? a.part + ((int64_t)part * 2 + which) * a.d : which == 0 ? a.dgain : a.dbias;
    if (out) out[col0 + c] = t;
  }
}

// A workgroup takes blockDim / lanes rows at a time, L lanes each, or with L = 0 row_waves waves;
// row_groups workgroups take the rows in turn, the ones past them sum columns.  SUMS: the row groups
// sum the columns in registers, into a.part if it is given.  With one vector a lane, a row is loaded
// while the one before it is reduced and written.
template <typename T, typename G, int NV, int L, bool SUMS>
__global__ __launch_bounds__(1024) void layer_norm_grad_kernel(LayerNormGradArgs a, int row_groups,
                                                               int row_waves) {
  if constexpr (!SUMS) {
    if ((int)blockIdx.x >= row_groups) {
      sum_columns<T>(a, (int)blockIdx.x - row_groups);
      return;
    }
  }
  constexpr bool AHEAD = SUMS && NV == 1, ONE = L == 1024;
  __shared__ float red[4][16];
  __shared__ float join[SUMS && !ONE ? 8 * 1024 : 1];
  const int lanes = L > 0 ? L : 64 * row_waves;
  const int grp = ONE ? 0 : L > 0 ? (int)threadIdx.x / L : uniform((int)threadIdx.x / lanes);
  const int li = (int)threadIdx.x - grp * lanes, rpb = ONE ? 1 : (int)blockDim.x / lanes;
  const int d = a.d;
  const bool tail = (d & 7) != 0;
  const G* gain = static_cast<const G*>(a.gain);
  const float inv_d = 1.f / (float)d;

  // gains of more than two vectors a lane are loaded where they are needed
  constexpr bool HELD = NV <= 2;
  Raw8<G> rg[NV];
  const auto load_gain = [&](int v) {
    const int e = (v * lanes + li) * 8;
    rg[v].zero();
    if (e + 8 <= d) rg[v].load(gain + e);
    else if (e < d) rg[v].load_n(gain + e, d - e);
  };
  float ag[SUMS ? NV : 1][8], ab[SUMS ? NV : 1][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if constexpr (HELD) load_gain(v);
    if constexpr (SUMS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) ag[v][i] = ab[v][i] = 0.f;
    }
  }
  Raw8<T> ry[NV], rh[NV], rr[NV];
  float rstd = 0.f, mean = 0.f;
  const auto load = [&](int64_t row) {  // past the last row: nothing, which adds nothing
    const bool have = ONE || row < a.rows;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
    const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
    const T* dres = static_cast<const T*>(a.dres) + row * a.dres_stride;
    if (!ONE) rstd = mean = 0.f;
    if (have) {
      rstd = a.rstd[row];
      mean = a.mean[row];
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * lanes + li) * 8;
      ry[v].zero();
      rh[v].zero();
      if (have && e + 8 <= d) {
        ry[v].load(dy + e);
        rh[v].load(h + e);
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * lanes + li) * 8;
      rr[v].zero();
      if (a.dres && have && e + 8 <= d) rr[v].load(dres + e);
    }
    if (tail) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = (v * lanes + li) * 8;
        if (have && e < d && e + 8 > d) {
          ry[v].load_n(dy + e, d - e);
          rh[v].load_n(h + e, d - e);
          if (a.dres) rr[v].load_n(dres + e, d - e);
        }
      }
    }
  };
  const int64_t step = (int64_t)row_groups * rpb;
  int turn = 0;
  if constexpr (AHEAD) load((int64_t)blockIdx.x * rpb + grp);
  for (int64_t row0 = (int64_t)blockIdx.x * rpb; row0 < a.rows; row0 += step, turn ^= 2) {
    const int64_t row = row0 + grp;
    if constexpr (!AHEAD) load(row);
    // what the output needs of this row, when the next one's loads take the place of its own
    float t[AHEAD ? 8 : 1], xh[AHEAD ? 8 : 1], res[AHEAD ? 8 : 1];
    const float rs = rstd;
    float st = 0.f, sx = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int n = d - (v * lanes + li) * 8;  // past the row's end a deviation is 0, not -mean
      if constexpr (!HELD) load_gain(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = n >= 8 || (tail && i < n) ? (rh[v].get(i) - mean) * rs : 0.f;
        const float y = ry[v].get(i), p = y * c, g = rg[v].get(i);
        if constexpr (SUMS) {
          ag[v][i] += p;
          ab[v][i] += y;
        }
        st += y * g;
        sx += p * g;
        if constexpr (AHEAD) {
          t[i] = y * g;
          xh[i] = c;
          res[i] = rr[v].get(i);
        }
      }
    }
    if constexpr (AHEAD) load(row + step);
    if constexpr (L == 0 || L == 1024) {
      group_sum2(st, sx, red[turn], red[turn + 1], L == 0 ? row_waves : 16, L == 0 ? grp * row_waves : 0);
    } else {
      st = lane_reduce<L>(st, Add());
      sx = lane_reduce<L>(sx, Add());
    }
    if (!ONE && row >= a.rows) continue;  // (of the last turn; the barrier is behind)
    const float ct = st * inv_d, cx = sx * inv_d;
    T* dx = static_cast<T*>(a.dx) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * lanes + li) * 8;
      if constexpr (!HELD) load_gain(v);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (AHEAD) o[i] = rs * (t[i] - ct - xh[i] * cx) + res[i];
        else o[i] = rs * (ry[v].get(i) * rg[v].get(i) - ct - (rh[v].get(i) - mean) * rs * cx) + rr[v].get(i);
      }
      if (e + 8 <= d) store8(dx + e, o);
      else if (e < d) store8_n(dx + e, o, d - e);
    }
  }
  if constexpr (SUMS) {
    if (!a.part) return;
    float* part = a.part + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!ONE && rpb > 1) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          __syncthreads();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            join[(grp * 8 + i) * lanes + li] = which == 0 ? ag[v][i] : ab[v][i];
          __syncthreads();
          for (int c = (int)threadIdx.x; c < 8 * lanes; c += (int)blockDim.x) {
            float s = 0.f;
            for (int g = 0; g < rpb; ++g) s += join[g * 8 * lanes + c];
            const int col = (v * lanes + c % lanes) * 8 + c / lanes;
            if (col < d) part[which * d + col] = s;
          }
        }
      } else {
        const int e = (v * lanes + li) * 8;
        if (e + 8 <= d) {
          store8(part + e, ag[v]);
          store8(part + d + e, ab[v]);
        } else if (e < d) {
          store8_n(part + e, ag[v], d - e);
          store8_n(part + d + e, ab[v], d - e);
        }
      }
    }
  }
}

// 32 of the 2 d columns of a workgroup; 32 row groups of 32 lanes each read every 32nd partial row.
__global__ __launch_bounds__(1024) void layer_norm_grad_sum_kernel(const float* part, int n,
                                                                   int32_t d, float* dgain,
                                                                   float* dbias) {
  __shared__ float join[32][33];
  const int c = (int)(threadIdx.x & 31), g = (int)(threadIdx.x >> 5);
  const int col = (int)blockIdx.x * 32 + c;
  float s = 0.f;
  if (col < 2 * d) {
#pragma unroll 4
    for (int r = g; r < n; r += 32) s += part[(int64_t)r * 2 * d + col];
  }
  join[g][c] = s;
  __syncthreads();
  if (g == 0 && col < 2 * d) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += join[i][c];
    float* out = col < d ? dgain : dbias;
    if (out) out[col < d ? col : col - d] = t;
  }
}

template <typename T, typename G>
hipError_t launch_t(const LayerNormGradArgs& a0, hipStream_t s) {
  const GradShape shape = grad_shape(a0.d);
  return with_row_shape<1024>(shape.row, [&](auto lanes, auto nv) {
    constexpr int L = decltype(lanes)::value, NV = decltype(nv)::value;
    LayerNormGradArgs a = a0;
    const int groups = row_groups(a.rows, a.d);
    const dim3 threads((unsigned)shape.threads());
    if constexpr (NV <= 2) {
      if (sums_in_rows(a.rows, a.d)) {
        layer_norm_grad_kernel<T, G, NV, L, true>
            <<<dim3((unsigned)groups), threads, 0, s>>>(a, groups, shape.row.waves);
        return hipGetLastError();
      }
    }
    a.sum_parts = sum_parts(a.rows, a.d);
    const int blocks = (a.d + GRAD_COLUMNS - 1) / GRAD_COLUMNS;
    const int sums = a.dgain || a.dbias ? a.sum_parts * blocks : 0;
    layer_norm_grad_kernel<T, G, NV, L, false>
        <<<dim3((unsigned)(groups + sums)), threads, 0, s>>>(a, groups, shape.row.waves);
    return hipGetLastError();
  });
}

}  // namespace

int layer_norm_grad_parts(int64_t rows, int32_t d) {
  if (rows == 0) return 0;
  if (sums_in_rows(rows, d)) return row_groups(rows, d);
  const int n = sum_parts(rows, d);
  return n > 1 ? n : 0;
}

hipError_t launch_layer_norm_grad(bool bf16, bool gain_f32, const LayerNormGradArgs& a,
                                  hipStream_t s) {
  if (!bf16) return launch_t<float, float>(a, s);
  return gain_f32 ? launch_t<uint16_t, float>(a, s) : launch_t<uint16_t, uint16_t>(a, s);
}

hipError_t launch_layer_norm_grad_sum(const float* part, int n, int32_t d, float* dgain,
                                      float* dbias, hipStream_t s) {
  layer_norm_grad_sum_kernel<<<dim3((unsigned)((2 * (int64_t)d + 31) / 32)), 1024, 0, s>>>(
      part, n, d, dgain, dbias);
  return hipGetLastError();
}

}  // namespace sffn
