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
#include "ops_common.hpp"

namespace sffn {
namespace {

constexpr int grad_threads(int L) { return L < 256 ? 256 : L; }

// Column sums of grad_columns(B) columns over the rows of one of a.sum_parts parts, by the B threads of a
// workgroup: 64 row groups of lanes of 4 columns, joined in order.
constexpr int grad_columns(int B) { return B / 16; }
template <typename T, int B>
__device__ __forceinline__ void sum_columns(const LayerNormGradArgs& a, int blk) {
  constexpr int GROUPS = 64, LANES = B / GROUPS, COLUMNS = grad_columns(B);
  __shared__ float join[2][GROUPS][COLUMNS + 1];
  const int blocks = (a.d + COLUMNS - 1) / COLUMNS, part = blk / blocks, col0 = blk % blocks * COLUMNS;
  const int c4 = (int)(threadIdx.x % LANES) * 4, g = (int)(threadIdx.x / LANES);
  const int col = col0 + c4, n = a.d - col;
  const int64_t per = (a.rows + a.sum_parts - 1) / a.sum_parts, first = part * per;
  const int64_t last = first + per < a.rows ? first + per : a.rows;
  float sg[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int64_t row = first + g; row < last; row += GROUPS) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride + col;
    const T* h = static_cast<const T*>(a.h) + row * a.h_stride + col;
    const float rstd = a.rstd[row], mean = a.mean[row];
    float y[4], x[4];
    load4<false>(dy, n, y);
    load4<false>(h, n, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sg[i] += y[i] * ((x[i] - mean) * rstd);
      sb[i] += y[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    join[0][g][c4 + i] = sg[i];
    join[1][g][c4 + i] = sb[i];
  }
  __syncthreads();
  const int c = (int)threadIdx.x % COLUMNS, which = (int)threadIdx.x / COLUMNS;
  if (which < 2 && col0 + c < a.d) {
    float t = 0.f;
#pragma unroll 16
    for (int i = 0; i < GROUPS; ++i) t += join[which][i][c];
    float* out = a.part ? a.part + ((int64_t)part * 2 + which) * a.d : which == 0 ? a.dgain : a.dbias;
    if (out) out[col0 + c] = t;
  }
}

// B threads: B / L rows at a time, by row_groups workgroups; the ones past them sum columns.
// SUMS: the row groups sum the columns in registers, into a.part if it is given.
template <typename T, typename G, int NV, int L, int B, bool SUMS>
__global__ __launch_bounds__(B) void layer_norm_grad_kernel(LayerNormGradArgs a, int row_groups) {
  if constexpr (!SUMS) {
    if ((int)blockIdx.x >= row_groups) {
      sum_columns<T, B>(a, (int)blockIdx.x - row_groups);
      return;
    }
  }
  constexpr int RPB = B / L;
  __shared__ float red[4][L > 64 ? L / 64 : 1];
  __shared__ float join[SUMS && RPB > 1 ? RPB * 8 * L : 1];
  const int li = (int)(threadIdx.x % L), grp = (int)(threadIdx.x / L);
  const int d = a.d;
  const bool tail = (d & 7) != 0;
  const G* gain = static_cast<const G*>(a.gain);
  const float inv_d = 1.f / (float)d;

  Raw8<G> rg[NV];
  float ag[SUMS ? NV : 1][8], ab[SUMS ? NV : 1][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = (v * L + li) * 8;
    rg[v].zero();
    if (e + 8 <= d) rg[v].load(gain + e);
    else if (e < d) rg[v].load_n(gain + e, d - e);
    if constexpr (SUMS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) ag[v][i] = ab[v][i] = 0.f;
    }
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + grp; row < a.rows;
       row += (int64_t)row_groups * RPB, turn ^= 2) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
    const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
    const T* dres = static_cast<const T*>(a.dres) + row * a.dres_stride;
    const float rstd = a.rstd[row], mean = a.mean[row];
    Raw8<T> ry[NV], rh[NV], rr[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * L + li) * 8;
      ry[v].zero();
      rh[v].zero();
      if (e + 8 <= d) {
        ry[v].load(dy + e);
        rh[v].load(h + e);
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * L + li) * 8;
      rr[v].zero();
      if (a.dres && e + 8 <= d) rr[v].load(dres + e);
    }
    if (tail) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = (v * L + li) * 8;
        if (e < d && e + 8 > d) {
          ry[v].load_n(dy + e, d - e);
          rh[v].load_n(h + e, d - e);
          if (a.dres) rr[v].load_n(dres + e, d - e);
        }
      }
    }
    float st = 0.f, sx = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int n = d - (v * L + li) * 8;  // past the row's end a deviation is 0, not -mean
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = n >= 8 || (tail && i < n) ? rh[v].get(i) - mean : 0.f;
        const float y = ry[v].get(i), p = y * (c * rstd), g = rg[v].get(i);
        if constexpr (SUMS) {
          ag[v][i] += p;
          ab[v][i] += y;
        }
        st += y * g;
        sx += p * g;
      }
    }
    row_reduce2<L>(st, sx, red[turn], red[turn + 1]);
    const float ct = st * inv_d, cx = sx * inv_d;
    T* dx = static_cast<T*>(a.dx) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * L + li) * 8;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i] = rstd * (ry[v].get(i) * rg[v].get(i) - ct - (rh[v].get(i) - mean) * rstd * cx) +
               rr[v].get(i);
      if (e + 8 <= d) store8(dx + e, o);
      else if (e < d) store8_n(dx + e, o, d - e);
    }
  }
  if constexpr (SUMS) {
    if (!a.part) return;
    float* part = a.part + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if constexpr (RPB > 1) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          __syncthreads();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            join[grp * 8 * L + i * L + li] = which == 0 ? ag[v][i] : ab[v][i];
          __syncthreads();
          for (int c = (int)threadIdx.x; c < 8 * L; c += B) {
            float s = 0.f;
#pragma unroll
            for (int g = 0; g < RPB; ++g) s += join[g * 8 * L + c];
            const int col = (v * L + c % L) * 8 + c / L;
            if (col < d) part[which * d + col] = s;
          }
        }
      } else {
        const int e = (v * L + li) * 8;
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

// Where the row groups sum the columns in registers: not above 16384 columns (they would spill), and
// not for few rows, for which reading dy and h once more is less than a second launch.
bool sums_in_rows(int64_t rows, int32_t d) {
  return d <= 16384 && !(rows <= 1024 && rows * d <= 1 << 20);
}
// Workgroups of the rows: each one's partial rows cost a write and a read, so there are only as many
// as keep the memory busy, with equal numbers of rows.
int row_groups(int64_t rows, int32_t d) {
  const int L = norm_lanes(d, true), rpb = grad_threads(L) / L;
  const int64_t need = (rows + rpb - 1) / rpb;
  const int64_t most = sums_in_rows(rows, d) ? (L > 512 ? 256 : 512) : 1 << 20;
  const int64_t turns = (need + most - 1) / most;
  return (int)((need + turns - 1) / turns);
}
// Parts of the rows whose columns other workgroups sum: one where that needs no second launch.
int sum_parts(int64_t rows, int32_t d) {
  if (rows <= 1024 && rows * d <= 1 << 20) return 1;
  const int64_t parts = (rows + 1023) / 1024;
  return (int)(parts < 64 ? parts : 64);
}

template <typename T, typename G>
hipError_t launch_t(const LayerNormGradArgs& a0, hipStream_t s) {
  return norm_shape<true>(a0.d, [&](auto lanes, auto nv) {
    constexpr int L = decltype(lanes)::value, NV = decltype(nv)::value, B = grad_threads(L);
    LayerNormGradArgs a = a0;
    const int groups = row_groups(a.rows, a.d);
    if constexpr (NV * L <= 2048) {
      if (sums_in_rows(a.rows, a.d)) {
        layer_norm_grad_kernel<T, G, NV, L, B, true><<<dim3((unsigned)groups), dim3(B), 0, s>>>(a, groups);
        return hipGetLastError();
      }
    }
    a.sum_parts = sum_parts(a.rows, a.d);
    const int sums = a.dgain || a.dbias ? a.sum_parts * ((a.d + grad_columns(B) - 1) / grad_columns(B)) : 0;
    layer_norm_grad_kernel<T, G, NV, L, B, false><<<dim3((unsigned)(groups + sums)), dim3(B), 0, s>>>(a, groups);
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
