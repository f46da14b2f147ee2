// Gradient of the root-mean-square norm.  With xh = h rstd and t = dy gain:
//
//   dx = rstd (t - xh mean(t xh)) + dres,   dgain[c] = sum over rows of dy[., c] xh[., c]
//
// One pass over dy, h and dres: the L lanes of a row keep its elements in registers between the
// row's sum and dx.  A lane sees the same columns in every row its group takes, so it sums
// dgain in registers too; a workgroup joins its row groups in LDS in a fixed order and writes
// one partial row, and a second kernel adds the partial rows in order (no atomics: the result
// depends on the sizes alone).  Bound by memory: 16384 x 2304 bf16 with dres moves 302 MB in
// 55 us (5.5 TB/s), the second kernel takes 4.8 (from a trace).  Above 16384 columns a lane's arrays no
// longer fit its 128 registers and spill: 1024 x 32768 takes 186 us for 270 MB.  (Loading a lane's next row before this one is
// reduced helped 8192 x 4096 by 3 us and cost 16384 x 2304 as much.)
#include "ops_common.hpp"

namespace sffn {
namespace {

// dgain of grad_columns(B) columns over all rows, by the B threads of a workgroup: 64 row groups
// of lanes of 4 columns, joined in order.
constexpr int grad_columns(int B) { return B / 16; }
template <typename T, int B>
__device__ __forceinline__ void sum_columns(const NormGradArgs& a, int blk) {
  constexpr int GROUPS = 64, LANES = B / GROUPS, COLUMNS = grad_columns(B);
  __shared__ float join[GROUPS][COLUMNS + 1];
  const int c4 = (int)(threadIdx.x % LANES) * 4, g = (int)(threadIdx.x / LANES);
  const int col = blk * COLUMNS + c4, n = a.d - col;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int64_t row = g; row < a.rows; row += GROUPS) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride + col;
    const T* h = static_cast<const T*>(a.h) + row * a.h_stride + col;
    const float rstd = a.rstd[row];
    float y[4], x[4];
    load4<false>(dy, n, y);
    load4<false>(h, n, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] += y[i] * (x[i] * rstd);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) join[g][c4 + i] = s[i];
  __syncthreads();
  const int c = (int)threadIdx.x;
  if (c < COLUMNS && blk * COLUMNS + c < a.d) {
    float t = 0.f;
#pragma unroll 16
    for (int i = 0; i < GROUPS; ++i) t += join[i][c];
    a.dgain[blk * COLUMNS + c] = t;
  }
}

// B threads: B / L rows at a time, by row_groups workgroups; the ones past them sum dgain.
template <typename T, typename G, int NV, int L, int B>
__global__ __launch_bounds__(B) void rms_norm_grad_kernel(NormGradArgs a, int row_groups) {
  if ((int)blockIdx.x >= row_groups) {
    sum_columns<T, B>(a, (int)blockIdx.x - row_groups);
    return;
  }
  constexpr int RPB = B / L;
  __shared__ float red[2][L > 64 ? L / 64 : 1];
  __shared__ float join[RPB > 1 ? RPB * 8 * L : 1];
  const int li = (int)(threadIdx.x % L), grp = (int)(threadIdx.x / L);
  const int d = a.d;
  const bool tail = (d & 7) != 0;
  const G* gain = static_cast<const G*>(a.gain);
  const float inv_d = 1.f / (float)d;

  Raw8<G> rg[NV];
  float acc[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = (v * L + li) * 8;
    rg[v].zero();
    if (e + 8 <= d) rg[v].load(gain + e);
    else if (e < d) rg[v].load_n(gain + e, d - e);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v][i] = 0.f;
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + grp; row < a.rows;
       row += (int64_t)row_groups * RPB, turn ^= 1) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
    const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
    const T* dres = static_cast<const T*>(a.dres) + row * a.dres_stride;
    const float rstd = a.rstd[row];
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
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = ry[v].get(i) * (rh[v].get(i) * rstd);
        acc[v][i] += p;
        dot += p * rg[v].get(i);
      }
    dot = row_reduce<L>(dot, Add(), red[turn]);
    const float c = dot * inv_d;
    T* dx = static_cast<T*>(a.dx) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * L + li) * 8;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i] = rstd * (ry[v].get(i) * rg[v].get(i) - rh[v].get(i) * rstd * c) + rr[v].get(i);
      if (e + 8 <= d) store8(dx + e, o);
      else if (e < d) store8_n(dx + e, o, d - e);
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * d;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) join[grp * 8 * L + i * L + li] = acc[v][i];
      __syncthreads();
      for (int c = (int)threadIdx.x; c < 8 * L; c += B) {
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < RPB; ++g) s += join[g * 8 * L + c];
        const int col = (v * L + c % L) * 8 + c / L;
        if (col < d) part[col] = s;
      }
    } else {
      const int e = (v * L + li) * 8;
      if (e + 8 <= d) store8(part + e, acc[v]);
      else if (e < d) store8_n(part + e, acc[v], d - e);
    }
  }
}

// 32 columns of a workgroup; 32 row groups of 32 lanes each read every 32nd partial row.
__global__ __launch_bounds__(1024) void rms_norm_grad_sum_kernel(const float* part, int n,
                                                                 int32_t d, float* dgain) {
  __shared__ float join[32][33];
  const int c = (int)(threadIdx.x & 31), g = (int)(threadIdx.x >> 5);
  const int col = (int)blockIdx.x * 32 + c;
  float s = 0.f;
  if (col < d) {
#pragma unroll 4
    for (int r = g; r < n; r += 32) s += part[(int64_t)r * d + col];
  }
  join[g][c] = s;
  __syncthreads();
  if (g == 0 && col < d) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += join[i][c];
    dgain[col] = t;
  }
}

constexpr int norm_grad_threads(int L) { return L < 256 ? 256 : L; }

// Whether dgain's columns are summed by further workgroups of the same launch, which read dy and h
// once more: for few rows that is less than a second launch (333 x 1537 fp32: a call 12.9 us with
// two).
bool one_launch(int64_t rows, int32_t d) { return rows <= 1024 && rows * d <= 1 << 20; }

// Each workgroup's partial row costs a write and a read, so there are only as many as keep the
// memory busy (16384 x 2304: 512 take 59.8 us, 768 63.4, 384 67.9), with equal numbers of rows.
int row_groups(int64_t rows, int32_t d) {
  const int L = norm_lanes(d, true), rpb = norm_grad_threads(L) / L;
  const int64_t need = (rows + rpb - 1) / rpb, most = L > 512 ? 256 : 512;
  if (one_launch(rows, d)) return (int)need;
  const int64_t turns = (need + most - 1) / most;
  return (int)((need + turns - 1) / turns);
}

template <typename T, typename G>
hipError_t launch_t(const NormGradArgs& a, hipStream_t s) {
  return norm_shape<true>(a.d, [&](auto lanes, auto nv) {
    constexpr int L = decltype(lanes)::value, NV = decltype(nv)::value, B = norm_grad_threads(L);
    const int groups = row_groups(a.rows, a.d),
              columns = a.dgain && !a.part ? (a.d + grad_columns(B) - 1) / grad_columns(B) : 0;
    rms_norm_grad_kernel<T, G, NV, L, B><<<dim3((unsigned)(groups + columns)), dim3(B), 0, s>>>(
        a, groups);
    return hipGetLastError();
  });
}

}  // namespace

int norm_grad_groups(int64_t rows, int32_t d) {
  return one_launch(rows, d) ? 0 : row_groups(rows, d);
}

hipError_t launch_rms_norm_grad(bool bf16, bool gain_f32, const NormGradArgs& a, hipStream_t s) {
  if (!bf16) return launch_t<float, float>(a, s);
  return gain_f32 ? launch_t<uint16_t, float>(a, s) : launch_t<uint16_t, uint16_t>(a, s);
}

hipError_t launch_rms_norm_grad_sum(const float* part, int n, int32_t d, float* dgain,
                                    hipStream_t s) {
  rms_norm_grad_sum_kernel<<<dim3((unsigned)((d + 31) / 32)), 1024, 0, s>>>(part, n, d, dgain);
  return hipGetLastError();
}

}  // namespace sffn
