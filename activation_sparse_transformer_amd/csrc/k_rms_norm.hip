// Root-mean-square norm with the residual's sum.
//
//   h = x + residual,  rstd = 1 / sqrt(sum(h^2) / d + eps),  y = h rstd gain
//   8 bits: scale = max(max|y| / 448, 2^-126), q = e4m3(y / scale)
//
// One pass: a row's elements stay in the registers of the L lanes that loaded them (NV vectors
// of 8 a lane) between the sum of squares and the output, so x and the residual are read once
// and h, y written once.  Bound by memory: 8192 x 2048 bf16 with the residual moves 134 MB in 22.4 us
// (6.0 TB/s; a copy reaches 4.8), 16384 x 2304 with 8 bits out 264 MB in 44 us (from a trace; calls
// one after another take 24.6 and 48).
#include "ops_common.hpp"

namespace sffn {
namespace {

template <typename T, typename G, int NV, int L, bool FP8>
__global__ __launch_bounds__(L > 256 ? 1024 : 256) void rms_norm_kernel(NormArgs a) {
  constexpr int RPB = L < 256 ? 256 / L : 1;  // rows of a workgroup
  __shared__ float red[2][L > 64 ? L / 64 : 1];
  const int64_t row = (int64_t)blockIdx.x * RPB + (int)(threadIdx.x / L);
  if (row >= a.rows) return;  // whole rows; only where no barrier follows (RPB > 1)
  const int li = (int)(threadIdx.x % L);
  const int d = a.d;
  const bool tail = (d & 7) != 0;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* res = static_cast<const T*>(a.residual) + row * a.residual_stride;
  const G* gain = static_cast<const G*>(a.gain);

  Raw8<T> rx[NV], rr[NV];
  Raw8<G> rg[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = (v * L + li) * 8;
    rx[v].zero();
    rr[v].zero();
    if (e + 8 <= d) {
      rx[v].load(x + e);
      if (a.residual) rr[v].load(res + e);
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = (v * L + li) * 8;
    rg[v].zero();
    if (e + 8 <= d) rg[v].load(gain + e);
  }
  if (tail) {  // the row's last, partial vector: one lane
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * L + li) * 8;
      if (e < d && e + 8 > d) {
        rx[v].load_n(x + e, d - e);
        if (a.residual) rr[v].load_n(res + e, d - e);
        rg[v].load_n(gain + e, d - e);
      }
    }
  }
  float h[NV][8];
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[v][i] = a.residual ? rx[v].get(i) + rr[v].get(i) : rx[v].get(i);
      ss += h[v][i] * h[v][i];
    }
  }
  if (a.h) {
    T* ho = static_cast<T*>(a.h) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * L + li) * 8;
      if (e + 8 <= d) store8(ho + e, h[v]);
      else if (e < d) store8_n(ho + e, h[v], d - e);
    }
  }
  ss = row_reduce<L>(ss, Add(), red[0]);
  const float rstd = inv_rms(ss / (float)d + a.eps);
  float big = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[v][i] = h[v][i] * rstd * rg[v].get(i);
      if (FP8) big = max_abs(big, h[v][i]);
    }
  float stat = rstd;
  if constexpr (FP8) {
    // lanes past the row's end hold 0 * rstd * 0, which is NaN when rstd is not finite; the
    // row's own values are then not finite either
    big = row_reduce<L>(big, MaxNan(), red[1]);
    const float t = big / E4M3_MAX;
    stat = t < SCALE_MIN ? SCALE_MIN : t;
    const Quotients over(stat);
    uint8_t* q = static_cast<uint8_t*>(a.y) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * L + li) * 8;
      if (e >= d) continue;
      over(h[v]);
      store_e4m3x8(q + e, h[v], d - e);
    }
  } else {
    T* y = static_cast<T*>(a.y) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * L + li) * 8;
      if (e + 8 <= d) store8(y + e, h[v]);
      else if (e < d) store8_n(y + e, h[v], d - e);
    }
  }
  if (li == 0 && a.stat) a.stat[row] = stat;
}

template <typename T, typename G, bool FP8>
hipError_t launch_t(const NormArgs& a, hipStream_t s) {
  // a launch has at most 2^32 - 1 threads
  const int64_t rows = a.rows, part = 1 << 21;
  for (int64_t r = 0; r < rows; r += part) {
    NormArgs b = a;
    b.rows = rows - r < part ? rows - r : part;
    b.x = static_cast<const T*>(a.x) + r * a.x_stride;
    if (a.residual) b.residual = static_cast<const T*>(a.residual) + r * a.residual_stride;
    b.y = static_cast<char*>(a.y) + r * a.d * (FP8 ? 1 : (int64_t)sizeof(T));
    if (a.stat) b.stat = a.stat + r;
    if (a.h) b.h = static_cast<T*>(a.h) + r * a.d;
    const hipError_t e = norm_shape<false>(a.d, [&](auto lanes, auto nv) {
      constexpr int L = decltype(lanes)::value, NV = decltype(nv)::value;
      constexpr int RPB = L < 256 ? 256 / L : 1;
      rms_norm_kernel<T, G, NV, L, FP8>
          <<<dim3((unsigned)((b.rows + RPB - 1) / RPB)), dim3(L > 256 ? L : 256), 0, s>>>(b);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_rms_norm(bool bf16, bool gain_f32, bool fp8, const NormArgs& a, hipStream_t s) {
  if (!bf16) return fp8 ? launch_t<float, float, true>(a, s) : launch_t<float, float, false>(a, s);
  if (gain_f32)
    return fp8 ? launch_t<uint16_t, float, true>(a, s) : launch_t<uint16_t, float, false>(a, s);
  return fp8 ? launch_t<uint16_t, uint16_t, true>(a, s)
             : launch_t<uint16_t, uint16_t, false>(a, s);
}

}  // namespace sffn
