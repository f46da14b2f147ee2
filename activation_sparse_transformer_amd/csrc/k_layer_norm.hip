// Layer norm with the residual's sum.
//
//   h = x + residual,  mean = sum(h) / d,  var = sum((h - mean)^2) / d
//   rstd = 1 / sqrt(var + eps),  y = (h - mean) rstd gain + bias
//   8 bits: scale = max(max|y| / 448, 2^-126), q = e4m3(y / scale)
//
// One pass over memory: a row's elements stay in the registers of the L lanes that loaded them (NV
// vectors of 8 a lane) through two reductions, that of the values and that of their deviations.
// What rounding left in the first mean, the sum of the deviations c = sum(h - mean) / d, corrects
// both statistics: mean + c and var - c^2.  Bound by memory: 8192 x 2048 bf16 with the residual and
// the bias moves 134 MB in 22.5 us, 16384 x 2304 302 MB in 53 (5.7 TB/s), with 8 bits out 264 MB in 47; fp32
// 268 MB in 42.5, 604 MB in 114 (5.3 TB/s) and 491 MB in 93 (replays of calls one after another into given
// outputs).  Above 16384 columns fewer bytes are in flight: 1024 x 32768 50 us in bf16, 122 in fp32 (4.4 TB/s).
#include "ops_common.hpp"

namespace sffn {
namespace {

// Gain and bias of more than two vectors a lane are loaded when they are needed: 1024 threads
// have 128 registers each.
constexpr bool early_gain(int nv, int size) { return nv * size <= 4; }

template <typename T, typename G, int NV, int L, bool FP8>
__global__ __launch_bounds__(L > 0 ? 256 : 1024) void layer_norm_kernel(LayerNormArgs a) {
  constexpr int RPB = rows_of(L);
  __shared__ float red[4][16];
  const int lanes = L > 0 ? L : (int)blockDim.x;
  const int64_t row = (int64_t)blockIdx.x * RPB + (L > 0 ? (int)threadIdx.x / lanes : 0);
  if (row >= a.rows) return;  // whole rows; only where no barrier follows (RPB > 1)
  const int li = L > 0 ? (int)threadIdx.x % lanes : (int)threadIdx.x;
  const int d = a.d;
  const bool tail = (d & 7) != 0;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* res = static_cast<const T*>(a.residual) + row * a.residual_stride;
  const G* gain = static_cast<const G*>(a.gain);
  const G* bias = static_cast<const G*>(a.bias);

  Raw8<T> rx[NV], rr[NV];
  Raw8<G> rg[NV], rb[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = (v * lanes + li) * 8;
    rx[v].zero();
    rr[v].zero();
    if (e + 8 <= d) {
      rx[v].load(x + e);
      if (a.residual) rr[v].load(res + e);
    }
  }
  const auto load_gain = [&] {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * lanes + li) * 8;
      rg[v].zero();
      rb[v].zero();
      if (e + 8 <= d) {
        rg[v].load(gain + e);
        if (a.bias) rb[v].load(bias + e);
      } else if (e < d) {
        rg[v].load_n(gain + e, d - e);
        if (a.bias) rb[v].load_n(bias + e, d - e);
      }
    }
  };
  if constexpr (early_gain(NV, sizeof(T))) load_gain();
  if (tail) {  // the row's last, partial vector: one lane
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * lanes + li) * 8;
      if (e < d && e + 8 > d) {
        rx[v].load_n(x + e, d - e);
        if (a.residual) rr[v].load_n(res + e, d - e);
      }
    }
  }
  float h[NV][8];
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[v][i] = a.residual ? rx[v].get(i) + rr[v].get(i) : rx[v].get(i);
      sum += h[v][i];
    }
  }
  if (a.h) {
    T* ho = static_cast<T*>(a.h) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * lanes + li) * 8;
      if (e + 8 <= d) store8(ho + e, h[v]);
      else if (e < d) store8_n(ho + e, h[v], d - e);
    }
  }
  const float m0 = group_reduce<L>(sum, Add(), red[0]) / (float)d;
  float dev = 0.f, ss = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int n = d - (v * lanes + li) * 8;  // elements of the vector
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[v][i] = n >= 8 || (tail && i < n) ? h[v][i] - m0 : 0.f;
      dev += h[v][i];
      ss += h[v][i] * h[v][i];
    }
  }
  if constexpr (L == 0) {
    group_sum2(dev, ss, red[1], red[2], (int)(blockDim.x >> 6), 0);
  } else {
    dev = lane_reduce<L>(dev, Add());
    ss = lane_reduce<L>(ss, Add());
  }
  const float c = dev / (float)d;
  const float var = ss / (float)d - c * c;
  const float rstd = inv_rms((var < 0.f ? 0.f : var) + a.eps);
  if constexpr (!early_gain(NV, sizeof(T))) load_gain();
  float big = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[v][i] = (h[v][i] - c) * rstd * rg[v].get(i) + rb[v].get(i);
      if (FP8) big = max_abs(big, h[v][i]);
    }
  if constexpr (FP8) {
    // lanes past the row's end hold (0 - c) rstd 0, which is NaN where c rstd is not finite; c is a
    // rounding error of the mean, so the row's own values are then not finite either
    big = group_reduce<L>(big, MaxNan(), red[3]);
    const float t = big / E4M3_MAX;
    const float scale = t < SCALE_MIN ? SCALE_MIN : t;
    const Quotients over(scale);
    uint8_t* q = static_cast<uint8_t*>(a.y) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * lanes + li) * 8;
      if (e >= d) continue;
      over(h[v]);
      store_e4m3x8(q + e, h[v], d - e);
    }
    if (li == 0) a.stat[row] = scale;
  } else {
    T* y = static_cast<T*>(a.y) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * lanes + li) * 8;
      if (e + 8 <= d) store8(y + e, h[v]);
      else if (e < d) store8_n(y + e, h[v], d - e);
    }
    if (li == 0) {
      if (a.mean) a.mean[row] = m0 + c;
      if (a.stat) a.stat[row] = rstd;
    }
  }
}

template <typename T, typename G, bool FP8>
hipError_t launch_t(const LayerNormArgs& a, hipStream_t s) {
  // a launch has at most 2^32 - 1 threads
  const int64_t rows = a.rows, part = 1 << 21;
  for (int64_t r = 0; r < rows; r += part) {
    LayerNormArgs b = a;
    b.rows = rows - r < part ? rows - r : part;
    b.x = static_cast<const T*>(a.x) + r * a.x_stride;
    if (a.residual) b.residual = static_cast<const T*>(a.residual) + r * a.residual_stride;
    b.y = static_cast<char*>(a.y) + r * a.d * (FP8 ? 1 : (int64_t)sizeof(T));
    if (a.mean) b.mean = a.mean + r;
    if (a.stat) b.stat = a.stat + r;
    if (a.h) b.h = static_cast<T*>(a.h) + r * a.d;
    const RowShape shape = row_shape(a.d, sizeof(T) == 2);
    const hipError_t e = with_row_shape<0>(shape, [&](auto lanes, auto nv) {
      constexpr int L = decltype(lanes)::value, NV = decltype(nv)::value;
      constexpr int RPB = rows_of(L);
      layer_norm_kernel<T, G, NV, L, FP8>
          <<<dim3((unsigned)((b.rows + RPB - 1) / RPB)), dim3(64 * shape.waves), 0, s>>>(b);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_layer_norm(bool bf16, bool gain_f32, bool fp8, const LayerNormArgs& a,
                             hipStream_t s) {
  if (!bf16) return fp8 ? launch_t<float, float, true>(a, s) : launch_t<float, float, false>(a, s);
  if (gain_f32)
    return fp8 ? launch_t<uint16_t, float, true>(a, s) : launch_t<uint16_t, float, false>(a, s);
  return fp8 ? launch_t<uint16_t, uint16_t, true>(a, s)
             : launch_t<uint16_t, uint16_t, false>(a, s);
}

}  // namespace sffn
