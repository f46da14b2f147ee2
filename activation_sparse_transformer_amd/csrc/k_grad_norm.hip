// Norm of many gradients together, and their scaling by the factor that clips it.
//
//   norm = sqrt(sum g^2),  factor = norm <= max_norm ? 1 : max_norm / norm,  out = g factor
//
// The norm reads every gradient once, so memory bounds it.  A workgroup sums the squares of one
// chunk of one tensor in 64 bits (the square of an fp32 value is exact there and cannot overflow or
// vanish; a product and sum in 64 bits costs the vector units less time than the load) and writes one
// partial sum; a second kernel of one workgroup adds those in order.  No atomics: the result depends
// on the sizes alone.
#include "ops_common.hpp"

namespace sffn {
namespace {

template <typename T>
__device__ __forceinline__ void add_squares(const Raw8<T>& r, double (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double v = (double)r.get(i);
    s[i & 3] = fma(v, v, s[i & 3]);
  }
}

// The lanes take vectors of 8 in turn, four of them in flight.
template <typename T>
__device__ __forceinline__ double sum_squares(const T* g, int64_t n) {
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  const int64_t whole = n / 8;
  int64_t i = threadIdx.x;
  for (; i + 3 * 256 < whole; i += 4 * 256) {
    Raw8<T> r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k].load(g + (i + k * 256) * 8);
#pragma unroll
    for (int k = 0; k < 4; ++k) add_squares(r[k], s);
  }
  for (; i < whole; i += 256) {
    Raw8<T> r;
    r.load(g + i * 8);
    add_squares(r, s);
  }
  if (i == whole && n % 8 != 0) {
    Raw8<T> r;
    r.load_n(g + whole * 8, (int)(n % 8));
    add_squares(r, s);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// The tensor of a workgroup: the last one whose first workgroup is not past it.
template <int N>
__device__ __forceinline__ int tensor_of(const uint32_t (&first)[N], uint32_t wg) {
  const int lane = (int)(threadIdx.x & 63);
  int n = 0;
#pragma unroll
  for (int b = 0; b < N; b += 64) {
    const bool in = b + lane < N;
    n += __popcll(ballot64(in && first[in ? b + lane : 0] <= wg));
  }
  return uniform(n - 1);
}

__global__ __launch_bounds__(256) void grad_norm_kernel(GradTable tab) {
  __shared__ double red[4];
  const uint32_t wg = blockIdx.x;
  const int t = tensor_of(tab.first, wg);
  const int64_t e0 = (int64_t)(wg - tab.first[t]) * tab.chunk, all = tab.n[t];
  const int64_t left = (all < 0 ? -all : all) - e0, n = left < tab.chunk ? left : tab.chunk;
  const double s = all < 0 ? sum_squares(static_cast<const uint16_t*>(tab.grad[t]) + e0, n)
                           : sum_squares(static_cast<const float*>(tab.grad[t]) + e0, n);
  const double w = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = w;
  __syncthreads();
  if (threadIdx.x == 0) tab.part[wg] = (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ __launch_bounds__(1024) void grad_norm_sum_kernel(const double* part, int64_t n,
                                                             double max_norm, float* norm,
                                                             float* factor) {
  __shared__ double red[16];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += part[i];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  s = 0.0;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += red[i];
  const float r = (float)sqrt(s);
  norm[0] = r;
  if (factor) factor[0] = (double)r <= max_norm ? 1.f : (float)(max_norm / (double)r);
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const T* g, T* o, int64_t n, float f) {
  const int count = n < SCALE_CHUNK ? (int)n : SCALE_CHUNK;
  constexpr int STEPS = SCALE_CHUNK / (256 * 8);
  Raw8<T> r[STEPS];
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const int e = (k * 256 + (int)threadIdx.x) * 8;
    if (e + 8 <= count) r[k].load(g + e);
    else if (e < count) r[k].load_n(g + e, count - e);
  }
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const int e = (k * 256 + (int)threadIdx.x) * 8;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r[k].get(i) * f;
    if (e + 8 <= count) store8(o + e, v);
    else if (e < count) store8_n(o + e, v, count - e);
  }
}

__global__ __launch_bounds__(256) void grad_scale_kernel(ScaleTable tab) {
  const uint32_t wg = blockIdx.x;
  const int t = tensor_of(tab.first, wg);
  const float f = ld_uniform(tab.factor);
  if (f == 1.f && tab.grad[t] == tab.out[t]) return;  // the product would be the value itself
  const int64_t e0 = (int64_t)(wg - tab.first[t]) * SCALE_CHUNK, all = tab.n[t];
  if (all < 0)
    scale_chunk(static_cast<const uint16_t*>(tab.grad[t]) + e0, static_cast<uint16_t*>(tab.out[t]) + e0, -all - e0, f);
  else
    scale_chunk(static_cast<const float*>(tab.grad[t]) + e0, static_cast<float*>(tab.out[t]) + e0, all - e0, f);
}

}  // namespace

hipError_t launch_grad_norm(const GradTable& t, uint32_t groups, hipStream_t s) {
  grad_norm_kernel<<<groups, 256, 0, s>>>(t);
  return hipGetLastError();
}

hipError_t launch_grad_norm_sum(const double* part, int64_t n, double max_norm, float* norm,
                                float* factor, hipStream_t s) {
  grad_norm_sum_kernel<<<1, 1024, 0, s>>>(part, n, max_norm, norm, factor);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const ScaleTable& t, uint32_t groups, hipStream_t s) {
  grad_scale_kernel<<<groups, 256, 0, s>>>(t);
  return hipGetLastError();
}

}  // namespace sffn
