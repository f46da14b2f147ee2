// Rounding of tokens to 4 bits (the format of the weights: e2m1 codes, one power of two per 32 columns),
// in the layout that the products of mx4_matmul read.
//
// A lane takes 8 consecutive values, so that a wave reads 512 columns of a row in one piece; the four
// lanes of a group find its absolute maximum and convert.  A workgroup collects 16
// rows of four blocks of 128 columns in LDS, whose codes and scales it writes in one piece each.
#include "ops_common.hpp"

namespace sffn {
namespace {

constexpr int SPAN = 4;  // blocks of 128 columns of a workgroup

template <typename T>
__global__ __launch_bounds__(256) void mx4_tokens_kernel(const T* x, int64_t stride, int32_t rows,
                                                         int32_t K, int32_t kb, uint8_t* tokens) {
  __shared__ u32x4 codes[SPAN * 64];  // as they are read: written by words, and the scales by bytes
  __shared__ uint32_t scales[SPAN * 16];
  const int lane = (int)(threadIdx.x & 63), wave = uniform((int)(threadIdx.x >> 6));
  const int spans = (kb + SPAN - 1) / SPAN;
  const int64_t tb = blockIdx.x / (uint32_t)spans, t0 = tb * 16;
  const int kb0 = (int)(blockIdx.x % (uint32_t)spans) * SPAN;
  const int64_t k0 = (int64_t)kb0 * 128 + lane * 8;
  const int n = K - k0 >= 8 ? 8 : K > k0 ? (int)(K - k0) : 0;
  Raw8<T> raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + i * 4 + wave;
    raw[i].zero();
    if (t < rows) {
      const T* p = x + t * stride + k0;
      if (n == 8) raw[i].load(p);
      else if (n > 0) raw[i].load_n(p, n);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 4 + wave;
    float big = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) big = max_abs(big, raw[i].get(j));
    big = max_abs(big, dpp<0xB1>(big));
    big = max_abs(big, dpp<0x4E>(big));
    const uint32_t scale = mx4_scale(big);
    const int b = lane >> 4, q = (lane >> 2) & 3;
    const int j = lane & 3, word = j == 0 || j == 3 ? j : 3 - j;  // in the order 0, 2, 1, 3
    reinterpret_cast<uint32_t*>(codes)[b * 256 + (q * 16 + r) * 4 + word] = mx4_codes8(raw[i], scale);
    // a group past the last column has the scale 1, as in the weights
    if ((lane & 3) == 0)
      reinterpret_cast<uint8_t*>(scales)[b * 64 + r * 4 + q] = (uint8_t)(k0 < K ? scale : 127u);
  }
  __syncthreads();
  const int b = (int)(threadIdx.x >> 6);
  uint8_t* out = tokens + (tb * kb + kb0) * MX4_BLOCK;
  if (kb0 + b < kb)
    *reinterpret_cast<u32x4*>(out + b * MX4_BLOCK + lane * 16) = codes[threadIdx.x];
  if (threadIdx.x < SPAN * 16 && kb0 + (int)(threadIdx.x >> 4) < kb)
    *reinterpret_cast<uint32_t*>(out + (threadIdx.x >> 4) * MX4_BLOCK + 1024 + (threadIdx.x & 15) * 4) =
        scales[threadIdx.x];
}

}  // namespace

hipError_t launch_mx4_tokens(bool bf16, const void* x, int64_t stride, int32_t T, int32_t K,
                             void* tokens, hipStream_t s) {
  const int kb = (int)(((int64_t)K + 127) / 128);
  const dim3 grid((unsigned)((int64_t)((kb + SPAN - 1) / SPAN) * ((T + 15) / 16)));  // below 2^24
  uint8_t* out = static_cast<uint8_t*>(tokens);
  if (bf16)
    mx4_tokens_kernel<uint16_t><<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(x), stride, T, K, kb, out);
  else
    mx4_tokens_kernel<float><<<grid, 256, 0, s>>>(static_cast<const float*>(x), stride, T, K, kb, out);
  return hipGetLastError();
}

}  // namespace sffn
