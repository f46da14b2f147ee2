// Device helpers and launchers of the operators around the layer (include/ffn_ops.h).
#pragma once

#include <type_traits>

#include "../../include/ffn_ops.h"
#include "layer_norm_shape.hpp"
#include "sffn_common.hpp"

namespace sffn {

constexpr float E4M3_MAX = 448.f;
constexpr float E4M3_TINY = 0x1p-9f;   // smallest positive e4m3 value
constexpr float SCALE_MIN = 0x1p-126f;  // keeps the division by a scale defined for zero rows

#if defined(__HIPCC__)
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// The same types at an element's alignment: global memory takes vector accesses at any
// address, so rows that start off a 16-byte boundary need no path of their own.
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// Eight consecutive elements as loaded (bf16: 16 bytes, fp32: 32 bytes).
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  u32x4 r;
  __device__ __forceinline__ void zero() { r = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const uint16_t* p) {
    r = *reinterpret_cast<const u32x4_a2*>(p);
  }
  __device__ __forceinline__ void load_n(const uint16_t* p, int n) {  // n < 8 elements
    uint16_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : (uint16_t)0;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (uint32_t)e[2 * i] | ((uint32_t)e[2 * i + 1] << 16);
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = r[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
};
template <>
struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void zero() { a = b = f32x4{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4_a4*>(p);
    b = *reinterpret_cast<const f32x4_a4*>(p + 4);
  }
  __device__ __forceinline__ void load_n(const float* p, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = i < n ? p[i] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = i + 4 < n ? p[i + 4] : 0.f;
  }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
};

__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = (uint32_t)f32_to_bf16(v[2 * i]) | ((uint32_t)f32_to_bf16(v[2 * i + 1]) << 16);
  *reinterpret_cast<u32x4_a2*>(p) = r;
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  *reinterpret_cast<f32x4_a4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4_a4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = f32_to_bf16(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
template <typename T>
__device__ __forceinline__ void store8_n(T* p, const float* v, int n) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) store1(p + i, v[i]);
}

// One vector access at any address of its elements' alignment; NT: past the caches, at the
// vector's own alignment.
template <bool NT, typename V>
__device__ __forceinline__ V load_v(const void* p) {
  if constexpr (NT) return __builtin_nontemporal_load(static_cast<const V*>(p));
  V v;
  __builtin_memcpy(&v, p, sizeof(v));
  return v;
}
template <bool NT, typename V>
__device__ __forceinline__ void store_v(void* p, V v) {
  if constexpr (NT) __builtin_nontemporal_store(v, static_cast<V*>(p));
  else __builtin_memcpy(p, &v, sizeof(v));
}
// Four consecutive elements, of which the first n exist.
template <bool NT>
__device__ __forceinline__ void load4(const float* p, int n, float* o) {
  if (n >= 4) {
    const f32x4 v = load_v<NT, f32x4>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = i < n ? p[i] : 0.f;
  }
}
template <bool NT>
__device__ __forceinline__ void load4(const uint16_t* p, int n, float* o) {
  u32x2 v = u32x2{0, 0};
  if (n >= 4) {
    v = load_v<NT, u32x2>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = __uint_as_float((i & 1) ? (v[i >> 1] & 0xffff0000u) : (v[i >> 1] << 16));
}

// Four / eight values to e4m3, to nearest-even.  |v| <= 448 up to rounding, or NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}
__device__ __forceinline__ u32x2 e4m3x8(const float* v) {
  return u32x2{e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7])};
}
__device__ __forceinline__ void store_e4m3x8(uint8_t* p, const float* v, int n) {
  const u32x2 q = e4m3x8(v);
  if (n >= 8) {
    *reinterpret_cast<u32x2_a1*>(p) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
      0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}
struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// max that keeps a NaN, as an absolute maximum over data has to
struct MaxNan {
  __device__ __forceinline__ float operator()(float a, float b) const {
    return (b > a || b != b) ? b : a;
  }
};
// The same of v's absolute value and a, which is one or 0: ordered as integers, NaN last.
__device__ __forceinline__ float max_abs(float a, float v) {
  const uint32_t x = __float_as_uint(a), y = __float_as_uint(v) & 0x7fffffffu;
  return __uint_as_float(x > y ? x : y);
}
// Reduction over 16 lanes, a half wave (32) or a wave (64); every lane gets the result.
// quad_perm, half-row and row mirrors combine the 16 lanes of a row, the lane swaps the rows
// (rows_reduce: those alone).
template <int LANES = 64, typename Op>
__device__ __forceinline__ float rows_reduce(float v, Op op) {
  if constexpr (LANES >= 32) {
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = op(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  if constexpr (LANES >= 64) {
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = op(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  return v;
}
template <int LANES, typename Op>
__device__ __forceinline__ float lane_reduce(float v, Op op) {
  v = op(v, dpp<0xB1>(v));   // quad_perm [1, 0, 3, 2]
  v = op(v, dpp<0x4E>(v));   // quad_perm [2, 3, 0, 1]
  v = op(v, dpp<0x141>(v));  // half-row mirror
  v = op(v, dpp<0x140>(v));  // row mirror
  return rows_reduce<LANES>(v, op);
}
// The same over the L lanes of a row (16, 32, 64, or whole waves of one workgroup); `red` holds
// L / 64 floats of LDS that nothing else uses before the next barrier.
template <int L, typename Op>
__device__ __forceinline__ float row_reduce(float v, Op op, float* red) {
  v = lane_reduce<(L < 64 ? L : 64)>(v, op);
  if constexpr (L > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < L / 64; ++i) v = op(v, red[i]);
  }
  return v;
}
// A row's reduction for any number of waves: L lanes (16, 32, 64), or with L = 0 all waves of the
// workgroup (at most 16), whose values 16 lanes of each wave take up again.  `red` holds 16 floats
// of LDS that nothing else uses before the next barrier; 0 is op's neutral element.
template <int L, typename Op>
__device__ __forceinline__ float group_reduce(float v, Op op, float* red) {
  v = lane_reduce<(L == 0 ? 64 : L)>(v, op);
  if constexpr (L == 0) {
    const int i = (int)(threadIdx.x & 15);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lane_reduce<16>(i < (int)(blockDim.x >> 6) ? red[i] : 0.f, op);
  }
  return v;
}
// Sums of two values over `waves` waves, of which `first` is the first, with one barrier of the
// workgroup.
__device__ __forceinline__ void group_sum2(float& a, float& b, float* red_a, float* red_b,
                                           int waves, int first) {
  a = lane_reduce<64>(a, Add());
  b = lane_reduce<64>(b, Add());
  const int i = (int)(threadIdx.x & 15);
  if ((threadIdx.x & 63) == 0) {
    red_a[threadIdx.x >> 6] = a;
    red_b[threadIdx.x >> 6] = b;
  }
  __syncthreads();
  a = lane_reduce<16>(i < waves ? red_a[first + i] : 0.f, Add());
  b = lane_reduce<16>(i < waves ? red_b[first + i] : 0.f, Add());
}
// A group of 32 values in 4 bits.  Its scale from the largest absolute value: the exponent less 2
// (e2m1's largest) as it is stored, at least 0; 255 with an infinity or a NaN among the values.
__device__ __forceinline__ uint32_t mx4_scale(float big) {
  const uint32_t bits = __float_as_uint(big);
  const int e = (int)(bits >> 23) - 2;
  return bits >= 0x7f800000u ? 255u : (uint32_t)(e < 0 ? 0 : e);
}
// Eight values at that scale as codes, to nearest-even, saturating (the instruction reads the scale's
// exponent field alone; compared with the thresholds of mx4_quantize on 4 million values at every
// scale, it differs in the sign of zeros only).  A group with the scale 255 has the codes 0.
template <typename V>
__device__ __forceinline__ uint32_t mx4_codes8(const V& v, uint32_t scale) {
  const float s = __uint_as_float(scale << 23);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v.get(0), v.get(1), s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v.get(2), v.get(3), s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v.get(4), v.get(5), s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v.get(6), v.get(7), s, 3);
  return scale == 255u ? 0u : c;
}
// Quotients of values up to 448 s by a positive scale s, bit for bit the divide's: the product with
// the rounded reciprocal is a few roundings off, and one fma with its remainder corrects it
// (P. Markstein, 1990; compared with the divide on 3.2e9 pairs, half of them next to the middle
// between two e4m3 values).  A scale so small that the remainder would fall below the smallest fp32
// values, or one that is not finite, takes the divide itself.  (With divides everywhere the 8-bit
// norm of 16384 x 2304 took 55 us a call instead of 48, AdamW with 8-bit states over 34 million
// values 114 instead of 109.)
struct Quotients {
  float s, inv;
  bool usual;  // for every lane of the wave
  __device__ __forceinline__ explicit Quotients(float scale)
      : s(scale), inv(1.f / scale), usual(ballot64(!(scale >= 0x1p-60f && scale < INFINITY)) == 0) {}
  template <int N>
  __device__ __forceinline__ void operator()(float (&x)[N]) const {
    if (usual) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float q = x[i] * inv;
        x[i] = fmaf(fmaf(-q, s, x[i]), inv, q);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] /= s;
    }
  }
};
// 1 / sqrt(ms) to fp32 accuracy: the divide and the root are correctly rounded.
__device__ __forceinline__ float inv_rms(float ms) { return 1.f / sqrtf(ms); }
#endif

// ---------------------------------------------------------------- launchers
// Lanes that share a row of d elements in the norm kernels; a lane keeps 8, 16, or (16 waves)
// up to 32 of them.  Few elements a lane leave registers for many rows in flight: 8192 x 4096
// takes 46 us with 4 waves a row and 51 with one (gradient 54 and 69), 16384 x 1024 27 and 25.
// The gradient, with more to keep, takes 8 waves above 2048 (16384 x 2304: 59.8 us, 61.5 with 4;
// the norm itself 60 and 49 with 8 bits out).
inline int norm_lanes(int32_t d, bool grad) {
  return d <= 128    ? 16
         : d <= 256  ? 32
         : d <= 1024 ? 64
         : d <= 2048 ? 256
         : d <= 4096 ? (grad ? 512 : 256)
                     : 1024;
}
struct NormArgs {
  const void* x;
  int64_t x_stride;
  const void* residual;
  int64_t residual_stride;
  const void* gain;
  float eps;
  int64_t rows;
  int32_t d;
  void* y;     // dtype, or e4m3 bytes
  float* stat;  // rstd, or the 8-bit scales
  void* h;
};
// Calls f(lanes, vectors of 8 a lane) with both as integral constants, for a row of d elements.
template <bool GRAD, typename F>
hipError_t norm_shape(int32_t d, F&& f) {
  const int L = norm_lanes(d, GRAD), nv = (d + 8 * L - 1) / (8 * L);
#define SFFN_SHAPE(l, n) \
  if (L == l && nv == n) return f(std::integral_constant<int, l>(), std::integral_constant<int, n>())
  SFFN_SHAPE(16, 1);
  SFFN_SHAPE(32, 1);
  SFFN_SHAPE(64, 1);
  SFFN_SHAPE(64, 2);
  SFFN_SHAPE(256, 1);
  if constexpr (GRAD) {
    SFFN_SHAPE(512, 1);
  } else {
    SFFN_SHAPE(256, 2);
  }
  SFFN_SHAPE(1024, 1);
  SFFN_SHAPE(1024, 2);
  SFFN_SHAPE(1024, 3);
  SFFN_SHAPE(1024, 4);
#undef SFFN_SHAPE
  return hipErrorInvalidValue;
}
hipError_t launch_rms_norm(bool bf16, bool gain_f32, bool fp8, const NormArgs& a, hipStream_t s);

struct NormGradArgs {
  const void* dy;
  int64_t dy_stride;
  const void* h;
  int64_t h_stride;
  const void* gain;
  const float* rstd;
  const void* dres;
  int64_t dres_stride;
  int64_t rows;
  int32_t d;
  void* dx;
  float* dgain;
  float* part;  // [norm_grad_groups(rows, d), d] partial sums of dgain, or null
};
// Partial rows of dgain, whose sum takes a second kernel; 0 where the first one's further
// workgroups sum dgain themselves.
int norm_grad_groups(int64_t rows, int32_t d);
hipError_t launch_rms_norm_grad(bool bf16, bool gain_f32, const NormGradArgs& a, hipStream_t s);
// dgain[c] = sum of the n partial rows (0 with none)
hipError_t launch_rms_norm_grad_sum(const float* part, int n, int32_t d, float* dgain,
                                    hipStream_t s);

// Calls f(lanes, vectors) with both as integral constants; MANY: the lanes of more than one vector.
template <int MANY, typename F>
hipError_t with_row_shape(const RowShape& r, F&& f) {
#define SFFN_SHAPE(l, n) \
  if (r.lanes == l && r.nv == n) return f(std::integral_constant<int, l>(), std::integral_constant<int, n>())
  SFFN_SHAPE(16, 1);
  SFFN_SHAPE(32, 1);
  SFFN_SHAPE(64, 1);
  SFFN_SHAPE(0, 1);
  SFFN_SHAPE(MANY, 2);
  SFFN_SHAPE(MANY, 3);
  SFFN_SHAPE(MANY, 4);
#undef SFFN_SHAPE
  return hipErrorInvalidValue;
}

struct LayerNormArgs {
  const void* x;
  int64_t x_stride;
  const void* residual;
  int64_t residual_stride;
  const void* gain;
  const void* bias;
  float eps;
  int64_t rows;
  int32_t d;
  void* y;      // dtype, or e4m3 bytes
  float* mean;
  float* stat;  // rstd, or the 8-bit scales
  void* h;
};
hipError_t launch_layer_norm(bool bf16, bool gain_f32, bool fp8, const LayerNormArgs& a,
                             hipStream_t s);

struct LayerNormGradArgs {
  const void* dy;
  int64_t dy_stride;
  const void* h;
  int64_t h_stride;
  const void* gain;
  const float* mean;
  const float* rstd;
  const void* dres;
  int64_t dres_stride;
  int64_t rows;
  int32_t d;
  void* dx;
  float* dgain;
  float* dbias;
  float* part;    // [layer_norm_grad_parts(rows, d), 2, d] partial sums of dgain and dbias, or null
  int sum_parts;  // the launcher's
};
// Partial rows of dgain and dbias, whose sum takes a second kernel; 0 where the first one writes the
// sums themselves.
int layer_norm_grad_parts(int64_t rows, int32_t d);
hipError_t launch_layer_norm_grad(bool bf16, bool gain_f32, const LayerNormGradArgs& a,
                                  hipStream_t s);
// dgain[c] and dbias[c] = sums of the n partial rows (0 with none); either may be null
hipError_t launch_layer_norm_grad_sum(const float* part, int n, int32_t d, float* dgain,
                                      float* dbias, hipStream_t s);

// The tiled 4-bit layout: for every 16 rows and 128 columns a block of MX4_BLOCK bytes: 1 KB of
// codes (lane l of a wave: row l % 16, word j of its four: columns 32 j + 8 (l / 16) and the
// seven after), then 64 scales (row by row, the four groups of 32 columns).  Blocks run over the
// columns first.
constexpr int MX4_BLOCK = 1024 + 64;
struct Mx4Dims {
  int32_t N, K;
  int32_t nb, kb;  // ceil(N / 16), ceil(K / 128)
  size_t bytes() const { return (size_t)nb * kb * MX4_BLOCK; }
};
inline Mx4Dims mx4_dims(int32_t N, int32_t K) {
  return Mx4Dims{N, K, (int32_t)(((int64_t)N + 15) / 16), (int32_t)(((int64_t)K + 127) / 128)};
}
hipError_t launch_mx4_quantize(bool bf16, const void* W, int64_t stride, int32_t N, int32_t K,
                               uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_mx4_tile(const uint8_t* codes, const uint8_t* scales, const Mx4Dims& d,
                           void* tiled, hipStream_t s);
struct Mx4Args {
  const void* tiled;
  Mx4Dims d;
  int32_t x_dtype;  // SFFN_F32, SFFN_BF16, SFFN_E4M3
  const void* x;
  int64_t x_stride;
  const float* x_scale;
  int32_t T;
  const float* bias;
  bool relu;
  bool y_bf16;
  void* y;
};
hipError_t launch_mx4_linear(const Mx4Args& a, hipStream_t s);

// Tokens in 4 bits: blocks of 16 tokens x 128 columns, the columns first, of MX4_BLOCK bytes: 1 KB of
// codes (lane l of a wave: token l % 16, columns 32 (l / 16) to 31 after it, in four words of 8 in the
// order 0, 2, 1, 3), then 64 scales (token by token, the four groups of 32 columns).
hipError_t launch_mx4_tokens(bool bf16, const void* x, int64_t stride, int32_t T, int32_t K,
                             void* tokens, hipStream_t s);
struct Mx4MatmulArgs {
  const void* tiled;
  Mx4Dims d;
  const void* tokens;  // in 4 bits, or of x_dtype (at most MX4_ROUND_T tokens, x_stride elements apart)
  int32_t x_dtype;     // SFFN_F32, SFFN_BF16, or MX4_TOKENS
  int64_t x_stride;
  int32_t T;
  const float* bias;
  bool relu;
  bool y_bf16;
  void* y;
  bool past_caches;  // the launcher's: bf16 results, and fp32 ones that would fill the caches, go past them
};
constexpr int32_t MX4_TOKENS = -1;
constexpr int32_t MX4_ROUND_T = 16;
hipError_t launch_mx4_matmul(const Mx4MatmulArgs& a, hipStream_t s);

// Gradients of one launch of the norm or of the scaling; the table travels as kernel arguments.
// n is negated for bf16.
constexpr int GRAD_TENSORS = 128;
struct GradTable {
  const void* grad[GRAD_TENSORS];
  int64_t n[GRAD_TENSORS];
  uint32_t first[GRAD_TENSORS];  // first workgroup of each tensor; 2^32 - 1 past the last one
  int64_t chunk;                 // elements of a workgroup, a multiple of 8
  double* part;                  // [workgroups] sums of squares
};
static_assert(sizeof(GradTable) <= 4096 - 256, "kernel arguments");
hipError_t launch_grad_norm(const GradTable& t, uint32_t groups, hipStream_t s);
// norm and factor (may be null) of the n partial sums
hipError_t launch_grad_norm_sum(const double* part, int64_t n, double max_norm, float* norm,
                                float* factor, hipStream_t s);
constexpr int SCALE_TENSORS = 96;
constexpr int SCALE_CHUNK = 8192;  // elements of one workgroup
struct ScaleTable {
  const void* grad[SCALE_TENSORS];
  void* out[SCALE_TENSORS];
  int64_t n[SCALE_TENSORS];  // negated for bf16
  uint32_t first[SCALE_TENSORS];
  const float* factor;
};
static_assert(sizeof(ScaleTable) <= 4096 - 256, "kernel arguments");
hipError_t launch_grad_scale(const ScaleTable& t, uint32_t groups, hipStream_t s);

// Tensors of one AdamW launch; the table travels as kernel arguments (at most 4 KB of them).
constexpr int ADAMW_TENSORS = 48;
struct AdamwTable {
  sffn_adamw_tensor_t t[ADAMW_TENSORS];
  uint32_t first[ADAMW_TENSORS];  // first workgroup of each tensor; 2^32 - 1 past the last one
  float lr_decay;   // lr * weight_decay
  float beta1, one_minus_beta1, beta2, one_minus_beta2;
  float step_size;  // lr / (1 - beta1^step)
  float inv_root_correction;  // 1 / sqrt(1 - beta2^step)
  float eps;
  const float* grad_scale;
};
static_assert(sizeof(AdamwTable) <= 4096 - 256, "kernel arguments");
constexpr int ADAMW_CHUNK = 2048;  // elements of one workgroup
hipError_t launch_adamw(bool param_bf16, bool grad_bf16, bool master, int state_bits,
                        const AdamwTable& t, uint32_t groups, hipStream_t s);

}  // namespace sffn
