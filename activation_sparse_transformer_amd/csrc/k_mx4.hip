// Products of a few tokens with 4-bit weights: y = act(x W^T * x_scale + bias),
// W[n, k] = e2m1(code) 2^(s - 127) with one s per 32 columns.
//
// One wave holds 16 x 128 weights in a 16-byte load a lane (the tiled layout: 1 KB contiguous),
// expands them to bf16 with the packed conversion that applies the scale (exact: a bf16 holds
// e2m1 times a power of two) and multiplies on the matrix cores: A = 16 weight rows, B = up to
// 16 tokens, v_mfma_f32_16x16x32_bf16.  Which k a lane's eight elements stand for is the same
// permutation for both operands, so a lane's 32 consecutive columns make four such products.
// Token types: bf16 as it is; e4m3 widened to bf16 (exact); fp32 as the sum of three bf16
// (truncations: 8 + 8 + 8 bits, exact), three products.  The waves of a workgroup split k and
// add their fp32 sums in LDS in wave order.
#include "ops_common.hpp"

namespace sffn {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// Eight e2m1 codes times 2^(s - 127) (the scale's exponent field is read as it is).
__device__ __forceinline__ bf16x8 expand8(uint32_t codes, float scale) {
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  return as_bf16x8(r);
}

// Eight consecutive columns of one token, and their operands for the bf16 products.
template <int XT>
struct Tok8;
template <>
struct Tok8<SFFN_BF16> {
  static constexpr int TERMS = 1;
  typedef uint16_t elem;
  u32x4 r;
  __device__ __forceinline__ void zero() { r = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const elem* p) { r = *reinterpret_cast<const u32x4_a2*>(p); }
  __device__ __forceinline__ void load_n(const elem* p, int n) {  // n < 8, after zero()
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) r[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
  }
  __device__ __forceinline__ void terms(bf16x8* t) const { t[0] = as_bf16x8(r); }
};
template <>
struct Tok8<SFFN_E4M3> {
  static constexpr int TERMS = 1;
  typedef uint8_t elem;
  u32x2 r;
  __device__ __forceinline__ void zero() { r = u32x2{0, 0}; }
  __device__ __forceinline__ void load(const elem* p) { r = *reinterpret_cast<const u32x2_a1*>(p); }
  __device__ __forceinline__ void load_n(const elem* p, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) r[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  }
  __device__ __forceinline__ void terms(bf16x8* t) const {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r[i], 1.f, false));
      o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r[i], 1.f, true));
    }
    t[0] = as_bf16x8(o);
  }
};
template <>
struct Tok8<SFFN_F32> {
  static constexpr int TERMS = 3;
  typedef float elem;
  f32x4 r[2];
  __device__ __forceinline__ void zero() { r[0] = r[1] = f32x4{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ void load(const elem* p) {
    r[0] = *reinterpret_cast<const f32x4_a4*>(p);
    r[1] = *reinterpret_cast<const f32x4_a4*>(p + 4);
  }
  __device__ __forceinline__ void load_n(const elem* p, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) r[j >> 2][j & 3] = p[j];
  }
  // x = hi + mid + lo, each the upper 16 bits of what is left; the rest of an infinity is 0
  // (its own difference would be NaN)
  __device__ __forceinline__ void terms(bf16x8* t) const {
    u32x4 o[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t b[2][3];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = r[i >> 1][(i & 1) * 2 + e];
        b[e][0] = __float_as_uint(x);
        const float hi = __uint_as_float(b[e][0] & 0xffff0000u);
        const float m = x == hi ? 0.f : x - hi;
        b[e][1] = __float_as_uint(m);
        const float l = m - __uint_as_float(b[e][1] & 0xffff0000u);
        b[e][2] = __float_as_uint(l);
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) o[k][i] = __builtin_amdgcn_perm(b[1][k], b[0][k], 0x07060302u);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) t[k] = as_bf16x8(o[k]);
  }
};

// Scale, bias and activation of four rows n .. n + 3 of one token, and their store.
__device__ __forceinline__ void mx4_store(const Mx4Args& a, f32x4 s, int tok, int n) {
  const int N = a.d.N;
  if (tok >= a.T || n >= N) return;
  const float xsc = a.x_scale ? a.x_scale[tok] : 1.f;
  float o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float v = s[e] * xsc;
    if (a.bias && n + e < N) v += a.bias[n + e];
    o[e] = a.relu && v < 0.f ? 0.f : v;
  }
  const int64_t at = (int64_t)tok * N + n;
  if (a.y_bf16) {
    uint16_t* y = static_cast<uint16_t*>(a.y) + at;
    if (n + 4 <= N) {
      typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
      *reinterpret_cast<u32x2_a2*>(y) =
          u32x2{(uint32_t)f32_to_bf16(o[0]) | ((uint32_t)f32_to_bf16(o[1]) << 16),
                (uint32_t)f32_to_bf16(o[2]) | ((uint32_t)f32_to_bf16(o[3]) << 16)};
    } else {
      for (int e = 0; e < N - n; ++e) y[e] = f32_to_bf16(o[e]);
    }
  } else {
    float* y = static_cast<float*>(a.y) + at;
    if (n + 4 <= N) {
      *reinterpret_cast<f32x4_a4*>(y) = f32x4{o[0], o[1], o[2], o[3]};
    } else {
      for (int e = 0; e < N - n; ++e) y[e] = o[e];
    }
  }
}

constexpr int MX4_WAVES = 8;

// RB blocks of 16 weight rows and TT of 16 tokens a wave; KS of a workgroup's waves split k, the
// others take further rows.
template <int XT, int TT, int RB, int KS>
__global__ __launch_bounds__(MX4_WAVES * 64) void mx4_linear_kernel(Mx4Args a) {
  typedef Tok8<XT> X;
  typedef typename X::elem E;
  __shared__ f32x4 part[MX4_WAVES][RB][TT][64];
  const int lane = (int)(threadIdx.x & 63), wave = uniform((int)(threadIdx.x >> 6));
  const int q = lane >> 4, r = lane & 15;
  const int wg0 = (int)blockIdx.x * (RB * MX4_WAVES / KS);
  const int rb0 = wg0 + wave / KS * RB, t0 = (int)blockIdx.y * (TT * 16);
  const int KB = a.d.kb, K = a.d.K;
  const uint8_t* wb = static_cast<const uint8_t*>(a.tiled);
  const E* x = static_cast<const E*>(a.x);

  f32x4 acc[RB][TT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[b][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int kb = wave % KS; kb < KB; kb += KS) {
    u32x4 c[RB];
    uint32_t sc[RB];
    X xs[TT][4];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      c[b] = u32x4{0, 0, 0, 0};
      sc[b] = 127;
      if (rb0 + b < a.d.nb) {
        const uint8_t* p = wb + ((size_t)(rb0 + b) * KB + kb) * MX4_BLOCK;
        c[b] = *reinterpret_cast<const u32x4*>(p + lane * 16);
        sc[b] = p[1024 + lane];
      }
    }
    const int k0 = (kb * 4 + q) * 32;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int tok = t0 + t * 16 + r;
#pragma unroll
      for (int j = 0; j < 4; ++j) xs[t][j].zero();
      if (tok < a.T && k0 + 32 <= K) {
        const E* p = x + (int64_t)tok * a.x_stride + k0;
#pragma unroll
        for (int j = 0; j < 4; ++j) xs[t][j].load(p + 8 * j);
      }
    }
    if (K & 31) {  // the last, partial group of 32 columns
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const int tok = t0 + t * 16 + r;
        if (tok < a.T && k0 < K && k0 + 32 > K) {
          const E* p = x + (int64_t)tok * a.x_stride + k0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int n = K - k0 - 8 * j;
            if (n >= 8) xs[t][j].load(p + 8 * j);
            else if (n > 0) xs[t][j].load_n(p + 8 * j, n);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x8 w[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b) w[b] = expand8(c[b][j], __uint_as_float(sc[b] << 23));
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        bf16x8 xt[X::TERMS];
        xs[t][j].terms(xt);
#pragma unroll
        for (int k = X::TERMS - 1; k >= 0; --k)
#pragma unroll
          for (int b = 0; b < RB; ++b)
            acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[b], xt[k], acc[b][t], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < TT; ++t) part[wave][b][t][lane] = acc[b][t];
  __syncthreads();

  constexpr int ITEMS = MX4_WAVES / KS * RB * TT * 64;
  for (int i = (int)threadIdx.x; i < ITEMS; i += MX4_WAVES * 64) {
    const int l = i & 63, t = (i >> 6) % TT, b = (i >> 6) / TT % RB, g = (i >> 6) / (TT * RB);
    f32x4 s = part[g * KS][b][t][l];
#pragma unroll
    for (int w = 1; w < KS; ++w) s += part[g * KS + w][b][t][l];
    mx4_store(a, s, t0 + t * 16 + (l & 15), (wg0 + g * RB + b) * 16 + (l >> 4) * 4);
  }
}

template <int XT, int TT, int RB, int KS>
hipError_t launch_ks(const Mx4Args& a, hipStream_t s) {
  constexpr int ROWS = RB * MX4_WAVES / KS;
  const dim3 grid((unsigned)((a.d.nb + ROWS - 1) / ROWS), (unsigned)((a.T + TT * 16 - 1) / (TT * 16)));
  mx4_linear_kernel<XT, TT, RB, KS><<<grid, MX4_WAVES * 64, 0, s>>>(a);
  return hipGetLastError();
}

template <int XT, int TT, int RB>
hipError_t launch_rb(const Mx4Args& a, hipStream_t s) {
  // Waves beyond the blocks of columns would idle: they take rows instead, while that leaves
  // two workgroups a CU (65536 x 256, one token: 3.9 against 5.3 us).
  int ks = MX4_WAVES;
  while (ks > 2 && ks > a.d.kb && (int64_t)a.d.nb * ks / (2 * RB * MX4_WAVES) >= 256) ks /= 2;
  if (ks == 8) return launch_ks<XT, TT, RB, 8>(a, s);
  if (ks == 4) return launch_ks<XT, TT, RB, 4>(a, s);
  return launch_ks<XT, TT, RB, 2>(a, s);
}

// A wave's work on a block of columns is that on its tokens (loads, conversions: about 1.5 TT
// times what a block of weights costs, three times that for fp32) and on RB blocks of weights;
// RB is the one with the least rounds of workgroups over the 256 CUs times that work.  Measured,
// one token, K 2048, RB 1 / 2 / 4: N 2048 3.2 / 3.4 / 4.3 us, 8192 4.0 / 3.6 / 4.4; 12 tokens,
// N 9216 - / 6.3 / 5.1, 65536 28.7 / 18.8 / 15.3.
template <int XT, int TT>
hipError_t launch_tt(const Mx4Args& a, hipStream_t s) {
  const int64_t blocks = (int64_t)a.d.nb * ((a.T + TT * 16 - 1) / (TT * 16));
  int best = 1;
  double least = 0;
  for (int rb = 1; rb <= 4; rb *= 2) {
    const double cost = (double)((blocks + rb * 256 - 1) / (rb * 256)) *
                        (1.5 * Tok8<XT>::TERMS * TT + rb);
    if (rb == 1 || cost < least) {
      best = rb;
      least = cost;
    }
  }
  if (best == 1) return launch_rb<XT, TT, 1>(a, s);
  if (best == 2) return launch_rb<XT, TT, 2>(a, s);
  return launch_rb<XT, TT, 4>(a, s);
}

template <int XT>
hipError_t launch_x(const Mx4Args& a, hipStream_t s) {
  return a.T <= 16 ? launch_tt<XT, 1>(a, s) : launch_tt<XT, 2>(a, s);
}

// ------------------------------------------------------------------ weights

// One thread a group of 32: exponent of the largest value less 2 (e2m1's largest exponent),
// values to nearest-even at that scale.
template <typename T>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const T* W, int64_t stride, int32_t N,
                                                           int32_t K, int32_t G, uint8_t* codes,
                                                           uint8_t* scales) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)N * G) return;
  const int64_t n = i / G;
  const int g = (int)(i % G);
  const int k0 = g * 32, len = K - k0 < 32 ? K - k0 : 32;
  const T* w = W + n * stride + k0;
  float v[32], big = 0.f;
  Raw8<T> raw[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    raw[j].zero();
    if (8 * j + 8 <= len) raw[j].load(w + 8 * j);
    else if (8 * j < len) raw[j].load_n(w + 8 * j, len - 8 * j);
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    v[j] = raw[j >> 3].get(j & 7);
    big = MaxNan()(big, fabsf(v[j]));
  }
  const uint32_t bits = __float_as_uint(big);
  int e = (int)(bits >> 23) - 127;             // floor(log2(big)) of a normal number
  if (bits < 0x00800000u) e = -127;            // zero or subnormal: at the smallest scale anyway
  const bool bad = bits >= 0x7f800000u;        // infinity or NaN
  int sexp = e - 2;
  if (sexp < -127) sexp = -127;
  scales[i] = bad ? 255 : (uint8_t)(sexp + 127);
  u32x4 out = u32x4{0, 0, 0, 0};
  if (!bad) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float a = ldexpf(fabsf(v[j]), -sexp);
      // midpoints between neighbours; a tie goes to the code that is even
      const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) +
                         (a >= 3.5f) + (a > 5.f);
      out[j >> 3] |= (c | (v[j] < 0.f ? 8u : 0u)) << (4 * (j & 7));
    }
  }
  *reinterpret_cast<u32x4_a1*>(codes + i * 16) = out;
}

// One thread for 16 bytes of codes and one scale of the tiled layout.
__global__ __launch_bounds__(256) void mx4_tile_kernel(const uint8_t* codes, const uint8_t* scales,
                                                       Mx4Dims d, uint8_t* tiled) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t blk = i >> 6;
  if (blk >= (int64_t)d.nb * d.kb) return;
  const int lane = (int)(i & 63);
  const int64_t n = blk / d.kb * 16 + (lane & 15);
  const int g = (int)(blk % d.kb) * 4 + (lane >> 4), G = (d.K + 31) / 32;
  u32x4 c = u32x4{0, 0, 0, 0};
  uint8_t sc = 127;
  if (n < d.N && g < G) {
    c = *reinterpret_cast<const u32x4_a1*>(codes + (n * G + g) * 16);
    sc = scales[n * G + g];
    const int len = d.K - g * 32;
    if (len < 32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int left = len - 8 * j;
        if (left <= 0) c[j] = 0;
        else if (left < 8) c[j] &= (1u << (4 * left)) - 1;
      }
    }
  }
  uint8_t* p = tiled + blk * MX4_BLOCK;
  *reinterpret_cast<u32x4*>(p + lane * 16) = c;
  p[1024 + lane] = sc;
}

}  // namespace

hipError_t launch_mx4_linear(const Mx4Args& a, hipStream_t s) {
  switch (a.x_dtype) {
    case SFFN_BF16: return launch_x<SFFN_BF16>(a, s);
    case SFFN_F32: return launch_x<SFFN_F32>(a, s);
    default: return launch_x<SFFN_E4M3>(a, s);
  }
}

hipError_t launch_mx4_quantize(bool bf16, const void* W, int64_t stride, int32_t N, int32_t K,
                               uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int G = (int)(((int64_t)K + 31) / 32);
  const dim3 grid((unsigned)(((int64_t)N * G + 255) / 256));
  if (bf16)
    mx4_quantize_kernel<uint16_t><<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(W), stride, N,
                                                       K, G, codes, scales);
  else
    mx4_quantize_kernel<float><<<grid, 256, 0, s>>>(static_cast<const float*>(W), stride, N, K, G,
                                                    codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx4_tile(const uint8_t* codes, const uint8_t* scales, const Mx4Dims& d,
                           void* tiled, hipStream_t s) {
  const int64_t n = (int64_t)d.nb * d.kb * 64;
  mx4_tile_kernel<<<dim3((unsigned)((n + 255) / 256)), 256, 0, s>>>(codes, scales, d,
                                                                     static_cast<uint8_t*>(tiled));
  return hipGetLastError();
}

}  // namespace sffn
