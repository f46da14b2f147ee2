// Products of a few tokens with 4-bit weights: y = act(x W^T * x_scale + bias),
// W[n, k] = e2m1(code) 2^(s - 127) with one s per 32 columns.
//
// One wave holds 16 x 128 weights in a 16-byte load a lane (the tiled layout: 1 KB contiguous),
// expands them to bf16 with the packed conversion that applies the scale (exact: a bf16 holds
// e2m1 times a power of two, from the smallest, 2^-128, to 2^128, where it overflows) and
// multiplies on the matrix cores: A = 16 weight rows, B = up to 16 tokens,
// v_mfma_f32_16x16x32_bf16, four for a block.  Token types: bf16 as it is; e4m3 widened to bf16
// (exact); fp32 as the sum of three bf16 (truncations: 8 + 8 + 8 bits, exact), three products.
// (The scaled 8-bit x 4-bit matrix instruction would need no expansion, but its sums over 128
// columns came out up to 1e-4 of the absolute products off; these are fp32.)
// The waves of a workgroup split k and add their fp32 sums in LDS in wave order.
//
// Bound by reading the weights at few tokens: 65536 x 8192 at 4 tokens 50.2 us (5.7 TB/s); at 64
// tokens and many rows by expansion and products (65536 x 2048 bf16 31 us, e4m3 28).
#include <utility>

#include "mx4_shape.hpp"
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

// 16 tokens x 128 columns on their way to the matrix cores.  A product wants lane (q, r) to hold
// token r, so its own loads would touch 16 rows in every group of 16 lanes, which costs four
// times a contiguous load: a wave loads whole rows instead (LPR lanes a row) and turns them in
// its own piece of LDS.  16-byte units are permuted within a row (by the token) so that the reads
// of 16 rows meet in no bank (the 8-byte ones of e4m3 still do in pairs; it costs no time).
template <int XT>
struct TokTile {
  typedef typename Tok8<XT>::elem E;
  static constexpr int LPR = 8 * (int)sizeof(E);  // lanes of a row
  static constexpr int RPL = 64 / LPR;            // rows of a load
  static constexpr int LOADS = 16 / RPL;
  static constexpr int BYTES = 16 * 128 * (int)sizeof(E);
  u32x4 v[LOADS];

  // tokens t0 .. t0 + 15 (those past the last one are not needed: the last one, or nothing)
  __device__ __forceinline__ void load(const E* x, int64_t stride, int t0, int T, int k0, int lane) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      if (t0 + i * RPL >= T) break;
      const int t = t0 + i * RPL + lane / LPR;
      const E* p = x + (int64_t)(t < T ? t : T - 1) * stride + k0 + lane % LPR * (128 / LPR);
      v[i] = *reinterpret_cast<const u32x4_a1*>(p);
    }
  }
  static __device__ __forceinline__ int unit(int t, int u) {
    return t * LPR + (u ^ (t & (LPR < 16 ? LPR - 1 : 15)));
  }
  __device__ __forceinline__ void put(u32x4* lds, int lane) const {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) lds[unit(i * RPL + lane / LPR, lane % LPR)] = v[i];
  }
  // columns 32 j + 8 q .. + 7 of token r
  static __device__ __forceinline__ Tok8<XT> get(const u32x4* lds, int j, int q, int r) {
    Tok8<XT> o;
    if constexpr (XT == SFFN_BF16) {
      o.r = lds[unit(r, 4 * j + q)];
    } else if constexpr (XT == SFFN_F32) {
      o.r[0] = __builtin_bit_cast(f32x4, lds[unit(r, 8 * j + 2 * q)]);
      o.r[1] = __builtin_bit_cast(f32x4, lds[unit(r, 8 * j + 2 * q + 1)]);
    } else {
      o.r = reinterpret_cast<const u32x2*>(lds + unit(r, 2 * j + (q >> 1)))[q & 1];
    }
    return o;
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

// Orders a wave's accesses to its own piece of LDS: the hardware carries them out in order, only
// the compiler has to keep it.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A wave's weights of one block of 128 columns: RB blocks of 16 rows.
template <int RB>
struct Mx4Weights {
  u32x4 c[RB];
  uint32_t sc[RB];

  __device__ __forceinline__ void load(const uint8_t* const* w, int kb, int lane) {
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const uint8_t* p = w[b] + (size_t)kb * MX4_BLOCK;
      c[b] = *reinterpret_cast<const u32x4*>(p + lane * 16);
      sc[b] = *reinterpret_cast<const uint32_t*>(p + 1024 + (lane & 15) * 4);
    }
  }
  // token(j, t): the lane's columns of word j of token tile t
  template <int XT, int TT, typename F>
  __device__ __forceinline__ void product(f32x4 (&acc)[RB][TT], F token) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x8 w[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b)
        w[b] = expand8(c[b][j], __uint_as_float(((sc[b] >> (8 * j)) & 0xffu) << 23));
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        bf16x8 xt[Tok8<XT>::TERMS];
        token(j, t).terms(xt);
#pragma unroll
        for (int k = Tok8<XT>::TERMS - 1; k >= 0; --k)
#pragma unroll
          for (int b = 0; b < RB; ++b)
            acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[b], xt[k], acc[b][t], 0, 0, 0);
      }
    }
  }
};

// KS of a workgroup's waves split k, the others take further rows.  Rows past the end are read as
// the last one and not stored; what a column without a token holds is not stored either (a
// product's columns do not mix).  More than 16 tokens are turned in LDS; up to 16 each lane loads
// its own (one token is then one access a group of lanes: 3.6 against 3.9 us at 8192 x 2048,
// launches one after another; 4.2 in a trace).
// Many waves hide the loads: a second block of columns in flight in a wave gained nothing.
template <int XT, int TT, int RB, int KS>
__global__ __launch_bounds__(MX4_WAVES * 64, (mx4_pairs(XT, TT, RB) ? 4 : 2)) void
mx4_linear_kernel(Mx4Args a) {
  typedef TokTile<XT> Tile;
  typedef typename Tile::E E;
  constexpr bool TURN = TT > 1;
  constexpr int UNITS = TURN ? TT * Tile::BYTES / 16 : 0;  // of a wave's tokens
  constexpr int PART = RB * TT * 64;                       // of a wave's sums
  __shared__ u32x4 lds[MX4_WAVES * (UNITS > PART ? UNITS : PART)];
  const int lane = (int)(threadIdx.x & 63), wave = uniform((int)(threadIdx.x >> 6));
  const int q = lane >> 4, r = lane & 15;
  const int wg0 = (int)blockIdx.x * (RB * MX4_WAVES / KS);
  const int rb0 = wg0 + wave / KS * RB, t0 = (int)blockIdx.y * (TT * 16);
  const int K = a.d.K, whole = K / 128;
  const E* x = static_cast<const E*>(a.x);

  const uint8_t* w[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int rb = rb0 + b < a.d.nb ? rb0 + b : a.d.nb - 1;
    w[b] = static_cast<const uint8_t*>(a.tiled) + (size_t)rb * a.d.kb * MX4_BLOCK;
  }
  f32x4 acc[RB][TT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[b][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  if constexpr (TURN) {
    u32x4* own = lds + wave * UNITS;
    for (int kb = wave % KS; kb < whole; kb += KS) {
      Mx4Weights<RB> wt;
      Tile tile[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) tile[t].load(x, a.x_stride, t0 + t * 16, a.T, kb * 128, lane);
      wt.load(w, kb, lane);
#pragma unroll
      for (int t = 0; t < TT; ++t) tile[t].put(own + t * (Tile::BYTES / 16), lane);
      wave_fence();
      wt.template product<XT, TT>(acc, [&](int j, int t) {
        return Tile::get(own + t * (Tile::BYTES / 16), j, q, r);
      });
      wave_fence();
    }
  } else {
    const E* x_row = x + (int64_t)(t0 + r) * a.x_stride + q * 8;
    const bool have = t0 + r < a.T;
    Tok8<XT> tok[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) tok[j].zero();
    for (int kb = wave % KS; kb < whole; kb += KS) {
      Mx4Weights<RB> wt;
      wt.load(w, kb, lane);
      if (have) {
#pragma unroll
        for (int j = 0; j < 4; ++j) tok[j].load(x_row + kb * 128 + 32 * j);
      }
      wt.template product<XT, TT>(acc, [&](int j, int) { return tok[j]; });
    }
  }
  if (whole < a.d.kb && wave % KS == whole % KS) {  // the last, partial block of columns
    Mx4Weights<RB> wt;
    wt.load(w, whole, lane);
    wt.template product<XT, TT>(acc, [&](int j, int t) {
      const int tok = t0 + t * 16 + r, k0 = whole * 128 + 32 * j + 8 * q, n = K - k0;
      Tok8<XT> o;
      o.zero();
      if (tok < a.T && n > 0) {
        const E* p = x + (int64_t)tok * a.x_stride + k0;
        if (n >= 8) o.load(p);
        else o.load_n(p, n);
      }
      return o;
    });
  }

  __syncthreads();  // the sums take the tokens' place
  f32x4* part = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < TT; ++t) part[wave * PART + (b * TT + t) * 64 + lane] = acc[b][t];
  __syncthreads();
  for (int i = (int)threadIdx.x; i < MX4_WAVES / KS * PART; i += MX4_WAVES * 64) {
    const int g = i / PART, at = i % PART, l = at & 63, t = (at >> 6) % TT, b = (at >> 6) / TT;
    f32x4 s = part[g * KS * PART + at];
#pragma unroll
    for (int v = 1; v < KS; ++v) s += part[(g * KS + v) * PART + at];
    mx4_store(a, s, t0 + t * 16 + (l & 15), (wg0 + g * RB + b) * 16 + (l >> 4) * 4);
  }
}

template <int XT, int TT, int RB, int KS>
hipError_t launch_form(const Mx4Args& a, hipStream_t s) {
  constexpr int ROWS = RB * MX4_WAVES / KS;
  const dim3 grid((unsigned)((a.d.nb + ROWS - 1) / ROWS), (unsigned)mx4_token_groups(a.T, TT));
  mx4_linear_kernel<XT, TT, RB, KS><<<grid, MX4_WAVES * 64, 0, s>>>(a);
  return hipGetLastError();
}

// I: one of the 4 x 4 x 3 forms, launched if it is f.
template <int XT, int I>
bool launch_if(const Mx4Args& a, const Mx4Shape& f, hipStream_t s, hipError_t* e) {
  constexpr int TT = I / 12 + 1, RB = I / 3 % 4 + 1, KS = 2 << I % 3;
  if constexpr (mx4_built(XT, TT, RB, KS)) {
    if (f.tt == TT && f.rb == RB && f.ks == KS) {
      *e = launch_form<XT, TT, RB, KS>(a, s);
      return true;
    }
  }
  return false;
}
template <int XT, int... I>
hipError_t launch_x(const Mx4Args& a, hipStream_t s, std::integer_sequence<int, I...>) {
  const Mx4Shape f = mx4_shape(XT, a.d.nb, a.d.kb, a.T);
  hipError_t e = hipErrorInvalidValue;
  (void)(launch_if<XT, I>(a, f, s, &e) || ...);
  return e;
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
  const int lane = (int)(i & 63), q = lane >> 4, G = (d.K + 31) / 32;
  const int64_t row0 = blk / d.kb * 16, n = row0 + (lane & 15);
  const int g0 = (int)(blk % d.kb) * 4;
  u32x4 c = u32x4{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (n >= d.N || g0 + j >= G) continue;
    c[j] = *reinterpret_cast<const u32_a1*>(codes + (n * G + g0 + j) * 16 + q * 4);
    const int len = d.K - (g0 + j) * 32 - q * 8;  // codes past the columns' end: 0
    if (len <= 0) c[j] = 0;
    else if (len < 8) c[j] &= (1u << (4 * len)) - 1;
  }
  uint8_t* p = tiled + blk * MX4_BLOCK;
  *reinterpret_cast<u32x4*>(p + lane * 16) = c;
  const int64_t sn = row0 + (lane >> 2);  // scales: row by row, the block's four groups each
  const int sg = g0 + (lane & 3);
  p[1024 + lane] = sn < d.N && sg < G ? scales[sn * G + sg] : 127;
}

}  // namespace

hipError_t launch_mx4_linear(const Mx4Args& a, hipStream_t s) {
  const auto forms = std::make_integer_sequence<int, 48>();
  switch (a.x_dtype) {
    case SFFN_BF16: return launch_x<SFFN_BF16>(a, s, forms);
    case SFFN_F32: return launch_x<SFFN_F32>(a, s, forms);
    default: return launch_x<SFFN_E4M3>(a, s, forms);
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
