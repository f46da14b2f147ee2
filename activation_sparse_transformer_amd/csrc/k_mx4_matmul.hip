// Products of 4-bit tokens with 4-bit weights: y = act(x W^T + bias).
//
// The scaled matrix instructions multiply e2m1 values whose groups of 32 columns have their own powers
// of two; a product of two of them has at most 4 bits, and their sum comes out within two fp32 roundings
// (exact where the scales of a row differ by up to 2^4).  A lane of an operand holds 32 columns of a row in
// 16 bytes, and their scale in a byte.
//
// Both operands come in blocks of 16 rows x 128 columns (MX4_BLOCK bytes): units of 16 bytes, lane by
// lane, lane (q, r) = 16 q + r being the one of row r.  In a block of tokens, unit (q, r) is columns 32 q to
// 32 q + 31, as the instructions take them, but for the order of its words, 8 columns each: 0, 2, 1, 3 (any
// order is right that the weights have too; this one costs no moves).  A block of weights is in the order of the few-token product
// of bf16 values: word g of unit (q, r) is columns 32 g + 8 q to 32 g + 8 q + 7, so what the instructions
// want is the transpose over q and the words; swaps of lane rows give it.
#include <utility>

#include "mx4_matmul_form.hpp"
#include "ops_common.hpp"

namespace sffn {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr;
constexpr int FEW_WAVES = 8;  // of a workgroup of the forms for few tokens

// s_waitcnt for at most n vector-memory operations in flight, and for all LDS operations.
constexpr int vmcnt(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }
constexpr int LGKM0 = 0xC07F;

__device__ __forceinline__ f32x4 mfma(u32x4 a, int sa, u32x4 b, int sb, f32x4 c) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, sa, 0, sb);
}

// Direct loads to LDS, 16 bytes a lane, lane after lane: of 1 KB at base + at (both uniform: a buffer load,
// which needs no address arithmetic in vector registers), and of each lane's own 16 bytes.
__device__ __forceinline__ void load_block(const uint8_t* base, uint32_t at, int lane, u32x4* lds) {
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, -1, 0x00027000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)lds, 16, lane * 16, at, 0, 0);
}
__device__ __forceinline__ void load_units(const uint8_t* from, u32x4* lds) {
  __builtin_amdgcn_global_load_lds(from, (lds_ptr)lds, 16, 0, 0);
}

// Orders a wave's accesses to its own piece of LDS: the hardware carries them out in order, only
// the compiler has to keep it.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16);
}
// Four bias values from n on, 0 past the last one.
__device__ __forceinline__ f32x4 bias4(const float* bias, int n, int N) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (!bias) return v;
  if (n + 4 <= N) return *reinterpret_cast<const f32x4_a4*>(bias + n);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < N) v[e] = bias[n + e];
  return v;
}

// ------------------------------------------------------------------ many tokens
// 32 x 32 x 64 products (6.1 to 6.6 PFLOP/s from registers alone, where 16 x 16 x 128 ones reach 4.3 to
// 5.4).  2 x 2 waves, each with NP pairs of blocks of weight rows by TP pairs of blocks of tokens.  The
// operands of 128 columns are a stage of LDS, filled by direct loads RING stages ahead; a wave reads the
// next stage's fragments while the current one's products run.
//
// 16384 x 9216 x 2304 (bf16 results) takes 218 us, 3.2 PFLOP/s; 8192 x 8192 x 8192 286 us, 3.8 PFLOP/s.  At the former
// the matrix units are busy 41% of the cycles, at 1.86 GHz: a CU has 18 tiles in 9 rounds, each with about 7 us of
// first loads and results in which they idle (65 us), and the waves wait to issue for 39% of their cycles; with
// zeros for codes the same instructions take 0.74 of the time, so a quarter is the power of the products.  With k
// of 16384 (2048 x 8192) they are busy 51% of the cycles, at 1.74 GHz (zeros: 0.70).  Tried without gain: products
// and reads interleaved by hand, fewer vector instructions, one wave a SIMD with 128 x 128 products (spills).
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int WAVES = 4;
constexpr int RING = 3;  // stages in LDS (4 to 8 gained nothing: the loads are hidden)

template <int NP, int TP>
struct Form {
  static constexpr int NW = 2 * NP * 2, TW = 2 * TP * 2;  // blocks of a workgroup
  static constexpr int BLOCKS = NW + TW;
  static constexpr int LOADS = BLOCKS / WAVES;  // of codes, of a wave and stage; and one of scales
  static constexpr int SCALE_LOADS = (BLOCKS + 15) / 16;
  static constexpr int UNITS = BLOCKS * 64 + SCALE_LOADS * 64;  // 16-byte units of a stage
  // where a wave turns its results: two waves' places in a stage's memory
  static constexpr int F32_PAIRS = NP >= 2 && 2 * 32 * 17 <= UNITS ? 2 : 1;
  static constexpr int REGION = 32 * ((F32_PAIRS * 8 > NP * 4 ? F32_PAIRS * 8 : NP * 4) + 1);
  static_assert(2 * REGION <= UNITS, "results in LDS");
  // workgroups of a CU, by LDS and by the registers of the sums and fragments
  static constexpr int REGS = NP * TP * 16 + NP * 18 + TP * 18 + 20;
  static constexpr int BY_LDS = 160 * 1024 / (RING * UNITS * 16), BY_REGS = 512 / REGS * 4 / WAVES;
  static constexpr int PER_CU = BY_LDS < BY_REGS ? BY_LDS : BY_REGS;
  static_assert(BLOCKS % WAVES == 0 && SCALE_LOADS <= WAVES && PER_CU >= 1, "loads of a stage");
};

// Calls f(0), f(1), ... with integral constants until one returns true.
template <int... I, typename F>
__device__ __forceinline__ bool until(std::integer_sequence<int, I...>, F&& f) {
  return (f(std::integral_constant<int, I>()) || ...);
}

template <int OP>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, int sa, u32x4 b, int sb, f32x16 c) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, OP, sa, OP, sb);
}

// The results of a wave, NP x TP products, from token tok0 and row n0 on; PAIRS: pairs of blocks of rows at a
// time.  Element e of a product, lane (h, row): weight row 8 (e / 4) + 4 h + e % 4, token `row`.
template <typename Y, int NP, int TP, int PAIRS>
__device__ __forceinline__ void write_tile(const Mx4MatmulArgs& a, const f32x16 (&acc)[NP][TP], u32x4* own,
                                           int64_t tok0, int n0, int lane) {
  constexpr int PER = 16 / (int)sizeof(Y);              // elements of a unit
  constexpr int ROW = PAIRS * 32 / PER, PITCH = ROW + 1;  // units of a token
  const int h = lane >> 5, row = lane & 31, N = a.d.N;
  const float floor = a.relu ? 0.f : -INFINITY;
#pragma unroll
  for (int g = 0; g < NP; g += PAIRS) {
    f32x4 bias[PAIRS][4];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) bias[i][j] = bias4(a.bias, n0 + (g + i) * 32 + 8 * j + 4 * h, N);
#pragma unroll
    for (int t = 0; t < TP; ++t) {
      wave_fence();
#pragma unroll
      for (int i = 0; i < PAIRS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = acc[g + i][t][4 * j + e] + bias[i][j][e];
            v[e] = v[e] < floor ? floor : v[e];
          }
          Y* to = reinterpret_cast<Y*>(own + row * PITCH) + i * 32 + 8 * j + 4 * h;
          if constexpr (sizeof(Y) == 2)
            *reinterpret_cast<u32x2*>(to) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
          else
            *reinterpret_cast<f32x4*>(to) = f32x4{v[0], v[1], v[2], v[3]};
        }
      wave_fence();
      constexpr int AT_ONCE = 64 / ROW;  // tokens of an access
#pragma unroll
      for (int k = 0; k < 32 / AT_ONCE; ++k) {
        const int r = k * AT_ONCE + lane / ROW, u = lane % ROW;
        const u32x4 o = own[r * PITCH + u];
        const int64_t tok = tok0 + t * 32 + r;
        const int n = n0 + g * 32 + u * PER;
        if (tok >= a.T) continue;
        Y* y = static_cast<Y*>(a.y) + tok * N + n;
        if (n + PER <= N) {
          if (a.past_caches) __builtin_nontemporal_store(o, reinterpret_cast<u32x4_a2*>(y));
          else store_v<false>(y, o);
        } else {
#pragma unroll
          for (int e = 0; e < PER; ++e)
            if (n + e < N) y[e] = sizeof(Y) == 2 ? (Y)(o[e >> 1] >> (16 * (e & 1))) : __uint_as_float(o[e & 3]);
        }
      }
    }
  }
}

template <int NP, int TP>
__global__ __launch_bounds__(WAVES * 64, (Form<NP, TP>::PER_CU)) void mx4_matmul_kernel(
    Mx4MatmulArgs a) {
  typedef Form<NP, TP> F;
  __shared__ u32x4 ring[RING][F::UNITS];
  const int lane = (int)(threadIdx.x & 63), wave = uniform((int)(threadIdx.x >> 6));
  const int h = lane >> 5, row = lane & 31;  // lane (h, row) of a 32-row operand
  const int wn = wave & 1, wt = wave >> 1;
  const int nb = a.d.nb, kbs = a.d.kb, tb = (a.T + 15) / 16;

  // The tile of this workgroup.  Workgroups go to the 8 XCDs in turn: each XCD takes consecutive tiles,
  // and those run over 8 tiles of tokens first, so that what its workgroups read at a time fits its L2.
  const int tn = (nb + F::NW - 1) / F::NW, tt = (tb + F::TW - 1) / F::TW, total = tn * tt;
  const int xcd = (int)blockIdx.x & 7, lin = (int)blockIdx.x / 8 + xcd * (total / 8) + (xcd < total % 8 ? xcd : total % 8);
  const int group = lin / (8 * tn), gt = tt - group * 8 < 8 ? tt - group * 8 : 8, rem = lin - group * 8 * tn;
  const int n0 = rem / gt * F::NW, t0 = (group * 8 + rem % gt) * F::TW;

  // Sources of this wave's direct loads, as buffers (the lane's and the stage's offsets need no address
  // arithmetic); blocks past the last one are read as the last one.
  const auto block_at = [&](int b) {
    const bool w = b < F::NW;
    int i = w ? n0 + b : t0 + b - F::NW;
    const int last = (w ? nb : tb) - 1;
    i = i < last ? i : last;
    return static_cast<const uint8_t*>(w ? a.tiled : a.tokens) + (size_t)i * kbs * MX4_BLOCK;
  };
  const uint8_t* src[F::LOADS];
#pragma unroll
  for (int i = 0; i < F::LOADS; ++i) src[i] = block_at(wave * F::LOADS + i);
  const int sl = wave % F::SCALE_LOADS;  // (several waves may load the same scales to the same place)
  const int sb = sl * 16 + (lane >> 2);
  const uint8_t* scale_src = block_at(sb < F::BLOCKS ? sb : F::BLOCKS - 1) + 1024 + (lane & 3) * 16;

  const auto issue = [&](int kb, u32x4* s) __attribute__((always_inline)) {
    const uint32_t at = (uint32_t)kb * MX4_BLOCK;
#pragma unroll
    for (int i = 0; i < F::LOADS; ++i)
      load_block(src[i], at, lane, s + (wave * F::LOADS + i) * 64);
    load_units(scale_src + at, s + F::BLOCKS * 64 + sl * 64);
  };

  // Fragments of a stage.  A row has four scales in a word; the lanes of h = 1 take the odd groups.
  const int unit = (row >> 4) * 64 + (row & 15);  // of lane row in a pair of blocks, q = 0
  const int w_at = wn * NP * 128 + unit + 32 * h, x_at = (F::NW + wt * TP * 2) * 64 + unit + 16 * h;
  const int ws_at = wn * NP * 32 + row, xs_at = (F::NW + wt * TP * 2) * 16 + row;
  u32x4 w[2][NP][2], x[2][TP][2];
  uint32_t ws[2][NP], xs[2][TP];
  const auto fragments = [&](const u32x4* s, int c) __attribute__((always_inline)) {
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(s + F::BLOCKS * 64);
#pragma unroll
    for (int t = 0; t < TP; ++t) {
#pragma unroll
      for (int k = 0; k < 2; ++k) x[c][t][k] = s[x_at + t * 128 + k * 32];
      xs[c][t] = sc[xs_at + t * 32];
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const u32x2 u = reinterpret_cast<const u32x2*>(s + w_at + i * 128)[k];
        const u32x2 v = reinterpret_cast<const u32x2*>(s + w_at + i * 128 + 16)[k];
        w[c][i][k] = u32x4{u[0], u[1], v[0], v[1]};
      }
      ws[c][i] = sc[ws_at + i * 32];
    }
  };
  f32x16 acc[NP][TP];
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int t = 0; t < TP; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][t][e] = 0.f;

  // A stage, whose fragments are in registers (set c).  Once every wave has them its buffer is free for the
  // stage RING ahead; the next stage is in when only those after it may still be loading, and its
  // fragments are read while this one's products run.  Past the end the last stage is loaded again, into
  // buffers that nothing reads.
  const auto stage = [&](int kb, u32x4* s, const u32x4* next, int c) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(vmcnt((RING - 2) * (F::LOADS + 1)));
    __builtin_amdgcn_s_waitcnt(LGKM0);
    __asm__ volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    issue(kb + RING < kbs ? kb + RING : kbs - 1, s);
    fragments(next, c ^ 1);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // words 2 k and 2 k + 1 of units 2 h and 2 h + 1: swapped, they are units 0, 2, 1, 3 of group 2 k
        // (h = 0) and 2 k + 1 (h = 1)
        const auto u = __builtin_amdgcn_permlane32_swap(w[c][i][k][0], w[c][i][k][1], false, false);
        const auto v = __builtin_amdgcn_permlane32_swap(w[c][i][k][2], w[c][i][k][3], false, false);
        w[c][i][k] = u32x4{u[0], u[1], v[0], v[1]};
      }
      ws[c][i] >>= 8 * h;
    }
#pragma unroll
    for (int t = 0; t < TP; ++t) xs[c][t] >>= 8 * h;
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int t = 0; t < TP; ++t) acc[i][t] = mfma32<0>(w[c][i][0], (int)ws[c][i], x[c][t][0], (int)xs[c][t], acc[i][t]);
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int t = 0; t < TP; ++t) acc[i][t] = mfma32<2>(w[c][i][1], (int)ws[c][i], x[c][t][1], (int)xs[c][t], acc[i][t]);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int i = 0; i < RING; ++i) issue(i < kbs ? i : kbs - 1, ring[i]);
  __builtin_amdgcn_s_waitcnt(vmcnt((RING - 1) * (F::LOADS + 1)));
  __asm__ volatile("s_barrier" ::: "memory");
  fragments(ring[0], 0);
  // turns of the ring, twice where a turn changes the fragments' set, until the last stage is done
  constexpr int TURN = RING % 2 ? 2 * RING : RING;
  int kb = 0;
  while (!until(std::make_integer_sequence<int, TURN>(), [&](auto i) __attribute__((always_inline)) {
    constexpr int I = decltype(i)::value;
    stage(kb, ring[I % RING], ring[(I + 1) % RING], I & 1);
    return ++kb == kbs;
  })) {
  }
  __builtin_amdgcn_s_waitcnt(vmcnt(0));  // the repeated loads land before LDS goes away

  // The results go through LDS, a wave's 32 tokens by 64 to 128 rows at a time, so that whole cache lines
  // are written where y's rows start on one: pieces of 32 bytes a token, as a wave holds them, took three times
  // as long.
  __asm__ volatile("s_barrier" ::: "memory");  // the fragments of every wave are read
  u32x4* own = ring[wave >> 1] + (wave & 1) * F::REGION;
  const int64_t tok0 = (int64_t)(t0 + wt * TP * 2) * 16;
  const int n = (n0 + wn * NP * 2) * 16;
  if (a.y_bf16) write_tile<uint16_t, NP, TP, NP>(a, acc, own, tok0, n, lane);
  else write_tile<float, NP, TP, F::F32_PAIRS>(a, acc, own, tok0, n, lane);
}

// ------------------------------------------------------------------ few tokens
// Eight waves split the columns; every wave loads its weights (RB blocks of rows) and tokens (TT blocks) as
// the 16 x 16 x 128 instruction takes them (weights: swapped lane rows), and the waves' sums are added
// in order.  Up to 16 tokens may come as they are (X: their type): a lane then rounds the 32 columns that
// it holds, every wave its own, which is less than a launch and a pass over memory.

// The transpose over a lane's words and the four lane rows, words 1 and 2 exchanged as in the tokens.
__device__ __forceinline__ u32x4 transpose(u32x4 w) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], d[0], c[1], d[1]};
}

// Lane (q, r)'s part of a block of tokens: from the layout, or rounded.
template <typename X>
struct TokenBlock {
  Raw8<X> v[4];
  __device__ __forceinline__ void load(const Mx4MatmulArgs& a, int tb, int kb, int q, int r) {
    const int64_t k0 = (int64_t)kb * 128 + 32 * q;
    const X* p = static_cast<const X*>(a.tokens) + (int64_t)r * a.x_stride + k0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = a.d.K - k0 - 8 * j;
      v[j].zero();
      if (r < a.T) {
        if (n >= 8) v[j].load(p + 8 * j);
        else if (n > 0) v[j].load_n(p + 8 * j, (int)n);
      }
    }
  }
  __device__ __forceinline__ void get(u32x4& codes, int& scale) const {
    float big = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) big = max_abs(big, v[j].get(e));
    const uint32_t s = mx4_scale(big);
    codes = u32x4{mx4_codes8(v[0], s), mx4_codes8(v[2], s), mx4_codes8(v[1], s), mx4_codes8(v[3], s)};
    scale = (int)s;
  }
};
template <>
struct TokenBlock<void> {
  u32x4 c;
  int s;
  __device__ __forceinline__ void load(const Mx4MatmulArgs& a, int tb, int kb, int q, int r) {
    const uint8_t* p = static_cast<const uint8_t*>(a.tokens) + ((size_t)tb * a.d.kb + kb) * MX4_BLOCK;
    c = *reinterpret_cast<const u32x4*>(p + (q * 16 + r) * 16);
    s = p[1024 + r * 4 + q];
  }
  __device__ __forceinline__ void get(u32x4& codes, int& scale) const {
    codes = c;
    scale = s;
  }
};

template <typename X, int TT, int RB>
__global__ __launch_bounds__(FEW_WAVES * 64, 2) void mx4_matmul_few_kernel(Mx4MatmulArgs a) {
  constexpr int PART = RB * TT * 64;
  __shared__ f32x4 part[FEW_WAVES * PART];
  const int lane = (int)(threadIdx.x & 63), wave = uniform((int)(threadIdx.x >> 6));
  const int q = lane >> 4, r = lane & 15, kbs = a.d.kb, tb = (a.T + 15) / 16;
  const int rb0 = (int)blockIdx.x * RB;
  const int tb0 = (int)blockIdx.y * TT;
  const uint8_t* w[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int i = rb0 + b < a.d.nb ? rb0 + b : a.d.nb - 1;
    w[b] = static_cast<const uint8_t*>(a.tiled) + (size_t)i * kbs * MX4_BLOCK;
  }
  f32x4 acc[RB][TT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[b][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // (many waves hide the loads: a block's loaded one turn ahead cost occupancy and time)
  for (int kb = wave; kb < kbs; kb += FEW_WAVES) {
    const size_t at = (size_t)kb * MX4_BLOCK;
    u32x4 wc[RB], xc[TT];
    int ws[RB], xs[TT];
    TokenBlock<X> x[TT];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      wc[b] = *reinterpret_cast<const u32x4*>(w[b] + at + lane * 16);
      ws[b] = w[b][at + 1024 + r * 4 + q];
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) x[t].load(a, tb0 + t < tb ? tb0 + t : tb - 1, kb, q, r);
#pragma unroll
    for (int t = 0; t < TT; ++t) x[t].get(xc[t], xs[t]);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const u32x4 wt = transpose(wc[b]);
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[b][t] = mfma(wt, ws[b], xc[t], xs[t], acc[b][t]);
    }
  }
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < TT; ++t) part[wave * PART + (b * TT + t) * 64 + lane] = acc[b][t];
  __syncthreads();
  // lane (q, r) of a product has rows 4 q .. 4 q + 3 for token r
  const int N = a.d.N;
  for (int i = (int)threadIdx.x; i < PART; i += FEW_WAVES * 64) {
    const int l = i & 63, t = (i >> 6) % TT, b = (i >> 6) / TT;
    f32x4 s = part[i];
#pragma unroll
    for (int v = 1; v < FEW_WAVES; ++v) s += part[v * PART + i];
    const int64_t tok = (int64_t)(tb0 + t) * 16 + (l & 15);
    const int n = (rb0 + b) * 16 + (l >> 4) * 4;
    if (tok >= a.T || n >= N) continue;
    const f32x4 bias = bias4(a.bias, n, N);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = s[e] + bias[e];
      v[e] = a.relu && v[e] < 0.f ? 0.f : v[e];
    }
    if (a.y_bf16) {
      uint16_t* y = static_cast<uint16_t*>(a.y) + tok * N + n;
      if (n + 4 <= N) {
        *reinterpret_cast<u32x2_a2*>(y) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      } else {
        for (int e = 0; e < N - n; ++e) y[e] = f32_to_bf16(v[e]);
      }
    } else {
      float* y = static_cast<float*>(a.y) + tok * N + n;
      if (n + 4 <= N) {
        *reinterpret_cast<f32x4_a4*>(y) = f32x4{v[0], v[1], v[2], v[3]};
      } else {
        for (int e = 0; e < N - n; ++e) y[e] = v[e];
      }
    }
  }
}

template <int NP, int TP>
hipError_t launch_form(const Mx4MatmulArgs& a, hipStream_t s) {
  typedef Form<NP, TP> F;
  const int64_t tn = (a.d.nb + F::NW - 1) / F::NW, tt = ((a.T + 15) / 16 + F::TW - 1) / F::TW;
  mx4_matmul_kernel<NP, TP><<<dim3((unsigned)(tn * tt)), WAVES * 64, 0, s>>>(a);
  return hipGetLastError();
}

template <typename X, int TT, int RB>
hipError_t launch_few(const Mx4MatmulArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.d.nb + RB - 1) / RB), (unsigned)(((a.T + 15) / 16 + TT - 1) / TT));
  mx4_matmul_few_kernel<X, TT, RB><<<grid, FEW_WAVES * 64, 0, s>>>(a);
  return hipGetLastError();
}
template <typename X>
hipError_t launch_rounding(const Mx4MatmulArgs& a, hipStream_t s) {
  switch (mx4_matmul_form(a.d.nb, a.d.kb, a.T, true, !a.y_bf16)) {
    case MX4_FEW_16x1: return launch_few<X, 1, 1>(a, s);
    case MX4_FEW_16x2: return launch_few<X, 1, 2>(a, s);
    default: return launch_few<X, 1, 4>(a, s);
  }
}

}  // namespace

hipError_t launch_mx4_matmul(const Mx4MatmulArgs& a0, hipStream_t s) {
  Mx4MatmulArgs a = a0;
  // bf16 results of the tile forms go past the caches whatever their size, fp32 ones where they would fill them.
  // (Prompts, us a call, past the caches and through them: bf16 results of 32 MB 33 and 35, 128 MB 100 and
  // 103, 288 MB 232 and 270; fp32 of 64 MB 40 and 37, 128 MB 75 and 66, 256 MB 123 and 130.  Small bf16 results with
  // a norm that reads them next, us of kernels: 1 MB 7.9 and 7.9, 4 MB 13.3 and 13.3, 16 MB 30.0 and 32.1, 32 MB
  // 42.7 and 43.7, 72 MB 98.5 and 98.5.  Rows that start off a line, 8191 columns of 16 MB: 32.7 and 33.3, but 9217 of
  // 72 MB: 103.5 and 98.2, the product alone 72 and 62.)
  a.past_caches = a.y_bf16 || (int64_t)a.T * a.d.N > 48 << 20;
  if (a.x_dtype == SFFN_F32) return launch_rounding<float>(a, s);
  if (a.x_dtype == SFFN_BF16) return launch_rounding<uint16_t>(a, s);
  switch (mx4_matmul_form(a.d.nb, a.d.kb, a.T, false, !a.y_bf16)) {
    case MX4_FEW_16x1: return launch_few<void, 1, 1>(a, s);
    case MX4_FEW_16x2: return launch_few<void, 1, 2>(a, s);
    case MX4_FEW_32x1: return launch_few<void, 2, 1>(a, s);
    case MX4_FEW_32x2: return launch_few<void, 2, 2>(a, s);
    case MX4_FEW_64x2: return launch_few<void, 4, 2>(a, s);
    case MX4_TILE_64x64: return launch_form<1, 1>(a, s);
    case MX4_TILE_128x64: return launch_form<2, 1>(a, s);
    case MX4_TILE_128x128: return launch_form<2, 2>(a, s);
    case MX4_TILE_128x256: return launch_form<2, 4>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sffn
