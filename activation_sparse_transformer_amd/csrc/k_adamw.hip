// AdamW step over many tensors in one launch, in place.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p - lr (decay p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// Elementwise: every byte of gradient, master, states and parameter is moved once, so memory
// bounds it.  A workgroup takes ADAMW_CHUNK consecutive elements of one tensor, 4 a lane (each
// load and store of a wave is one contiguous piece: 8 a lane took 10% longer); the table of
// tensors comes with the kernel's arguments.  Nothing is read again before the next step, so
// tensors that start on a cache line are moved past the caches (non-temporal: 4% faster; a piece
// that ends inside a line would be written twice, so others are not).  8-bit states: a wave
// holds a block of 256 values, whose absolute maxima (of m and of r = sqrt(v)) it reduces for the
// block's new scales.
//
// 85 million values with 32-bit states and a master: 432 us, 5.9 TB/s; 34 million with 8-bit
// states: 107 us, 5.7 TB/s (from a trace).
#include "ops_common.hpp"

namespace sffn {
namespace {

// Four consecutive elements, of which the first n exist.  NT: past the caches.
template <bool NT>
__device__ __forceinline__ void store4(float* p, const float* v, int n) {
  if (n >= 4) {
    store_v<NT>(p, f32x4{v[0], v[1], v[2], v[3]});
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
  }
}
template <bool NT>
__device__ __forceinline__ void store4(uint16_t* p, const float* v, int n) {
  if (n >= 4) {
    store_v<NT>(p,
                u32x2{(uint32_t)f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16),
                      (uint32_t)f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16)});
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = f32_to_bf16(v[i]);
  }
}
template <bool NT>
__device__ __forceinline__ void load_codes4(const uint8_t* p, int n, float* o) {
  uint32_t q = 0;
  if (n >= 4) {
    q = load_v<NT, uint32_t>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) q |= (uint32_t)p[i] << (8 * i);
  }
  o[0] = __builtin_amdgcn_cvt_f32_fp8((int)q, 0);
  o[1] = __builtin_amdgcn_cvt_f32_fp8((int)q, 1);
  o[2] = __builtin_amdgcn_cvt_f32_fp8((int)q, 2);
  o[3] = __builtin_amdgcn_cvt_f32_fp8((int)q, 3);
}
template <bool NT>
__device__ __forceinline__ void store_codes4(uint8_t* p, const float* v, int n) {
  const uint32_t q = e4m3x4(v[0], v[1], v[2], v[3]);
  if (n >= 4) {
    store_v<NT>(p, q);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = (uint8_t)(q >> (8 * i));
  }
}

// The workgroup's part of tensor t from element e0 on (this lane's), n <= 4 of them.
template <typename P, typename G, bool MASTER, bool BITS8, bool NT>
__device__ __forceinline__ void adamw_part(const AdamwTable& tab, const sffn_adamw_tensor_t& t,
                                           int64_t e0, int n) {
  P* param = static_cast<P*>(t.param) + e0;
  const int64_t blk = e0 / SFFN_ADAMW_BLOCK;
  float g[4] = {}, m[4] = {}, v[4] = {}, w[4] = {}, root[4];
  float ms = 0.f, rs = 0.f;
  if (n > 0) {
    load4<NT>(static_cast<const G*>(t.grad) + e0, n, g);
    if constexpr (MASTER) load4<NT>(t.master + e0, n, w);
    else load4<NT>(static_cast<const P*>(param), n, w);
    if constexpr (BITS8) {
      load_codes4<NT>(static_cast<const uint8_t*>(t.m) + e0, n, m);
      load_codes4<NT>(static_cast<const uint8_t*>(t.v) + e0, n, v);
      ms = t.m_scale[blk];
      rs = t.v_scale[blk];
    } else {
      load4<NT>(static_cast<const float*>(t.m) + e0, n, m);
      load4<NT>(static_cast<const float*>(t.v) + e0, n, v);
    }
  }
  const float gs = tab.grad_scale ? ld_uniform(tab.grad_scale) : 1.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g[i] *= gs;
    if constexpr (BITS8) {
      m[i] *= ms;
      v[i] *= rs;
      v[i] *= v[i];
    }
    m[i] = tab.beta1 * m[i] + tab.one_minus_beta1 * g[i];
    v[i] = tab.beta2 * v[i] + tab.one_minus_beta2 * (g[i] * g[i]);
    root[i] = sqrtf(v[i]);
    w[i] = w[i] - tab.lr_decay * w[i] -
           tab.step_size * (m[i] / (root[i] * tab.inv_root_correction + tab.eps));
  }
  if constexpr (BITS8) {
    float bm = 0.f, br = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = i < n;  // past the end: codes 0 and gradient 0, but the scale may be anything
      bm = in ? max_abs(bm, m[i]) : bm;
      br = in ? max_abs(br, root[i]) : br;
    }
    bm = lane_reduce<64>(bm, MaxNan()) / E4M3_MAX;
    br = lane_reduce<64>(br, MaxNan()) / E4M3_MAX;
    bm = bm < SCALE_MIN ? SCALE_MIN : bm;
    br = br < SCALE_MIN ? SCALE_MIN : br;
    const Quotients over_m(bm), over_r(br);
    over_m(m);
    float b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = root[i];
    over_r(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = root[i] > 0.f && b[i] < E4M3_TINY ? E4M3_TINY : b[i];
    if (n > 0) {
      store_codes4<NT>(static_cast<uint8_t*>(t.m) + e0, m, n);
      store_codes4<NT>(static_cast<uint8_t*>(t.v) + e0, b, n);
      if ((threadIdx.x & 63) == 0) {
        t.m_scale[blk] = bm;
        t.v_scale[blk] = br;
      }
    }
  } else if (n > 0) {
    store4<NT>(static_cast<float*>(t.m) + e0, m, n);
    store4<NT>(static_cast<float*>(t.v) + e0, v, n);
  }
  if (n > 0) {
    if constexpr (MASTER) store4<NT>(t.master + e0, w, n);
    store4<NT>(param, w, n);
  }
}

template <typename P, typename G, bool MASTER, bool BITS8>
__global__ __launch_bounds__(ADAMW_CHUNK / 4) void adamw_kernel(AdamwTable tab) {
  // the tensor of this workgroup: the last one whose first workgroup is not past it
  const uint32_t wg = blockIdx.x;
  const int lane = (int)(threadIdx.x & 63);
  const bool at_or_before = lane < ADAMW_TENSORS && tab.first[lane < ADAMW_TENSORS ? lane : 0] <= wg;
  const int ti = uniform(__popcll(ballot64(at_or_before)) - 1);
  const sffn_adamw_tensor_t t = tab.t[ti];
  const int64_t e0 = (int64_t)(wg - tab.first[ti]) * ADAMW_CHUNK + (int)threadIdx.x * 4;
  const int64_t left = t.n - e0;
  const int n = left < 0 ? 0 : left < 4 ? (int)left : 4;
  const uintptr_t at = (uintptr_t)t.param | (uintptr_t)t.grad | (uintptr_t)t.m | (uintptr_t)t.v |
                       (uintptr_t)t.master;
  if ((at & 127) == 0) adamw_part<P, G, MASTER, BITS8, true>(tab, t, e0, n);
  else adamw_part<P, G, MASTER, BITS8, false>(tab, t, e0, n);
}

template <typename P, typename G, bool MASTER>
hipError_t launch_b(int bits, const AdamwTable& t, uint32_t groups, hipStream_t s) {
  if (bits == 8) adamw_kernel<P, G, MASTER, true><<<groups, ADAMW_CHUNK / 4, 0, s>>>(t);
  else adamw_kernel<P, G, MASTER, false><<<groups, ADAMW_CHUNK / 4, 0, s>>>(t);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw(bool param_bf16, bool grad_bf16, bool master, int bits,
                        const AdamwTable& t, uint32_t groups, hipStream_t s) {
  if (!param_bf16)
    return grad_bf16 ? launch_b<float, uint16_t, false>(bits, t, groups, s)
                     : launch_b<float, float, false>(bits, t, groups, s);
  if (master)
    return grad_bf16 ? launch_b<uint16_t, uint16_t, true>(bits, t, groups, s)
                     : launch_b<uint16_t, float, true>(bits, t, groups, s);
  return grad_bf16 ? launch_b<uint16_t, uint16_t, false>(bits, t, groups, s)
                   : launch_b<uint16_t, float, false>(bits, t, groups, s);
}

}  // namespace sffn
