// AdamW step over many tensors in one launch, in place.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p - lr (decay p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// Elementwise: every byte of gradient, master, states and parameter is moved once.  A workgroup
// takes ADAMW_CHUNK consecutive elements of one tensor, 8 a lane; the table of tensors comes
// with the kernel's arguments.  8-bit states: 32 lanes hold a block of 256 values, whose
// absolute maxima (of m and of r = sqrt(v)) they reduce for the block's new scales.
#include "ops_common.hpp"

namespace sffn {
namespace {

__device__ __forceinline__ void from_e4m3x4(uint32_t w, float* o) {
  o[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
  o[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
  o[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
  o[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
}

template <typename T>
__device__ __forceinline__ void load_any(const T* p, int n, Raw8<T>& r) {
  if (n >= 8) r.load(p);
  else r.load_n(p, n);
}
template <typename T>
__device__ __forceinline__ void store_any(T* p, const float* v, int n) {
  if (n >= 8) store8(p, v);
  else store8_n(p, v, n);
}
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int n) {
  u32x2 q = u32x2{0, 0};
  if (n >= 8) {
    q = *reinterpret_cast<const u32x2_a1*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
  }
  return q;
}

template <typename P, typename G, bool MASTER, bool BITS8>
__global__ __launch_bounds__(256) void adamw_kernel(AdamwTable tab) {
  // the tensor of this workgroup: the last one whose first workgroup is not past it
  const uint32_t wg = blockIdx.x;
  const int lane = (int)(threadIdx.x & 63);
  const bool at_or_before = lane < ADAMW_TENSORS && tab.first[lane < ADAMW_TENSORS ? lane : 0] <= wg;
  const int ti = uniform(__popcll(ballot64(at_or_before)) - 1);
  const sffn_adamw_tensor_t t = tab.t[ti];
  const int64_t e0 = (int64_t)(wg - tab.first[ti]) * ADAMW_CHUNK + (int)threadIdx.x * 8;
  const int64_t left = t.n - e0;
  const int n = left < 0 ? 0 : left < 8 ? (int)left : 8;
  P* param = static_cast<P*>(t.param) + e0;
  const G* grad = static_cast<const G*>(t.grad) + e0;

  Raw8<G> rg;
  Raw8<float> rm, rv, rw;
  Raw8<P> rp;
  u32x2 qm = u32x2{0, 0}, qr = u32x2{0, 0};
  float ms = 0.f, rs = 0.f;
  const int64_t blk = e0 / SFFN_ADAMW_BLOCK;
  rg.zero();
  rm.zero();
  rv.zero();
  rw.zero();
  rp.zero();
  if (n > 0) {
    load_any(grad, n, rg);
    if constexpr (MASTER) load_any(t.master + e0, n, rw);
    else load_any(static_cast<const P*>(param), n, rp);
    if constexpr (BITS8) {
      qm = load_codes(static_cast<const uint8_t*>(t.m) + e0, n);
      qr = load_codes(static_cast<const uint8_t*>(t.v) + e0, n);
      ms = t.m_scale[blk];
      rs = t.v_scale[blk];
    } else {
      load_any(static_cast<const float*>(t.m) + e0, n, rm);
      load_any(static_cast<const float*>(t.v) + e0, n, rv);
    }
  }
  const float gs = tab.grad_scale ? ld_uniform(tab.grad_scale) : 1.f;
  float m[8], v[8], w[8], root[8];
  if constexpr (BITS8) {
    from_e4m3x4(qm[0], m);
    from_e4m3x4(qm[1], m + 4);
    from_e4m3x4(qr[0], v);
    from_e4m3x4(qr[1], v + 4);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float g = rg.get(i) * gs;
    if constexpr (BITS8) {
      m[i] *= ms;
      v[i] *= rs;
      v[i] *= v[i];
    } else {
      m[i] = rm.get(i);
      v[i] = rv.get(i);
    }
    w[i] = MASTER ? rw.get(i) : rp.get(i);
    m[i] = tab.beta1 * m[i] + tab.one_minus_beta1 * g;
    v[i] = tab.beta2 * v[i] + tab.one_minus_beta2 * (g * g);
    root[i] = sqrtf(v[i]);
    w[i] = w[i] - tab.lr_decay * w[i] -
           tab.step_size * (m[i] / (root[i] * tab.inv_root_correction + tab.eps));
  }
  if constexpr (BITS8) {
    float bm = 0.f, br = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = i < n;  // past the end: codes 0 and gradient 0, but the scale may be anything
      bm = in ? MaxNan()(bm, fabsf(m[i])) : bm;
      br = in ? MaxNan()(br, root[i]) : br;
    }
    bm = lane_reduce<32>(bm, MaxNan()) / E4M3_MAX;
    br = lane_reduce<32>(br, MaxNan()) / E4M3_MAX;
    bm = bm < SCALE_MIN ? SCALE_MIN : bm;
    br = br < SCALE_MIN ? SCALE_MIN : br;
    const float im = 1.f / bm, ir = 1.f / br;
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = m[i] * im;
      const float r = root[i] * ir;
      b[i] = root[i] > 0.f && r < E4M3_TINY ? E4M3_TINY : r;
    }
    if (n > 0) {
      store_e4m3x8(static_cast<uint8_t*>(t.m) + e0, a, n);
      store_e4m3x8(static_cast<uint8_t*>(t.v) + e0, b, n);
      if ((threadIdx.x & 31) == 0) {
        t.m_scale[blk] = bm;
        t.v_scale[blk] = br;
      }
    }
  } else if (n > 0) {
    store_any(static_cast<float*>(t.m) + e0, m, n);
    store_any(static_cast<float*>(t.v) + e0, v, n);
  }
  if (n > 0) {
    if constexpr (MASTER) store_any(t.master + e0, w, n);
    store_any(param, w, n);
  }
}

template <typename P, typename G, bool MASTER>
hipError_t launch_b(int bits, const AdamwTable& t, uint32_t groups, hipStream_t s) {
  if (bits == 8) adamw_kernel<P, G, MASTER, true><<<groups, 256, 0, s>>>(t);
  else adamw_kernel<P, G, MASTER, false><<<groups, 256, 0, s>>>(t);
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
