// Host side of the C ABI declared in include/ffn_ops.h: argument checks (always before any HIP
// call) and launches on the caller's stream.
#include <cmath>
#include <cstring>

#include "entry.hpp"
#include "ops_common.hpp"

using namespace sffn;

namespace {

#define OPS_TRY(expr)                        \
  do {                                       \
    const sffn_status_t s__ = (expr);        \
    if (s__ != SFFN_OK) return s__;          \
  } while (0)

sffn_status_t invalid(const char* msg) { return api_fail(SFFN_ERR_INVALID_ARGUMENT, msg); }
sffn_status_t unsupported(const char* msg) { return api_fail(SFFN_ERR_UNSUPPORTED, msg); }

bool misaligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }
size_t size_of(int32_t dtype) { return dtype == SFFN_F32 ? 4 : dtype == SFFN_BF16 ? 2 : 1; }

sffn_status_t check_types(int32_t dtype, int32_t gain_dtype) {
  if (dtype != SFFN_F32 && dtype != SFFN_BF16) return invalid("dtype must be SFFN_F32 or SFFN_BF16");
  if (gain_dtype != dtype && gain_dtype != SFFN_F32)
    return invalid("gain_dtype must be dtype or SFFN_F32");
  return SFFN_OK;
}

sffn_status_t check_rows(int64_t rows, int32_t d) {
  if (rows < 0 || rows > (int64_t)1 << 40) return invalid("rows must be in [0, 2^40]");
  if (d < 1) return invalid("d must be positive");
  if (d > SFFN_NORM_MAX_D) return unsupported("d must be at most SFFN_NORM_MAX_D");
  return SFFN_OK;
}

// A matrix argument of `rows` rows: pointer, row stride, element alignment.
sffn_status_t check_matrix(const void* p, int64_t stride, int64_t rows, int32_t d, int32_t dtype,
                           const char* null_msg, const char* stride_msg) {
  if (!p) return invalid(null_msg);
  if (rows > 1 && (stride < d || stride > (int64_t)1 << 40)) return invalid(stride_msg);
  if (misaligned(p, size_of(dtype))) return invalid("a pointer is not aligned to its element");
  return SFFN_OK;
}

// Rows of bytes in device memory: `rows` of `width`, `pitch` apart (from one block: one row).
struct Rows {
  uintptr_t at;
  uint64_t rows, pitch, width;
};
Rows block(const void* p, uint64_t bytes) { return Rows{reinterpret_cast<uintptr_t>(p), 1, 0, bytes}; }
// A [rows, d] matrix; rows that follow one another without a gap are one block.
Rows matrix(const void* p, int64_t stride, int64_t rows, int64_t d, size_t size) {
  if (rows <= 1 || stride == d) return block(p, (uint64_t)rows * d * size);
  return Rows{reinterpret_cast<uintptr_t>(p), (uint64_t)rows, stride * size, d * size};
}
// Whether a block of memory meets any of the rows (neither is there if its address is NULL).
bool overlap(const Rows& out, const Rows& r) {
  if (!out.at || !r.at || !out.width || !r.width) return false;
  const uintptr_t end = out.at + out.width;
  if (end <= r.at) return false;
  uint64_t i = 0;  // the first row that ends past the block's start
  if (out.at >= r.at + r.width) {
    if (r.rows == 1) return false;
    i = (out.at - r.at - r.width) / r.pitch + 1;
  }
  return i < r.rows && r.at + i * r.pitch < end;
}
// Refuses outputs (blocks) that overlap an input or each other.
template <size_t N, size_t M>
sffn_status_t check_overlap(const Rows (&out)[N], const Rows (&in)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (const Rows& r : in)
      if (overlap(out[i], r)) return invalid("an output overlaps an input");
    for (size_t j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return invalid("two outputs overlap");
  }
  return SFFN_OK;
}

sffn_status_t norm(int32_t dtype, int32_t gain_dtype, const void* x, int64_t x_stride,
                   const void* residual, int64_t residual_stride, const void* gain, float eps,
                   int64_t rows, int32_t d, void* y, float* stat, void* h, bool fp8,
                   void* stream) {
  OPS_TRY(check_types(dtype, gain_dtype));
  OPS_TRY(check_rows(rows, d));
  if (!(eps >= 0.f)) return invalid("eps must not be negative");
  if (h && !residual) return invalid("h without a residual");
  if (rows == 0) return SFFN_OK;
  OPS_TRY(check_matrix(x, x_stride, rows, d, dtype, "x is NULL", "x_stride is less than d"));
  if (residual)
    OPS_TRY(check_matrix(residual, residual_stride, rows, d, dtype, "residual is NULL",
                         "residual_stride is less than d"));
  if (!gain || !y) return invalid("gain or the output is NULL");
  if (fp8 && !stat) return invalid("scale is NULL");
  if (misaligned(gain, size_of(gain_dtype)) || misaligned(y, fp8 ? 1 : size_of(dtype)) ||
      misaligned(h, size_of(dtype)) || misaligned(stat, 4))
    return invalid("a pointer is not aligned to its element");
  const size_t size = size_of(dtype);
  const Rows xr = matrix(x, x_stride, rows, d, size),
             rr = matrix(residual, residual_stride, rows, d, size),
             yr = block(y, (uint64_t)rows * d * (fp8 ? 1 : size)),
             hr = block(h, (uint64_t)rows * d * size),
             sr = block(stat, (uint64_t)rows * 4);
  // a row is in registers before any of it is written, so that h, and y of the same type, may take
  // the place of x or the residual
  const Rows none = block(nullptr, 0), gr = block(gain, (uint64_t)d * size_of(gain_dtype));
  const auto in_place = [](const Rows& o, const Rows& i) {
    return o.at == i.at && o.width == i.width && i.rows == 1;
  };
  for (const Rows* i : {&xr, &rr}) {
    OPS_TRY(check_overlap({hr}, {in_place(hr, *i) ? none : *i}));
    OPS_TRY(check_overlap({yr}, {!fp8 && in_place(yr, *i) ? none : *i}));
  }
  OPS_TRY(check_overlap({yr, hr, sr}, {gr}));
  OPS_TRY(check_overlap({sr}, {xr, rr}));
  const NormArgs a{x, x_stride, residual, residual ? residual_stride : 0, gain, eps, rows, d, y, stat, h};
  auto f = [&] {
    return launch_rms_norm(dtype == SFFN_BF16, gain_dtype == SFFN_F32, fp8, a,
                           static_cast<hipStream_t>(stream));
  };
  return api_run(fp8 ? "rms_norm_fp8" : "rms_norm", static_cast<hipStream_t>(stream), f);
}

sffn_status_t check_mx4(int32_t N, int32_t K) {
  if (N < 0) return invalid("N must not be negative");
  if (K < 1) return invalid("K must be positive");
  if (K > 1 << 30) return unsupported("K must be at most 2^30");
  if (N > 1 << 26) return unsupported("N must be at most 2^26");  // 2^32 threads a launch
  const Mx4Dims d = mx4_dims(N, K);
  if ((int64_t)d.nb * d.kb >= (int64_t)1 << 25) return unsupported("N * K must be below 2^36");
  return SFFN_OK;
}

}  // namespace

extern "C" {

sffn_status_t sffn_rms_norm(int32_t dtype, int32_t gain_dtype, const void* x, int64_t x_stride,
                            const void* residual, int64_t residual_stride, const void* gain,
                            float eps, int64_t rows, int32_t d, void* y, float* rstd, void* h,
                            void* stream) {
  return norm(dtype, gain_dtype, x, x_stride, residual, residual_stride, gain, eps, rows, d, y,
              rstd, h, false, stream);
}

sffn_status_t sffn_rms_norm_fp8(int32_t dtype, int32_t gain_dtype, const void* x, int64_t x_stride,
                                const void* residual, int64_t residual_stride, const void* gain,
                                float eps, int64_t rows, int32_t d, void* q, float* scale, void* h,
                                void* stream) {
  return norm(dtype, gain_dtype, x, x_stride, residual, residual_stride, gain, eps, rows, d, q,
              scale, h, true, stream);
}

sffn_status_t sffn_rms_norm_backward_workspace(int64_t rows, int32_t d, size_t* bytes) {
  OPS_TRY(check_rows(rows, d));
  if (!bytes) return invalid("bytes is NULL");
  *bytes = (size_t)norm_grad_groups(rows, d) * d * sizeof(float);
  return SFFN_OK;
}

sffn_status_t sffn_rms_norm_backward(int32_t dtype, int32_t gain_dtype, const void* dy,
                                     int64_t dy_stride, const void* h, int64_t h_stride,
                                     const void* gain, const float* rstd, const void* dres,
                                     int64_t dres_stride, int64_t rows, int32_t d, void* dx,
                                     float* dgain, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  OPS_TRY(check_types(dtype, gain_dtype));
  OPS_TRY(check_rows(rows, d));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int groups = norm_grad_groups(rows, d);
  float* part = static_cast<float*>(workspace);
  if (misaligned(dgain, 4)) return invalid("a pointer is not aligned to its element");
  if (rows > 0) {
    OPS_TRY(check_matrix(dy, dy_stride, rows, d, dtype, "dy is NULL", "dy_stride is less than d"));
    OPS_TRY(check_matrix(h, h_stride, rows, d, dtype, "h is NULL", "h_stride is less than d"));
    if (dres)
      OPS_TRY(check_matrix(dres, dres_stride, rows, d, dtype, "dres is NULL",
                           "dres_stride is less than d"));
    if (!gain || !rstd || !dx) return invalid("gain, rstd or dx is NULL");
    if (misaligned(gain, size_of(gain_dtype)) || misaligned(rstd, 4) ||
        misaligned(dx, size_of(dtype)))
      return invalid("a pointer is not aligned to its element");
    if (dgain && groups > 0 && (!workspace || misaligned(workspace, 16) ||
                                workspace_bytes < (size_t)groups * d * sizeof(float)))
      return invalid("workspace is NULL, misaligned or too small");
    const size_t size = size_of(dtype);
    const Rows dxr = block(dx, (uint64_t)rows * d * size), dgr = block(dgain, (uint64_t)d * 4),
               wr = block(dgain && groups > 0 ? workspace : nullptr, (uint64_t)groups * d * 4),
               dyr = matrix(dy, dy_stride, rows, d, size), hr = matrix(h, h_stride, rows, d, size),
               gr = block(gain, (uint64_t)d * size_of(gain_dtype)),
               sr = block(rstd, (uint64_t)rows * 4),
               rr = matrix(dres, dres_stride, rows, d, size);
    OPS_TRY(check_overlap({dxr, dgr, wr}, {dyr, hr, gr, sr}));
    OPS_TRY(check_overlap({dgr, wr}, {rr}));
    if (dx != dres || rr.rows > 1) OPS_TRY(check_overlap({dxr}, {rr}));
    const NormGradArgs a{dy, dy_stride, h, h_stride, gain, rstd, dres, dres ? dres_stride : 0,
                         rows, d, dx, dgain, dgain && groups > 0 ? part : nullptr};
    auto f = [&] { return launch_rms_norm_grad(dtype == SFFN_BF16, gain_dtype == SFFN_F32, a, s); };
    OPS_TRY(api_run("rms_norm_grad", s, f));
  }
  if (!dgain || (rows > 0 && groups == 0)) return SFFN_OK;
  auto f = [&] { return launch_rms_norm_grad_sum(part, groups, d, dgain, s); };
  return api_run("rms_norm_grad_sum", s, f);
}

sffn_status_t sffn_mx4_quantize(int32_t dtype, const void* W, int64_t w_stride, int32_t N,
                                int32_t K, uint8_t* codes, uint8_t* scales, void* stream) {
  if (dtype != SFFN_F32 && dtype != SFFN_BF16) return invalid("dtype must be SFFN_F32 or SFFN_BF16");
  OPS_TRY(check_mx4(N, K));
  if (N == 0) return SFFN_OK;
  OPS_TRY(check_matrix(W, w_stride, N, K, dtype, "W is NULL", "w_stride is less than K"));
  if (!codes || !scales) return invalid("codes or scales is NULL");
  const uint64_t groups = (uint64_t)N * ((K + 31) / 32);
  OPS_TRY(check_overlap({block(codes, groups * 16), block(scales, groups)},
                        {matrix(W, w_stride, N, K, size_of(dtype))}));
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto f = [&] { return launch_mx4_quantize(dtype == SFFN_BF16, W, w_stride, N, K, codes, scales, s); };
  return api_run("mx4_quantize", s, f);
}

sffn_status_t sffn_mx4_bytes(int32_t N, int32_t K, size_t* bytes) {
  OPS_TRY(check_mx4(N, K));
  if (!bytes) return invalid("bytes is NULL");
  *bytes = mx4_dims(N, K).bytes();
  return SFFN_OK;
}

sffn_status_t sffn_mx4_tile(const uint8_t* codes, const uint8_t* scales, int32_t N, int32_t K,
                            void* tiled, void* stream) {
  OPS_TRY(check_mx4(N, K));
  if (N == 0) return SFFN_OK;
  if (!codes || !scales || !tiled) return invalid("codes, scales or tiled is NULL");
  if (misaligned(tiled, 16)) return invalid("tiled must be 16-byte aligned");
  const uint64_t groups = (uint64_t)N * ((K + 31) / 32);
  OPS_TRY(check_overlap({block(tiled, mx4_dims(N, K).bytes())},
                        {block(codes, groups * 16), block(scales, groups)}));
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto f = [&] { return launch_mx4_tile(codes, scales, mx4_dims(N, K), tiled, s); };
  return api_run("mx4_tile", s, f);
}

sffn_status_t sffn_mx4_linear(const void* tiled, int32_t N, int32_t K, int32_t x_dtype,
                              const void* x, int64_t x_stride, const float* x_scale, int32_t T,
                              const float* bias, int32_t relu, int32_t y_dtype, void* y,
                              void* stream) {
  OPS_TRY(check_mx4(N, K));
  if (x_dtype != SFFN_F32 && x_dtype != SFFN_BF16 && x_dtype != SFFN_E4M3)
    return invalid("x_dtype must be SFFN_F32, SFFN_BF16 or SFFN_E4M3");
  if (y_dtype != SFFN_F32 && y_dtype != SFFN_BF16)
    return invalid("y_dtype must be SFFN_F32 or SFFN_BF16");
  if (T < 0) return invalid("T must not be negative");
  if (T > 1 << 20) return unsupported("T must be at most 2^20");
  if (x_dtype == SFFN_E4M3 && !x_scale) return invalid("x_scale is NULL");
  if (T == 0 || N == 0) return SFFN_OK;
  OPS_TRY(check_matrix(x, x_stride, T, K, x_dtype, "x is NULL", "x_stride is less than K"));
  if (!tiled || !y) return invalid("tiled or y is NULL");
  if (misaligned(tiled, 16)) return invalid("tiled must be 16-byte aligned");
  if (misaligned(y, size_of(y_dtype)) || misaligned(x_scale, 4) || misaligned(bias, 4))
    return invalid("a pointer is not aligned to its element");
  OPS_TRY(check_overlap({block(y, (uint64_t)T * N * size_of(y_dtype))},
                        {block(tiled, mx4_dims(N, K).bytes()),
                         matrix(x, x_stride, T, K, size_of(x_dtype)),
                         block(x_scale, (uint64_t)T * 4), block(bias, (uint64_t)N * 4)}));
  const Mx4Args a{tiled, mx4_dims(N, K), x_dtype, x, x_stride, x_scale, T, bias, relu != 0,
                  y_dtype == SFFN_BF16, y};
  auto f = [&] { return launch_mx4_linear(a, static_cast<hipStream_t>(stream)); };
  return api_run("mx4_linear", static_cast<hipStream_t>(stream), f);
}

sffn_status_t sffn_adamw_step(const sffn_adamw_tensor_t* tensors, int32_t n_tensors,
                              int32_t param_dtype, int32_t grad_dtype, int32_t state_bits,
                              const sffn_adamw_hyper_t* hyper, const float* grad_scale,
                              void* stream) {
  if (n_tensors < 0 || (n_tensors > 0 && !tensors)) return invalid("tensors is NULL or its count negative");
  if (!hyper) return invalid("hyper is NULL");
  if (param_dtype != SFFN_F32 && param_dtype != SFFN_BF16)
    return invalid("param_dtype must be SFFN_F32 or SFFN_BF16");
  if (grad_dtype != SFFN_F32 && grad_dtype != SFFN_BF16)
    return invalid("grad_dtype must be SFFN_F32 or SFFN_BF16");
  if (state_bits != 8 && state_bits != 32) return invalid("state_bits must be 8 or 32");
  const sffn_adamw_hyper_t& hp = *hyper;
  if (!(hp.beta1 >= 0.0 && hp.beta1 < 1.0 && hp.beta2 >= 0.0 && hp.beta2 < 1.0))
    return invalid("beta1 and beta2 must be in [0, 1)");
  if (!(hp.eps >= 0.0) || !(hp.weight_decay >= 0.0) || !std::isfinite(hp.lr))
    return invalid("eps and weight_decay must not be negative, lr must be finite");
  if (hp.step < 1) return invalid("step must be at least 1");
  if (misaligned(grad_scale, 4)) return invalid("a pointer is not aligned to its element");
  const size_t pa = size_of(param_dtype), ga = size_of(grad_dtype), sa = state_bits == 8 ? 1 : 4;
  bool master = false, first = true;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const sffn_adamw_tensor_t& t = tensors[i];
    if (t.n < 0 || t.n > (int64_t)1 << 40) return invalid("n of a tensor must be in [0, 2^40]");
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v) return invalid("a tensor's pointer is NULL");
    if (state_bits == 8 && (!t.m_scale || !t.v_scale)) return invalid("a tensor's scales are NULL");
    if (t.master && param_dtype != SFFN_BF16) return invalid("a master copy needs SFFN_BF16 parameters");
    if (!first && (t.master != nullptr) != master)
      return invalid("either all tensors have a master copy or none");
    master = t.master != nullptr;
    first = false;
    if (misaligned(t.param, pa) || misaligned(t.grad, ga) || misaligned(t.m, sa) ||
        misaligned(t.v, sa) || misaligned(t.master, 4) || misaligned(t.m_scale, 4) ||
        misaligned(t.v_scale, 4))
      return invalid("a pointer is not aligned to its element");
    const uint64_t n = (uint64_t)t.n, blocks = (n + SFFN_ADAMW_BLOCK - 1) / SFFN_ADAMW_BLOCK,
                   scales = state_bits == 8 ? blocks * 4 : 0;
    OPS_TRY(check_overlap({block(t.param, n * pa), block(t.master, n * 4), block(t.m, n * sa),
                           block(t.v, n * sa), block(t.m_scale, scales), block(t.v_scale, scales)},
                          {block(t.grad, n * ga)}));
  }
  // Complements and powers in double: in fp32, 1 - beta2 would lose the digits of a small
  // difference.
  AdamwTable tab;
  std::memset(&tab, 0, sizeof(tab));
  tab.lr_decay = (float)(hp.lr * hp.weight_decay);
  tab.beta1 = (float)hp.beta1;
  tab.one_minus_beta1 = (float)(1.0 - hp.beta1);
  tab.beta2 = (float)hp.beta2;
  tab.one_minus_beta2 = (float)(1.0 - hp.beta2);
  tab.step_size = (float)(hp.lr / (1.0 - std::pow(hp.beta1, (double)hp.step)));
  tab.inv_root_correction = (float)(1.0 / std::sqrt(1.0 - std::pow(hp.beta2, (double)hp.step)));
  tab.eps = (float)hp.eps;
  tab.grad_scale = grad_scale;
  // A launch takes up to ADAMW_TENSORS tensors and MAX_GROUPS workgroups (half of the 2^32
  // threads that a launch must stay below); a longer tensor is cut into parts of whole chunks.
  constexpr int64_t MAX_GROUPS = ((int64_t)1 << 31) / (ADAMW_CHUNK / 4);
  hipStream_t s = static_cast<hipStream_t>(stream);
  int used = 0;
  int64_t groups = 0;
  auto flush = [&]() -> sffn_status_t {
    if (used == 0) return SFFN_OK;
    for (int i = used; i < ADAMW_TENSORS; ++i) tab.first[i] = 0xffffffffu;
    auto f = [&] {
      return launch_adamw(param_dtype == SFFN_BF16, grad_dtype == SFFN_BF16, master, state_bits,
                          tab, (uint32_t)groups, s);
    };
    const sffn_status_t st = api_run("adamw", s, f);
    used = 0;
    groups = 0;
    return st;
  };
  for (int32_t i = 0; i < n_tensors; ++i) {
    int64_t at = 0;
    while (at < tensors[i].n) {
      if (used == ADAMW_TENSORS || groups == MAX_GROUPS) OPS_TRY(flush());
      const int64_t room = (MAX_GROUPS - groups) * ADAMW_CHUNK;
      sffn_adamw_tensor_t t = tensors[i];
      const int64_t n = t.n - at < room ? t.n - at : room;
      t.param = static_cast<char*>(t.param) + at * (int64_t)pa;
      t.grad = static_cast<const char*>(t.grad) + at * (int64_t)ga;
      if (t.master) t.master += at;
      t.m = static_cast<char*>(t.m) + at * (int64_t)sa;
      t.v = static_cast<char*>(t.v) + at * (int64_t)sa;
      if (t.m_scale) t.m_scale += at / SFFN_ADAMW_BLOCK;
      if (t.v_scale) t.v_scale += at / SFFN_ADAMW_BLOCK;
      t.n = n;
      tab.t[used] = t;
      tab.first[used++] = (uint32_t)groups;
      groups += (n + ADAMW_CHUNK - 1) / ADAMW_CHUNK;
      at += n;
    }
  }
  return flush();
}

}  // extern "C"
