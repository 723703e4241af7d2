// C entry points of the RMS norm, the e4m3 block quantizers, the 8-bit linear and the
// linear grouped by expert: host-side validation and launches.
#include <cuda_runtime.h>

#include "block8.cuh"
#include "expert_gemm.cuh"
#include "internal.cuh"

using namespace qlb;

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline cudaStream_t S(qlora_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

#define QLB_TRY(x)                         \
  do {                                     \
    qlora_status _st = (x);                \
    if (_st != QLORA_OK) return _st;       \
  } while (0)

qlora_status device_ok() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return QLORA_ERR_CUDA;
  return qlora_device_check(dev);
}

// Rows of activations and sides of a weight: TMA and the index arithmetic of the
// kernels hold for these.
constexpr int64_t kMaxSide = int64_t(1) << 24;
constexpr int64_t kMaxRows = int64_t(1) << 30;

bool side_ok(int64_t n) { return n > 0 && n <= kMaxSide && n % 16 == 0; }

qlora_status check_expert_weight(const qlora_expert_weight* w) {
  if (!w) return QLORA_ERR_NULL;
  if (w->experts < 1 || w->experts > kMaxExperts || !side_ok(w->out) || !side_ok(w->in)) return QLORA_ERR_SHAPE;
  if (w->is_bf16 != 0 && w->is_bf16 != 1) return QLORA_ERR_DTYPE;
  if (w->is_bf16) {
    if (!w->w_bf16) return QLORA_ERR_NULL;
    if (!aligned16(w->w_bf16)) return QLORA_ERR_ALIGN;
  } else {
    if (!w->codes || !w->scale) return QLORA_ERR_NULL;
    if (!aligned16(w->codes) || !aligned4(w->scale)) return QLORA_ERR_ALIGN;
  }
  return QLORA_OK;
}

qlora_status check_status_ws(const void* ws, size_t bytes) {
  return (!ws || !aligned16(ws) || bytes < kStatusBytes) ? QLORA_ERR_WORKSPACE : QLORA_OK;
}

// One product of rows `a` (bf16, or codes with scales `sa`) with the experts' weights.
qlora_status check_rows(const qlora_expert_weight* w, const void* a, const float* sa, int64_t M,
                        bool may_be_bf16 = false) {
  if (M <= 0 || M > kMaxRows) return QLORA_ERR_SHAPE;
  if (!a) return QLORA_ERR_NULL;
  if (!aligned16(a)) return QLORA_ERR_ALIGN;
  if (!w->is_bf16) {
    if (!sa && !(may_be_bf16 && M <= kFewQuantRows)) return QLORA_ERR_NULL;
    if (!aligned4(sa)) return QLORA_ERR_ALIGN;
  }
  return QLORA_OK;
}

qlora_status product(ExpertMode mode, const qlora_expert_weight* w, const void* a, const float* sa, int64_t M,
                     const int32_t* offsets, uint16_t* d, void* ws, qlora_stream_t stream) {
  ExpertArgs e = {};
  e.mode = mode;
  e.f8 = !w->is_bf16;
  e.M = M;
  e.E = w->experts;
  e.out = w->out;
  e.in = w->in;
  e.offsets = offsets;
  e.a = a;
  e.b = w->is_bf16 ? static_cast<const void*>(w->w_bf16) : w->codes;
  e.sa = sa;
  e.sb = w->scale;
  e.d = d;
  e.status = static_cast<int*>(ws);
  if (e.f8 && !sa) return launch_few_rows(e, true, S(stream));
  return launch_expert_gemm(e, S(stream));
}

}  // namespace

extern "C" {

qlora_status qlora_rms_norm_fwd(const uint16_t* x, const uint16_t* residual, const void* weight, int32_t w_dtype,
                                int64_t M, int64_t H, float eps, uint16_t* h, uint16_t* y, uint8_t* y_codes,
                                float* y_scale, float* rstd, qlora_stream_t stream) {
  if (w_dtype != QLORA_DTYPE_BF16 && w_dtype != QLORA_DTYPE_F32) return QLORA_ERR_DTYPE;
  if (M <= 0 || M > kMaxRows || H <= 0 || H > kMaxNormHidden || H % 8) return QLORA_ERR_SHAPE;
  if (!(eps >= 0.f)) return QLORA_ERR_UNSUPPORTED;
  if (!x || !weight || !rstd || (residual && !h) || (!y && !y_codes) || (y_codes && !y_scale)) return QLORA_ERR_NULL;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(h) || !aligned16(y) ||
      !aligned16(y_codes) || !aligned4(y_scale) || !aligned4(rstd))
    return QLORA_ERR_ALIGN;
  QLB_TRY(device_ok());
  NormFwd a = {x, residual, weight, w_dtype == QLORA_DTYPE_F32, M, H, eps, h, y, y_codes, y_scale, rstd};
  return launch_rms_norm_fwd(a, S(stream));
}

size_t qlora_rms_norm_bwd_workspace_size(int64_t M, int64_t H) {
  if (M <= 0 || M > kMaxRows || H <= 0 || H > kMaxNormHidden || H % 8) return 0;
  return size_t(norm_bwd_parts(M, H)) * size_t(H) * sizeof(float);
}

qlora_status qlora_rms_norm_bwd(const uint16_t* dy, const uint16_t* dh, const uint16_t* h, const float* rstd,
                                const void* weight, int32_t w_dtype, int64_t M, int64_t H, uint16_t* dx, float* dw,
                                void* workspace, size_t workspace_bytes, qlora_stream_t stream) {
  if (w_dtype != QLORA_DTYPE_BF16 && w_dtype != QLORA_DTYPE_F32) return QLORA_ERR_DTYPE;
  if (M <= 0 || M > kMaxRows || H <= 0 || H > kMaxNormHidden || H % 8) return QLORA_ERR_SHAPE;
  if (!dy || !h || !rstd || !weight || !dx) return QLORA_ERR_NULL;
  if (!aligned16(dy) || !aligned16(dh) || !aligned16(h) || !aligned4(rstd) || !aligned16(weight) || !aligned16(dx) ||
      !aligned16(dw))
    return QLORA_ERR_ALIGN;
  if (dw && (!workspace || !aligned16(workspace) || workspace_bytes < qlora_rms_norm_bwd_workspace_size(M, H)))
    return QLORA_ERR_WORKSPACE;
  QLB_TRY(device_ok());
  NormBwd a = {dy, dh, h, rstd, weight, w_dtype == QLORA_DTYPE_F32, M, H, dx, dw, static_cast<float*>(workspace)};
  return launch_rms_norm_bwd(a, S(stream));
}

qlora_status fp8_quantize_rows(const uint16_t* X, int64_t M, int64_t in, uint8_t* codes, float* scale,
                               qlora_stream_t stream) {
  if (M <= 0 || M > kMaxRows || !side_ok(in)) return QLORA_ERR_SHAPE;
  if (!X || !codes || !scale) return QLORA_ERR_NULL;
  if (!aligned16(X) || !aligned16(codes) || !aligned4(scale)) return QLORA_ERR_ALIGN;
  QLB_TRY(device_ok());
  return launch_quantize_rows8(X, M, in, codes, scale, S(stream));
}

qlora_status fp8_quantize_weight(const void* W, int32_t w_dtype, int64_t experts, int64_t out, int64_t in,
                                 uint8_t* codes, float* scale, void* workspace, size_t workspace_bytes,
                                 qlora_stream_t stream) {
  if (w_dtype != QLORA_DTYPE_BF16 && w_dtype != QLORA_DTYPE_F32) return QLORA_ERR_DTYPE;
  if (experts < 1 || experts > kMaxExperts || !side_ok(out) || !side_ok(in)) return QLORA_ERR_SHAPE;
  if (!W || !codes || !scale) return QLORA_ERR_NULL;
  if (!aligned16(W) || !aligned16(codes) || !aligned4(scale)) return QLORA_ERR_ALIGN;
  QLB_TRY(check_status_ws(workspace, workspace_bytes));
  QLB_TRY(device_ok());
  return launch_quantize_weight8(W, w_dtype == QLORA_DTYPE_F32, experts, out, in, codes, scale,
                                 static_cast<int*>(workspace), S(stream));
}

size_t qlora_expert_workspace_size(void) { return kStatusBytes; }

int64_t fp8_linear_bf16_rows(void) { return kFewQuantRows; }

static qlora_status fp8_linear(bool fwd, const qlora_expert_weight* w, const void* rows, const float* scale,
                               int64_t M, uint16_t* d, void* ws, size_t ws_bytes, qlora_stream_t stream) {
  QLB_TRY(check_expert_weight(w));
  if (w->is_bf16) return QLORA_ERR_UNSUPPORTED;
  if (w->experts != 1) return QLORA_ERR_SHAPE;
  QLB_TRY(check_rows(w, rows, scale, M, fwd));
  if (!d) return QLORA_ERR_NULL;
  if (!aligned16(d)) return QLORA_ERR_ALIGN;
  QLB_TRY(check_status_ws(ws, ws_bytes));
  QLB_TRY(device_ok());
  return product(fwd ? ExpertMode::Fwd : ExpertMode::Dx, w, rows, scale, M, nullptr, d, ws, stream);
}

qlora_status fp8_linear_fwd(const qlora_expert_weight* w, const void* X, const float* x_scale, int64_t M,
                            uint16_t* Y, void* workspace, size_t workspace_bytes, qlora_stream_t stream) {
  return fp8_linear(true, w, X, x_scale, M, Y, workspace, workspace_bytes, stream);
}

qlora_status fp8_linear_bwd(const qlora_expert_weight* w, const uint8_t* dy_codes, const float* dy_scale, int64_t M,
                            uint16_t* dX, void* workspace, size_t workspace_bytes, qlora_stream_t stream) {
  return fp8_linear(false, w, dy_codes, dy_scale, M, dX, workspace, workspace_bytes, stream);
}

qlora_status qlora_grouped_linear_fwd(const qlora_expert_weight* w, const void* X, const float* x_scale, int64_t M,
                                      const int32_t* offsets, uint16_t* Y, void* workspace, size_t workspace_bytes,
                                      qlora_stream_t stream) {
  QLB_TRY(check_expert_weight(w));
  QLB_TRY(check_rows(w, X, x_scale, M));
  if (!offsets || !Y) return QLORA_ERR_NULL;
  if (!aligned4(offsets) || !aligned16(Y)) return QLORA_ERR_ALIGN;
  QLB_TRY(check_status_ws(workspace, workspace_bytes));
  QLB_TRY(device_ok());
  return product(ExpertMode::Fwd, w, X, x_scale, M, offsets, Y, workspace, stream);
}

qlora_status qlora_grouped_linear_bwd(const qlora_expert_weight* w, const uint16_t* X, const void* dY,
                                      const float* dy_scale, int64_t M, const int32_t* offsets, uint16_t* dX,
                                      float* dW, void* workspace, size_t workspace_bytes, qlora_stream_t stream) {
  QLB_TRY(check_expert_weight(w));
  if (dW && !w->is_bf16) return QLORA_ERR_UNSUPPORTED;
  QLB_TRY(check_rows(w, dY, dy_scale, M));
  if (!offsets || (!dX && !dW) || (dW && !X)) return QLORA_ERR_NULL;
  if (!aligned4(offsets) || !aligned16(dX) || !aligned16(dW) || !aligned16(X)) return QLORA_ERR_ALIGN;
  QLB_TRY(check_status_ws(workspace, workspace_bytes));
  QLB_TRY(device_ok());
  if (dX) QLB_TRY(product(ExpertMode::Dx, w, dY, dy_scale, M, offsets, dX, workspace, stream));
  if (dW) {
    ExpertArgs e = {};
    e.mode = ExpertMode::Dw;
    e.M = M;
    e.E = w->experts;
    e.out = w->out;
    e.in = w->in;
    e.offsets = offsets;
    e.a = dY;
    e.b = X;
    e.d = dW;
    e.status = static_cast<int*>(workspace);
    QLB_TRY(launch_expert_gemm(e, S(stream)));
  }
  return QLORA_OK;
}

}  // extern "C"
