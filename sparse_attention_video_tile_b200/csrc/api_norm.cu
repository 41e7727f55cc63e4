// api_norm.cu - the C entry points of layer norm and dropout (include/sta.h):
// argument checks, then one or two kernel launches on the caller's stream.
#include <cmath>

#include "checks.h"
#include "internal.h"
#include "norm.h"

namespace sta {
namespace {

int64_t dtype_size(int32_t dtype) { return dtype == STA_FP32 ? 4 : 2; }

sta_status check_shape(int64_t rows, int32_t cols, int32_t dtype) {
  if (dtype != STA_BF16 && dtype != STA_FP16 && dtype != STA_FP32) return STA_ERR_ARG;
  if (rows < 0 || cols < 1) return STA_ERR_SHAPE;
  // flat element numbers and byte offsets stay far inside 63 bits, grids inside 31
  if (rows > (int64_t(1) << 40) / cols) return STA_ERR_SHAPE;
  return STA_OK;
}

sta_status make_dropout(float p, const int64_t* rng, NormDropout* d) {
  if (!(p >= 0.f && p <= 1.f)) return STA_ERR_ARG;   // NaN fails both
  d->thr = static_cast<uint32_t>(std::floor(static_cast<double>(p) * 65536.0 + 0.5));
  d->scale = d->thr < 65536 ? static_cast<float>(65536.0 / (65536.0 - d->thr)) : 0.f;
  d->rng = rng;
  if (d->thr > 0 && !rng) return STA_ERR_NULL;
  if (!aligned_to(rng, 8)) return STA_ERR_ALIGN;
  return STA_OK;
}

sta_status finish(cudaError_t e) { return e == cudaSuccess ? STA_OK : cuda_fail(e); }

}  // namespace
}  // namespace sta

using namespace sta;

extern "C" {

sta_status sta_layer_norm_fwd(const void* x, const void* residual, const void* weight, const void* bias, void* y,
                              void* h, float* mean, float* rstd, int64_t rows, int32_t cols, int32_t dtype,
                              int32_t param_dtype, float eps, float dropout_p, const int64_t* rng, void* stream) {
  sta_status s = check_shape(rows, cols, dtype);
  if (s != STA_OK) return s;
  if (cols > kNormMaxCols) return STA_ERR_SHAPE;
  if (param_dtype != dtype && param_dtype != STA_FP32) return STA_ERR_ARG;
  if (!(eps >= 0.f) || std::isinf(eps)) return STA_ERR_ARG;
  if (rows > 0 && (!x || !y)) return STA_ERR_NULL;
  NormFwdArgs a{};
  if ((s = make_dropout(dropout_p, rng, &a.drop)) != STA_OK) return s;
  for (const void* p : {x, residual, weight, bias, static_cast<const void*>(y), static_cast<const void*>(h)})
    if (!aligned_to(p, 16)) return STA_ERR_ALIGN;
  if (!aligned_to(mean, 4) || !aligned_to(rstd, 4)) return STA_ERR_ALIGN;
  const int64_t n = rows * cols * dtype_size(dtype), np = cols * dtype_size(param_dtype);
  const Range r[] = {{y, n}, {h, n}, {mean, rows * 4}, {rstd, rows * 4}, {x, n}, {residual, n}, {weight, np}, {bias, np},
                     {rng, 16}};
  if (any_overlap(r, 4, 9)) return STA_ERR_ALIAS;
  if ((s = check_device(nullptr)) != STA_OK) return s;
  a.x = x; a.residual = residual; a.weight = weight; a.bias = bias;
  a.y = y; a.h = h; a.mean = mean; a.rstd = rstd;
  a.rows = rows; a.cols = cols; a.eps = eps;
  a.n = static_cast<float>(cols); a.inv_n = 1.0f / a.n;
  a.wfp32 = param_dtype == STA_FP32;
  return finish(launch_norm_fwd(dtype, a, static_cast<cudaStream_t>(stream)));
}

int64_t sta_layer_norm_bwd_workspace(int64_t rows, int32_t cols) {
  if (check_shape(rows, cols, STA_FP32) != STA_OK || cols > kNormMaxCols) return -1;
  const int64_t bytes = 2 * static_cast<int64_t>(norm_bwd_parts(rows, cols)) * cols * 4;
  return (bytes + 255) / 256 * 256;
}

sta_status sta_layer_norm_bwd(const void* dy, const void* h, const float* mean, const float* rstd, const void* weight,
                              const void* dh, void* dx, void* dresidual, void* dweight, void* dbias, int64_t rows,
                              int32_t cols, int32_t dtype, int32_t param_dtype, float dropout_p, const int64_t* rng,
                              void* workspace, int64_t workspace_bytes, void* stream) {
  sta_status s = check_shape(rows, cols, dtype);
  if (s != STA_OK) return s;
  if (cols > kNormMaxCols) return STA_ERR_SHAPE;
  if (param_dtype != dtype && param_dtype != STA_FP32) return STA_ERR_ARG;
  if (rows > 0 && (!dy || !h || !mean || !rstd || (!dx && !dresidual))) return STA_ERR_NULL;
  NormBwdArgs a{};
  if ((s = make_dropout(dropout_p, rng, &a.drop)) != STA_OK) return s;
  for (const void* p : {dy, h, weight, dh, static_cast<const void*>(dx), static_cast<const void*>(dresidual),
                        static_cast<const void*>(dweight), static_cast<const void*>(dbias),
                        static_cast<const void*>(workspace)})
    if (!aligned_to(p, 16)) return STA_ERR_ALIGN;
  if (!aligned_to(mean, 4) || !aligned_to(rstd, 4)) return STA_ERR_ALIGN;
  const bool sums = dweight != nullptr || dbias != nullptr;
  const int64_t need = sums ? sta_layer_norm_bwd_workspace(rows, cols) : 0;
  if (need > 0 && !workspace) return STA_ERR_NULL;
  if (need > 0 && workspace_bytes < need) return STA_ERR_SCRATCH;
  const int64_t n = rows * cols * dtype_size(dtype), np = cols * dtype_size(param_dtype);
  const Range r[] = {{dx, n}, {dresidual, n}, {dweight, np}, {dbias, np}, {workspace, need}, {dy, n}, {h, n},
                     {mean, rows * 4}, {rstd, rows * 4}, {weight, np}, {dh, n}, {rng, 16}};
  if (any_overlap(r, 5, 12)) return STA_ERR_ALIAS;
  if ((s = check_device(nullptr)) != STA_OK) return s;
  a.dy = dy; a.h = h; a.weight = weight; a.dh = dh; a.mean = mean; a.rstd = rstd;
  a.dx = dx; a.dres = dresidual; a.dweight = dweight; a.dbias = dbias;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  a.rows = rows; a.cols = cols;
  a.wfp32 = param_dtype == STA_FP32;
  return finish(launch_norm_bwd(dtype, a, static_cast<cudaStream_t>(stream)));
}

sta_status sta_dropout(const void* x, void* y, int64_t rows, int32_t cols, int32_t dtype, float dropout_p,
                       const int64_t* rng, void* stream) {
  sta_status s = check_shape(rows, cols, dtype);
  if (s != STA_OK) return s;
  if (rows > 0 && (!x || !y)) return STA_ERR_NULL;
  NormDropout d{};
  if ((s = make_dropout(dropout_p, rng, &d)) != STA_OK) return s;
  if (!aligned_to(x, 16) || !aligned_to(y, 16)) return STA_ERR_ALIGN;
  const int64_t n = rows * cols * dtype_size(dtype);
  const Range r[] = {{y, n}, {x, n}, {rng, 16}};
  if (any_overlap(r, 1, 3)) return STA_ERR_ALIAS;
  if ((s = check_device(nullptr)) != STA_OK) return s;
  return finish(launch_dropout(dtype, x, y, rows, cols, d, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
