// norm.h - launchers of layer norm and dropout (norm.cu, norm_bwd.cu).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace sta {

constexpr int32_t kNormMaxCols = 8192;

struct NormDropout {
  const int64_t* rng;   // seed, offset on the device; null when thr is 0
  uint32_t thr;         // round(65536 p)
  float scale;          // 65536 / (65536 - thr), 0 when thr is 65536
};

// dtype codes of sta.h: 0 bf16, 1 fp16, 2 fp32; wfp32: weight and bias are fp32 (else dtype).
struct NormFwdArgs {
  const void *x, *residual, *weight, *bias;
  void *y, *h;
  float *mean, *rstd;
  int64_t rows;
  int32_t cols;
  float n, inv_n;   // cols and 1 / cols: operands from the parameters take no registers
  float eps;
  bool wfp32;
  NormDropout drop;
};

struct NormBwdArgs {
  const void *dy, *h, *weight, *dh;
  const float *mean, *rstd;
  void *dx, *dres, *dweight, *dbias;
  float* partial;       // workspace: [2][parts][cols]
  int64_t rows;
  int32_t cols;
  bool wfp32;
  NormDropout drop;
};

cudaError_t launch_norm_fwd(int dtype, const NormFwdArgs& a, cudaStream_t stream);

// Upper bound of the parts of norm_bwd's column sums, whatever the device's SM count.
int norm_bwd_parts(int64_t rows, int32_t cols);
cudaError_t launch_norm_bwd(int dtype, const NormBwdArgs& a, cudaStream_t stream);

cudaError_t launch_dropout(int dtype, const void* x, void* y, int64_t rows, int32_t cols, const NormDropout& drop,
                           cudaStream_t stream);

}  // namespace sta
