// norm.cu - layer norm forward (with an optional dropout and residual sum in front)
// and dropout, for sm_100a.
//
//   h = residual + dropout(x)   (h = x without them)
//   y = (h - mean) rstd w + b,  mean = sum h / n,  rstd = 1 / sqrt(sum (h - mean)^2 / n + eps)
//
// The work is moving bytes: x (and residual) read once, y (and h) written once.  A
// row stays in registers between its load and its store, so the variance is the sum
// of squared differences from the mean, with no cancellation and no second read; all
// sums are fp32.  y is taken from the fp32 h, before h is rounded for its store.
#include "norm_common.cuh"

namespace sta {
namespace {

using namespace norm;

// TPR threads share a row (0: the whole block); each holds CH chunks of R rows.
template <typename T, bool VEC, int TPR, int CH, int R>
__global__ void __launch_bounds__(TPR > 0 ? 256 : 512) norm_fwd_kernel(const NormFwdArgs a) {
  __shared__ float red[32];
  const int lane = TPR > 0 ? static_cast<int>(threadIdx.x) % TPR : static_cast<int>(threadIdx.x);
  const int step = TPR > 0 ? TPR : static_cast<int>(blockDim.x);
  const int64_t group = TPR > 0 ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / TPR) + threadIdx.x / TPR : blockIdx.x;
  const int64_t row0 = group * R;
  const int32_t n8 = (a.cols + 7) >> 3;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  PhiloxKey key{};
  if (a.drop.thr > 0) key = philox_key(a.drop.rng);
  float f[R][CH][8];
  {
    Chunk<T> cx[R][CH], cr[R][CH];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int32_t ch = lane + k * step;
        const int n = VEC ? 8 : min(8, a.cols - ch * 8);
        cx[r][k].clear();
        if (row0 + r < a.rows && ch < n8) {
          const int64_t at = (row0 + r) * a.cols + ch * 8;
          if (VEC) cx[r][k].load(x + at); else cx[r][k].load_n(x + at, n);
        }
      }
    if (res != nullptr) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int32_t ch = lane + k * step;
          const int n = VEC ? 8 : min(8, a.cols - ch * 8);
          cr[r][k].clear();
          if (row0 + r < a.rows && ch < n8) {
            const int64_t at = (row0 + r) * a.cols + ch * 8;
            if (VEC) cr[r][k].load(res + at); else cr[r][k].load_n(res + at, n);
          }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int32_t ch = lane + k * step;
        cx[r][k].get(f[r][k]);
        if (a.drop.thr > 0) {
          // dropped values are replaced, not multiplied by zero: an infinity or NaN there stays out
          const uint32_t keep = philox_keep(philox_block(static_cast<uint64_t>(row0 + r) * n8 + ch, key), a.drop.thr);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[r][k][i] = (keep >> i) & 1u ? f[r][k][i] * a.drop.scale : 0.f;
        }
        if (res != nullptr) {
          float g[8];
          cr[r][k].get(g);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[r][k][i] += g[i];
        }
      }
  }
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  float mean[R], rstd[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += f[r][k][i];   // columns past the row hold zero
    mean[r] = row_sum<TPR>(s, red) * inv_n;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int32_t c0 = (lane + k * step) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = f[r][k][i] - mean[r];
        if (c0 + (VEC ? 0 : i) < a.cols) s = fmaf(e, e, s);
      }
    }
    rstd[r] = 1.0f / sqrtf(fmaf(row_sum<TPR>(s, red), inv_n, a.eps));
  }
  T* y = static_cast<T*>(a.y);
  T* h = static_cast<T*>(a.h);
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int32_t ch = lane + k * step;
    if (ch >= n8) continue;
    const int n = VEC ? 8 : min(8, a.cols - ch * 8);
    float w[8], b[8];
    if (a.weight != nullptr) load_param<T, VEC>(a.weight, a.wfp32, ch * 8, n, w);
    if (a.bias != nullptr) load_param<T, VEC>(a.bias, a.wfp32, ch * 8, n, b);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r >= a.rows) continue;
      const int64_t at = (row0 + r) * a.cols + ch * 8;
      Chunk<T> o;
      if (h != nullptr) {
        o.put(f[r][k]);
        if (VEC) o.store(h + at); else o.store_n(h + at, n);
      }
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = (f[r][k][i] - mean[r]) * rstd[r];
        if (a.weight != nullptr) v[i] *= w[i];
        if (a.bias != nullptr) v[i] += b[i];
      }
      o.put(v);
      if (VEC) o.store(y + at); else o.store_n(y + at, n);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (lane == 0 && row0 + r < a.rows) {
      if (a.mean != nullptr) a.mean[row0 + r] = mean[r];
      if (a.rstd != nullptr) a.rstd[row0 + r] = rstd[r];
    }
}

template <typename T, bool VEC, int TPR, int CH, int R>
cudaError_t launch_fwd(const NormFwdArgs& a, cudaStream_t stream) {
  int threads = 256;
  int64_t blocks;
  if (TPR > 0) {
    const int64_t groups = (a.rows + R - 1) / R, per = threads / TPR;
    blocks = (groups + per - 1) / per;
  } else {
    const int n8 = (a.cols + 7) >> 3;
    threads = ((n8 + CH - 1) / CH + 31) / 32 * 32;
    blocks = (a.rows + R - 1) / R;
  }
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  norm_fwd_kernel<T, VEC, (TPR > 0 ? TPR : 0), CH, R><<<static_cast<unsigned>(blocks), threads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t pick_fwd(const NormFwdArgs& a, cudaStream_t stream) {
  const int n8 = (a.cols + 7) >> 3;
  if (n8 <= 1) return launch_fwd<T, VEC, 1, 1, 2>(a, stream);
  if (n8 <= 4) return launch_fwd<T, VEC, 4, 1, 4>(a, stream);
  if (n8 <= 16) return launch_fwd<T, VEC, 16, 1, 4>(a, stream);
  if (n8 <= 32) return launch_fwd<T, VEC, 32, 1, 4>(a, stream);
  if (n8 <= 64) return launch_fwd<T, VEC, 32, 2, 2>(a, stream);
  if (n8 <= 128) return launch_fwd<T, VEC, 32, 4, 1>(a, stream);
  if (n8 <= 192) return launch_fwd<T, VEC, 32, 6, 1>(a, stream);
  if (n8 <= 1024) return launch_fwd<T, VEC, 0, 2, 1>(a, stream);
  return launch_fwd<T, VEC, 0, 4, 1>(a, stream);
}

// Dropout, rows of a multiple of eight columns: chunk i of the flat array is counter block i.
template <typename T>
__global__ void __launch_bounds__(256) dropout_kernel(const T* __restrict__ x, T* __restrict__ y, int64_t chunks,
                                                      const NormDropout drop) {
  constexpr int U = 4;
  PhiloxKey key{};
  if (drop.thr > 0) key = philox_key(drop.rng);
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (256 * U) + threadIdx.x;
  Chunk<T> c[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (base + u * 256 < chunks) c[u].load(x + (base + u * 256) * 8);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = base + u * 256;
    if (i >= chunks) continue;
    if (drop.thr > 0) {
      const uint32_t keep = philox_keep(philox_block(static_cast<uint64_t>(i), key), drop.thr);
      float f[8];
      c[u].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (keep >> e) & 1u ? f[e] * drop.scale : 0.f;
      c[u].put(f);
    }
    c[u].store(y + i * 8);
  }
}

// Dropout, any number of columns: a thread takes eight consecutive elements of the
// flat array (16-byte aligned), which lie in one or more rows, and evaluates every
// counter block that they touch (two in most places).
template <typename T>
__global__ void __launch_bounds__(256) dropout_any_kernel(const T* __restrict__ x, T* __restrict__ y, int64_t total,
                                                          int32_t cols, const NormDropout drop) {
  const int64_t e0 = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (e0 >= total) return;
  const int n = total - e0 < 8 ? static_cast<int>(total - e0) : 8;
  Chunk<T> c;
  if (n == 8) c.load(x + e0); else c.load_n(x + e0, n);
  if (drop.thr > 0) {
    const PhiloxKey key = philox_key(drop.rng);
    const uint32_t n8 = static_cast<uint32_t>((cols + 7) >> 3);
    int64_t row;
    int32_t col;
    if (total <= 0x7fffffff) {
      const uint32_t r = static_cast<uint32_t>(e0) / static_cast<uint32_t>(cols);
      row = r;
      col = static_cast<int32_t>(static_cast<uint32_t>(e0) - r * static_cast<uint32_t>(cols));
    } else {
      row = e0 / cols;
      col = static_cast<int32_t>(e0 - row * cols);
    }
    uint32_t keep = 0;
    for (int j = 0; j < n;) {
      const uint32_t word = philox_keep(philox_block(static_cast<uint64_t>(row) * n8 + (col >> 3), key), drop.thr);
      const int first = col & 7;
      const int take = min(min(8 - first, cols - col), n - j);
      keep |= ((word >> first) & ((1u << take) - 1u)) << j;
      j += take;
      col += take;
      if (col == cols) {
        col = 0;
        ++row;
      }
    }
    float f[8];
    c.get(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (keep >> e) & 1u ? f[e] * drop.scale : 0.f;
    c.put(f);
  }
  if (n == 8) c.store(y + e0); else c.store_n(y + e0, n);
}

template <typename T>
cudaError_t dropout_t(const void* x, void* y, int64_t rows, int32_t cols, const NormDropout& drop, cudaStream_t stream) {
  const int64_t total = rows * cols;
  const bool flat = (cols & 7) == 0;
  const int64_t per = flat ? 256 * 4 * 8 : 256 * 8;
  const int64_t blocks = (total + per - 1) / per;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (blocks < 1) return cudaSuccess;
  if (flat)
    dropout_kernel<T><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(static_cast<const T*>(x), static_cast<T*>(y),
                                                                        total / 8, drop);
  else
    dropout_any_kernel<T><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(static_cast<const T*>(x),
                                                                            static_cast<T*>(y), total, cols, drop);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_fwd(int dtype, const NormFwdArgs& a, cudaStream_t stream) {
  if (a.rows < 1) return cudaSuccess;
  const bool vec = (a.cols & 7) == 0;   // then every row starts on a 16-byte boundary
  switch (dtype) {
    case 0: return vec ? pick_fwd<__nv_bfloat16, true>(a, stream) : pick_fwd<__nv_bfloat16, false>(a, stream);
    case 1: return vec ? pick_fwd<__half, true>(a, stream) : pick_fwd<__half, false>(a, stream);
    default: return vec ? pick_fwd<float, true>(a, stream) : pick_fwd<float, false>(a, stream);
  }
}

cudaError_t launch_dropout(int dtype, const void* x, void* y, int64_t rows, int32_t cols, const NormDropout& drop,
                           cudaStream_t stream) {
  switch (dtype) {
    case 0: return dropout_t<__nv_bfloat16>(x, y, rows, cols, drop, stream);
    case 1: return dropout_t<__half>(x, y, rows, cols, drop, stream);
    default: return dropout_t<float>(x, y, rows, cols, drop, stream);
  }
}

}  // namespace sta
