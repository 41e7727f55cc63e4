// norm_bwd.cu - layer norm backward for sm_100a.
//
// With z = (h - mean) rstd and g = dy w (n columns):
//   dh = rstd (g - sum g / n - z sum(g z) / n) + (the gradient that arrives at h itself)
//   dx = dropout mask * dh,  dresidual = dh,  dw = sum_rows dy z,  db = sum_rows dy.
//
// One pass over dy and h makes all of them.  A thread keeps the same columns of all
// its rows, so the column sums stay in its registers (fp32); each block writes its
// part once, and a second kernel adds the parts in a fixed order, so the weight's
// gradient is the same in every run.  The dropout mask is evaluated again from the
// generator.
#include "norm_common.cuh"

namespace sta {
namespace {

using namespace norm;

// Two sums over a row at once (see row_sum).
template <int TPR>
__device__ __forceinline__ void row_sum2(float& u, float& v, float2* red) {
  if constexpr (TPR > 0) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) {
      u += __shfl_xor_sync(0xffffffffu, u, o);
      v += __shfl_xor_sync(0xffffffffu, v, o);
    }
  } else {
    for (int o = 16; o > 0; o >>= 1) {
      u += __shfl_xor_sync(0xffffffffu, u, o);
      v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    const int lane = static_cast<int>(threadIdx.x) & 31, warps = static_cast<int>(blockDim.x) >> 5;
    if (lane == 0) red[threadIdx.x >> 5] = make_float2(u, v);
    __syncthreads();
    const float2 s = lane < warps ? red[lane] : make_float2(0.f, 0.f);
    u = s.x;
    v = s.y;
    for (int o = 16; o > 0; o >>= 1) {
      u += __shfl_xor_sync(0xffffffffu, u, o);
      v += __shfl_xor_sync(0xffffffffu, v, o);
    }
  }
}

template <typename T, bool VEC, int TPR, int CH, int R>
__global__ void __launch_bounds__(TPR > 0 ? 256 : 512) norm_bwd_kernel(const NormBwdArgs a) {
  // block mode: partial row sums, a buffer per row in flight and per step parity
  __shared__ float2 red[2][R][32];
  const int lane = TPR > 0 ? static_cast<int>(threadIdx.x) % (TPR > 0 ? TPR : 1) : static_cast<int>(threadIdx.x);
  const int step = TPR > 0 ? TPR : static_cast<int>(blockDim.x);
  const int per_block = TPR > 0 ? 256 / (TPR > 0 ? TPR : 1) : 1;
  const int my = TPR > 0 ? static_cast<int>(threadIdx.x) / (TPR > 0 ? TPR : 1) : 0;
  const int32_t n8 = (a.cols + 7) >> 3;
  const T* dy = static_cast<const T*>(a.dy);
  const T* h = static_cast<const T*>(a.h);
  const T* dh = static_cast<const T*>(a.dh);
  T* dx = static_cast<T*>(a.dx);
  T* dres = static_cast<T*>(a.dres);
  PhiloxKey key{};
  if (a.drop.thr > 0) key = philox_key(a.drop.rng);
  float w[CH][8], dw[CH][8], db[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int32_t ch = lane + k * step;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[k][i] = 1.f;
      dw[k][i] = 0.f;
      db[k][i] = 0.f;
    }
    if (a.weight != nullptr && ch < n8)
      load_param<T, VEC>(a.weight, a.wfp32, ch * 8, VEC ? 8 : min(8, a.cols - ch * 8), w[k]);
  }
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  int par = 0;
  // the block's rows: every thread makes the same number of steps (the sums synchronise)
  for (int64_t b0 = static_cast<int64_t>(blockIdx.x) * per_block * R; b0 < a.rows;
       b0 += static_cast<int64_t>(gridDim.x) * per_block * R, par ^= 1) {
    const int64_t row0 = b0 + static_cast<int64_t>(my) * R;
    Chunk<T> cy[R][CH], cz[R][CH];
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool live = row0 + r < a.rows;
      mean[r] = live ? __ldg(a.mean + row0 + r) : 0.f;
      rstd[r] = live ? __ldg(a.rstd + row0 + r) : 0.f;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int32_t ch = lane + k * step;
        cy[r][k].clear();
        cz[r][k].clear();
        if (live && ch < n8) {
          const int64_t at = (row0 + r) * a.cols + ch * 8;
          const int n = VEC ? 8 : min(8, a.cols - ch * 8);
          if (VEC) cy[r][k].load(dy + at); else cy[r][k].load_n(dy + at, n);
          if (VEC) cz[r][k].load(h + at); else cz[r][k].load_n(h + at, n);
        }
      }
    }
    float c1[R], c2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      c1[r] = 0.f;
      c2[r] = 0.f;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float y8[8], z8[8];
        cy[r][k].get(y8);
        cz[r][k].get(z8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float z = (z8[i] - mean[r]) * rstd[r], g = y8[i] * w[k][i];
          dw[k][i] = fmaf(y8[i], z, dw[k][i]);
          db[k][i] += y8[i];
          c1[r] += g;
          c2[r] = fmaf(g, z, c2[r]);
        }
      }
      row_sum2<TPR>(c1[r], c2[r], red[par][r]);
      c1[r] *= inv_n;
      c2[r] *= inv_n;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r >= a.rows) continue;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int32_t ch = lane + k * step;
        if (ch >= n8) continue;
        const int64_t at = (row0 + r) * a.cols + ch * 8;
        const int n = VEC ? 8 : min(8, a.cols - ch * 8);
        float y8[8], z8[8], o[8];
        cy[r][k].get(y8);
        cz[r][k].get(z8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float z = (z8[i] - mean[r]) * rstd[r];
          o[i] = (fmaf(y8[i], w[k][i], -c1[r]) - z * c2[r]) * rstd[r];
        }
        Chunk<T> c;
        if (dh != nullptr) {
          if (VEC) c.load(dh + at); else c.load_n(dh + at, n);
          float g[8];
          c.get(g);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += g[i];
        }
        if (dres != nullptr) {
          c.put(o);
          if (VEC) c.store(dres + at); else c.store_n(dres + at, n);
        }
        if (dx != nullptr) {
          if (a.drop.thr > 0) {
            const uint32_t keep = philox_keep(philox_block(static_cast<uint64_t>(row0 + r) * n8 + ch, key), a.drop.thr);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = (keep >> i) & 1u ? o[i] * a.drop.scale : 0.f;
          }
          c.put(o);
          if (VEC) c.store(dx + at); else c.store_n(dx + at, n);
        }
      }
    }
  }
  if (a.partial == nullptr) return;
  float* pw = a.partial + static_cast<int64_t>(blockIdx.x) * a.cols;
  float* pb = pw + static_cast<int64_t>(gridDim.x) * a.cols;
  if constexpr (TPR > 0) {
    // the block's groups: those of a warp by shuffles, the warps through shared memory
    __shared__ float acc[8][32 * CH * 8];
    const int warp = static_cast<int>(threadIdx.x) >> 5;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      if (pass) __syncthreads();
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float s = pass ? db[k][i] : dw[k][i];
#pragma unroll
          for (int o = 16; o >= TPR; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if ((static_cast<int>(threadIdx.x) & 31) < TPR) acc[warp][(lane + k * TPR) * 8 + i] = s;
        }
      __syncthreads();
      for (int32_t c = static_cast<int32_t>(threadIdx.x); c < a.cols; c += 256) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += acc[q][c];
        (pass ? pb : pw)[c] = s;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int32_t c0 = (lane + k * step) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + i < a.cols) {
          pw[c0 + i] = dw[k][i];
          pb[c0 + i] = db[k][i];
        }
    }
  }
}

// Column c of dw (y = 0) or db (y = 1): the parts in order, 32 threads each.
template <typename T>
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* __restrict__ partial, int parts, int32_t cols,
                                                           void* dweight, void* dbias, bool wfp32) {
  void* out = blockIdx.y == 0 ? dweight : dbias;
  if (out == nullptr) return;
  __shared__ float acc[32][33];
  const int x = static_cast<int>(threadIdx.x) & 31, y = static_cast<int>(threadIdx.x) >> 5;
  const int32_t c = static_cast<int32_t>(blockIdx.x) * 32 + x;
  const float* p = partial + static_cast<int64_t>(blockIdx.y) * parts * cols;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int q = y; q < parts; q += 32) s += p[static_cast<int64_t>(q) * cols + c];
  }
  acc[y][x] = s;
  __syncthreads();
  // thread (x, y) takes column y's 32 sums
  s = acc[x][y];
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int32_t cc = static_cast<int32_t>(blockIdx.x) * 32 + y;
  if (x == 0 && cc < cols) {
    if (wfp32)
      static_cast<float*>(out)[cc] = s;
    else
      static_cast<T*>(out)[cc] = from_f<T>(s);
  }
}

// Launch shape of the first kernel: threads of a block, rows of a block's step, blocks.
struct BwdShape {
  int tpr, ch, r;       // template arguments
  int threads;
  int64_t blocks;
};

BwdShape bwd_shape(int64_t rows, int32_t cols) {
  const int n8 = (cols + 7) >> 3;
  BwdShape s{};
  if (n8 <= 1) { s.tpr = 1; s.ch = 1; s.r = 2; }
  else if (n8 <= 4) { s.tpr = 4; s.ch = 1; s.r = 2; }
  else if (n8 <= 16) { s.tpr = 16; s.ch = 1; s.r = 2; }
  else if (n8 <= 32) { s.tpr = 32; s.ch = 1; s.r = 2; }
  else if (n8 <= 64) { s.tpr = 32; s.ch = 2; s.r = 1; }
  else if (n8 <= 512) { s.tpr = 0; s.ch = 1; s.r = 2; }
  else if (n8 <= 1024) { s.tpr = 0; s.ch = 2; s.r = 1; }
  else { s.tpr = 0; s.ch = 4; s.r = 1; }
  int per_sm;
  int64_t block_rows;
  if (s.tpr > 0) {
    s.threads = 256;
    block_rows = static_cast<int64_t>(256 / s.tpr) * s.r;
    per_sm = 3;
  } else {
    s.threads = ((n8 + s.ch - 1) / s.ch + 31) / 32 * 32;
    block_rows = s.r;
    per_sm = 768 / s.threads;
    per_sm = per_sm < 1 ? 1 : (per_sm > 8 ? 8 : per_sm);
  }
  const int64_t need = (rows + block_rows - 1) / block_rows;
  s.blocks = need < 148 * per_sm ? need : 148 * per_sm;
  return s;
}

template <typename T, bool VEC>
cudaError_t bwd_t(const NormBwdArgs& a, cudaStream_t stream) {
  const BwdShape s = bwd_shape(a.rows, a.cols);
  const unsigned g = static_cast<unsigned>(s.blocks);
  if (a.rows > 0) {
    if (s.tpr == 1) norm_bwd_kernel<T, VEC, 1, 1, 2><<<g, s.threads, 0, stream>>>(a);
    else if (s.tpr == 4) norm_bwd_kernel<T, VEC, 4, 1, 2><<<g, s.threads, 0, stream>>>(a);
    else if (s.tpr == 16) norm_bwd_kernel<T, VEC, 16, 1, 2><<<g, s.threads, 0, stream>>>(a);
    else if (s.tpr == 32 && s.ch == 1) norm_bwd_kernel<T, VEC, 32, 1, 2><<<g, s.threads, 0, stream>>>(a);
    else if (s.tpr == 32) norm_bwd_kernel<T, VEC, 32, 2, 1><<<g, s.threads, 0, stream>>>(a);
    else if (s.ch == 1) norm_bwd_kernel<T, VEC, 0, 1, 2><<<g, s.threads, 0, stream>>>(a);
    else if (s.ch == 2) norm_bwd_kernel<T, VEC, 0, 2, 1><<<g, s.threads, 0, stream>>>(a);
    else norm_bwd_kernel<T, VEC, 0, 4, 1><<<g, s.threads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.dweight != nullptr || a.dbias != nullptr) {
    const dim3 grid(static_cast<unsigned>((a.cols + 31) / 32), 2);
    norm_reduce_kernel<T><<<grid, 1024, 0, stream>>>(a.partial, static_cast<int>(s.blocks), a.cols, a.dweight, a.dbias,
                                                     a.wfp32);
  }
  return cudaGetLastError();
}

}  // namespace

int norm_bwd_parts(int64_t rows, int32_t cols) { return static_cast<int>(bwd_shape(rows, cols).blocks); }

cudaError_t launch_norm_bwd(int dtype, const NormBwdArgs& a, cudaStream_t stream) {
  const bool vec = (a.cols & 7) == 0;
  switch (dtype) {
    case 0: return vec ? bwd_t<__nv_bfloat16, true>(a, stream) : bwd_t<__nv_bfloat16, false>(a, stream);
    case 1: return vec ? bwd_t<__half, true>(a, stream) : bwd_t<__half, false>(a, stream);
    default: return vec ? bwd_t<float, true>(a, stream) : bwd_t<float, false>(a, stream);
  }
}

}  // namespace sta
