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
//
// Measured (a plain copy moves 6400 GB/s): 1 382 400 x 128 bf16 in 118 us, 6000 GB/s; 57 600 x
// 1536 bf16 with residual and dropout in 119 us, 5950 GB/s; fp32 5000 to 5900 GB/s, from 2048
// columns on 4100 to 5900.  Rows of an odd width pass shared memory four times and are bound by
// that, their shifts and their barriers: 36 377 x 1153 bf16 2000 GB/s, fp32 3290; 173 318 x 121 fp32
// 4360; 2 M x 20 bf16 2160.
#include "norm_common.cuh"

namespace sta {
namespace {

using namespace norm;

// s / n from s and 1 / n: the product, and what it lacks of s, s - q n, which an fma gives without
// rounding, divided in the same way.  The sum of up to 8192 equal bf16 or fp16 values is exact in
// fp32, and so is their mean then: a constant row's y is the bias (with the product alone, 1 / n's
// rounding times 1 / sqrt(eps)).  The two fma cost nothing without dropout and 2 to 3 % with it,
// where the vector kernels leave them out; a division took 2 to 13 % of the bf16 kernels' time.
__device__ __forceinline__ float mean_of(float s, float n, float inv_n) {
  const float q = s * inv_n, r = fmaf(-q, n, s);
  return fmaf(r == r ? r : 0.f, inv_n, q);   // an infinite sum stays one
}

// TPR threads share a row (0: the whole block); a thread holds CH chunks of R rows at a
// time.  A warp (or block) takes consecutive rows; STAGES - 1 of its steps are on their way
// to shared memory while one is in registers, so the bytes in flight do not depend on the
// registers: with the next rows prefetched into registers the kernel moved 3.8 TB/s.
template <typename T, int TPR, int CH, int R, int STAGES>
__global__ void __launch_bounds__(TPR > 0 ? 256 : 512) norm_fwd_kernel(const NormFwdArgs a) {
  constexpr bool kBlock = TPR == 0;
  constexpr int kGroups = kBlock ? 1 : 32 / (TPR > 0 ? TPR : 1);
  constexpr int kRows = kGroups * R;              // rows of a step
  constexpr bool kOwnRows = kBlock || CH > 2;    // how a row goes out
  __shared__ float red[2][R][32];   // block mode: sums of a row, of its values and of its squares
  extern __shared__ __align__(16) uint8_t bufs[];
  const int lane = kBlock ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x & 31) % (TPR > 0 ? TPR : 1);
  const int grp = kBlock ? 0 : static_cast<int>(threadIdx.x & 31) / (TPR > 0 ? TPR : 1);
  const int step = kBlock ? static_cast<int>(blockDim.x) : TPR;
  const int st = kBlock ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x & 31);
  const int snt = kBlock ? static_cast<int>(blockDim.x) : 32;
  const int64_t unit = kBlock ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t units = kBlock ? gridDim.x : static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  const int32_t n8 = (a.cols + 7) >> 3;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  T* y = static_cast<T*>(a.y);
  T* h = static_cast<T*>(a.h);
  PhiloxKey key{};
  if (a.drop.thr > 0) key = philox_key(a.drop.rng);
  const uint32_t one = span_stage<T>(kRows, a.cols), stage = res != nullptr ? 2 * one : one;
  uint8_t* mine = bufs + (kBlock ? 0 : (threadIdx.x >> 5) * STAGES * stage);
  uint64_t w[CH][4], b[CH][4];   // they stay in registers
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int32_t ch = lane + k * step;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[k][i] = both(1.f);
      b[k][i] = 0;
    }
    if (ch < n8) {
      const int n = min(8, a.cols - ch * 8);
      if (a.weight != nullptr) load_param2<T>(a.weight, a.wfp32, ch * 8, n, w[k]);
      if (a.bias != nullptr) load_param2<T>(a.bias, a.wfp32, ch * 8, n, b[k]);
    }
  }
  auto rows_at = [&](int64_t base) { return static_cast<int>(min(static_cast<int64_t>(kRows), a.rows - base)); };
  auto fetch = [&](int64_t base, int slot) {   // the step that starts at row `base`, if there is one
    if (base < a.rows) {
      const int n = rows_at(base) * a.cols;
      uint8_t* p = mine + slot * stage;
      span_load(p, x + base * a.cols, n, st, snt);
      if (res != nullptr) span_load(p + one, res + base * a.cols, n, st, snt);
    }
    span_commit();
  };
  int64_t ahead = unit * kRows;
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i, ahead += units * kRows) fetch(ahead, i);
  int slot = 0;
  for (int64_t base = unit * kRows; base < a.rows; base += units * kRows, ahead += units * kRows) {
    fetch(ahead, slot == 0 ? STAGES - 1 : slot - 1);
    span_wait<STAGES - 1>();
    span_sync<kBlock>();
    const int live = rows_at(base);
    uint8_t* p = mine + slot * stage;
    uint64_t f[R][CH][4];
    const T* ex = span_elems(p, x + base * a.cols);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int q = r * kGroups + grp, c0 = (lane + k * step) * 8;
        span_get<T, TPR == 1>(ex, q * a.cols + c0, q < live ? a.cols - c0 : 0, f[r][k]);
      }
    if (a.drop.thr > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < CH; ++k)
          drop_pairs(f[r][k], static_cast<uint64_t>(base + r * kGroups + grp) * n8 + (lane + k * step), key, a.drop);
    }
    if (res != nullptr) {
      const T* er = span_elems(p + one, res + base * a.cols);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int q = r * kGroups + grp, c0 = (lane + k * step) * 8;
          uint64_t g[4];
          span_get<T, TPR == 1>(er, q * a.cols + c0, q < live ? a.cols - c0 : 0, g);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[r][k][i] = add_f32x2(f[r][k][i], g[i]);
        }
    }
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint64_t s[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i & 1] = add_f32x2(s[i & 1], f[r][k][i]);   // columns past the row hold zero
      mean[r] = mean_of(row_sum<TPR>(sum_f32x2(add_f32x2(s[0], s[1])), red[0][r]), a.n, a.inv_n);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t nm = both(-mean[r]);
      uint64_t s[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int32_t left = a.cols - (lane + k * step) * 8;   // columns of the chunk that exist
        if (left >= 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t e = add_f32x2(f[r][k][i], nm);
            s[i & 1] = fma_f32x2(e, e, s[i & 1]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float u, v;
            f32x2_split(add_f32x2(f[r][k][i], nm), u, v);
            const uint64_t e = f32x2(2 * i < left ? u : 0.f, 2 * i + 1 < left ? v : 0.f);
            s[i & 1] = fma_f32x2(e, e, s[i & 1]);
          }
        }
      }
      rstd[r] = rsqrtf(fmaf(row_sum<TPR>(sum_f32x2(add_f32x2(s[0], s[1])), red[1][r]), a.inv_n, a.eps));
    }
    // rows out: h as it is, y normalised
#pragma unroll
    for (int out = 0; out < 2; ++out) {
      T* dst = out == 0 ? h : y;
      if (dst == nullptr) continue;
      span_sync<kBlock>();   // the slot's values are in registers (or stored): it carries the output
      // long rows lie on boundaries of their own (row_put), shorter ones as the span
      T* eo = span_elems(p, dst + base * a.cols);
      const uint32_t pitch = static_cast<uint32_t>(n8) * 8 * sizeof(T);
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int32_t ch = lane + k * step;
        if (ch >= n8) continue;
        const int n = min(8, a.cols - ch * 8);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int q = r * kGroups + grp;
          if (q >= live) continue;
          uint64_t v[4];
          const uint64_t nm = both(-mean[r]), rs = both(rstd[r]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = out == 0 ? f[r][k][i] : fma_f32x2(mul_f32x2(add_f32x2(f[r][k][i], nm), rs), w[k][i], b[k][i]);
          if constexpr (kOwnRows) {
            row_put<T>(static_cast<uint32_t>(__cvta_generic_to_shared(p)) + q * pitch + ch * 8 * sizeof(T), v);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float u, t;
              f32x2_split(v[i], u, t);
              if (2 * i < n) eo[q * a.cols + ch * 8 + 2 * i] = from_f<T>(u);
              if (2 * i + 1 < n) eo[q * a.cols + ch * 8 + 2 * i + 1] = from_f<T>(t);
            }
          }
        }
      }
      span_sync<kBlock>();
      if constexpr (kOwnRows) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int q = r * kGroups + grp;
          if (q < live) row_store(p + q * pitch, dst + (base + q) * a.cols, a.cols, lane, step);
        }
      } else {
        span_store(p, dst + base * a.cols, live * a.cols, st, snt);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int q = r * kGroups + grp;
      if (lane == 0 && q < live) {
        if (a.mean != nullptr) a.mean[base + q] = mean[r];
        if (a.rstd != nullptr) a.rstd[base + q] = rstd[r];
      }
    }
    span_sync<kBlock>();   // every thread is done with the slot: the next step's fetch fills it
    slot = slot + 1 == STAGES ? 0 : slot + 1;
  }
  span_wait<0>();
}

// The same for rows of a multiple of eight columns (see Own): no shared spans, addresses
// that advance by one constant, half the instructions.
// DROP: with dropout, whose generator takes registers that the other calls use for more warps.
template <typename T, bool DROP, int TPR, int CH, int R, int STAGES>
__global__ void __launch_bounds__(TPR > 0 ? 256 : 512, TPR > 0 && CH <= 2 ? 2 : 1) norm_fwd_vec_kernel(const NormFwdArgs a) {
  constexpr bool kBlock = TPR == 0;
  constexpr int kGroups = kBlock ? 1 : 32 / (TPR > 0 ? TPR : 1);
  constexpr int kRows = kGroups * R;              // rows of a step
  constexpr int kParts = Own<T>::kParts;
  constexpr int kChunkBytes = 16 * kParts;
  __shared__ float red[2][R][32];   // block mode: sums of a row, of its values and of its squares
  extern __shared__ __align__(16) uint8_t bufs[];
  const int lane = kBlock ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x & 31) % (TPR > 0 ? TPR : 1);
  const int grp = kBlock ? 0 : static_cast<int>(threadIdx.x & 31) / (TPR > 0 ? TPR : 1);
  const int step = kBlock ? static_cast<int>(blockDim.x) : TPR;
  const uint32_t part = 16u * (kBlock ? blockDim.x : 256u);   // 16 bytes of every thread
  const int64_t unit = kBlock ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t units = kBlock ? gridDim.x : static_cast<int64_t>(gridDim.x) * 8;
  const int32_t n8 = a.cols >> 3;
  const bool has_res = a.residual != nullptr;
  const uint32_t arr = static_cast<uint32_t>(R * CH * kParts) * part;   // one array of one stage
  const uint32_t stage = has_res ? 2 * arr : arr;
  const uint32_t sm = static_cast<uint32_t>(__cvta_generic_to_shared(bufs)) + 16 * threadIdx.x;
  PhiloxKey key{};
  if (DROP) key = philox_key(a.drop.rng);
  const int psize = a.wfp32 ? 4 : static_cast<int>(sizeof(T)), p_bytes = step * 8 * psize;
  const char* wp = static_cast<const char*>(a.weight) + lane * 8 * psize;   // this thread's first parameters
  const char* bp = static_cast<const char*>(a.bias) + lane * 8 * psize;
  uint64_t w[CH][4], b[CH][4];   // they stay in registers
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int32_t ch = lane + k * step;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[k][i] = both(1.f);
      b[k][i] = 0;
    }
    if (ch < n8) {
      if (a.weight != nullptr) read_param2<T>(wp + k * p_bytes, a.wfp32, w[k]);
      if (a.bias != nullptr) read_param2<T>(bp + k * p_bytes, a.wfp32, b[k]);
    }
  }
  // Addresses: one pointer per array, at this thread's first chunk of a step's first row; a
  // step, a row of the step and a chunk each add a constant.  Rows are counted down from
  // the thread's first one in 32 bits (capped where it cannot matter).
  const int64_t row_bytes = static_cast<int64_t>(a.cols) * sizeof(T);
  const int64_t step_bytes = units * kRows * row_bytes, r_bytes = kGroups * row_bytes;
  const int k_bytes = step * kChunkBytes;
  const int64_t row0 = unit * kRows + grp, off0 = row0 * row_bytes + lane * kChunkBytes;
  const int64_t step_rows = units * kRows;
  const char* px = static_cast<const char*>(a.x) + off0;
  const char* pr = static_cast<const char*>(a.residual) + off0;
  int64_t left_in = a.rows - row0;
  auto fetch = [&](uint32_t at) {
    const int left = static_cast<int>(left_in < 4096 ? left_in : 4096);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        // what does not exist reads as zero
        const bool ok = r * kGroups < left && lane + k * step < n8;
        const int64_t o = ok ? r * r_bytes + k * k_bytes : 0;
        const uint32_t d = at + static_cast<uint32_t>((r * CH + k) * kParts) * part;
        Own<T>::copy_or_zero(d, part, (ok ? px : static_cast<const char*>(a.x)) + o, ok);
        if (has_res) Own<T>::copy_or_zero(d + arr, part, (ok ? pr : static_cast<const char*>(a.residual)) + o, ok);
      }
    span_commit();
    left_in -= step_rows;
    px += step_bytes;
    pr += step_bytes;
  };
  const bool partial = n8 != step * CH;   // some threads have fewer chunks
  int64_t row = row0, left64 = left_in;
  char *py = static_cast<char*>(a.y) + off0, *ph = static_cast<char*>(a.h) + off0;
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(sm + i * stage);
  uint32_t cur = 0;   // the stage in use
  for (int64_t base = unit * kRows; base < a.rows; base += step_rows) {
    const int left = static_cast<int>(left64 < 4096 ? left64 : 4096);
    fetch(sm + (cur == 0 ? (STAGES - 1) * stage : cur - stage));
    span_wait<STAGES - 1>();
    uint64_t f[R][CH][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const uint32_t d = sm + cur + static_cast<uint32_t>((r * CH + k) * kParts) * part;
        Own<T>::read(d, part, f[r][k]);
        if (DROP)
          drop_pairs(f[r][k], static_cast<uint64_t>(row + r * kGroups) * n8 + (lane + k * step), key, a.drop);
        if (has_res) {
          uint64_t g[4];
          Own<T>::read(d + arr, part, g);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[r][k][i] = add_f32x2(f[r][k][i], g[i]);
        }
      }
    cur = cur + stage == STAGES * stage ? 0 : cur + stage;
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint64_t s[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i & 1] = add_f32x2(s[i & 1], f[r][k][i]);   // missing chunks hold zero
      const float t = row_sum<TPR>(sum_f32x2(add_f32x2(s[0], s[1])), red[0][r]);
      mean[r] = DROP ? t * a.inv_n : mean_of(t, a.n, a.inv_n);   // a row with dropped values is not constant
    }
    if (a.h != nullptr) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < CH; ++k)
          if (r * kGroups < left && lane + k * step < n8) Own<T>::write(ph + r * r_bytes + k * k_bytes, f[r][k]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t nm = both(-mean[r]);
      uint64_t s[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        if (partial && lane + k * step >= n8) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[r][k][i] = add_f32x2(f[r][k][i], nm);
          s[i & 1] = fma_f32x2(f[r][k][i], f[r][k][i], s[i & 1]);
        }
      }
      rstd[r] = rsqrtf(fmaf(row_sum<TPR>(sum_f32x2(add_f32x2(s[0], s[1])), red[1][r]), a.inv_n, a.eps));
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int32_t ch = lane + k * step;
      if (ch >= n8) continue;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint64_t rs = both(rstd[r]);
        uint64_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fma_f32x2(mul_f32x2(f[r][k][i], rs), w[k][i], b[k][i]);
        if (r * kGroups < left) Own<T>::write(py + r * r_bytes + k * k_bytes, v);
      }
    }
    if (lane == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r * kGroups < left) {
          if (a.mean != nullptr) (a.mean + row)[r * kGroups] = mean[r];
          if (a.rstd != nullptr) (a.rstd + row)[r * kGroups] = rstd[r];
        }
    }
    left64 -= step_rows;
    row += step_rows;
    py += step_bytes;
    ph += step_bytes;
  }
  span_wait<0>();
}

template <typename T, bool VEC, int TPR, int CH, int R, int STAGES>
cudaError_t launch_fwd(const NormFwdArgs& a, cudaStream_t stream) {
  void (*kern)(NormFwdArgs);
  if constexpr (VEC)
    kern = a.drop.thr > 0 ? norm_fwd_vec_kernel<T, true, TPR, CH, R, STAGES>
                          : norm_fwd_vec_kernel<T, false, TPR, CH, R, STAGES>;
  else
    kern = norm_fwd_kernel<T, TPR, CH, R, STAGES>;
  constexpr int rows = (TPR > 0 ? 32 / (TPR > 0 ? TPR : 1) : 1) * R;   // of a warp's (block's) step
  int threads = 256;
  if (TPR == 0) threads = (((a.cols + 7) / 8 + CH - 1) / CH + 31) / 32 * 32;
  const int per_block = (TPR > 0 ? threads / 32 : 1);
  const int stage = VEC ? R * CH * threads * 8 * static_cast<int>(sizeof(T))
                        : per_block * static_cast<int>(span_stage<T>(rows, a.cols));
  const int smem = STAGES * (a.residual != nullptr ? 2 : 1) * stage + (VEC ? 0 : kSpanSlack);
  int sms = 0, dev = 0, fit = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = allow_smem(kern, 2 * R * 32 * 4);   // red
  if (e != cudaSuccess) return e;
  const int64_t need = ((a.rows + rows - 1) / rows + per_block - 1) / per_block;
  int64_t blocks = need;
  if (need > sms) {   // a persistent grid: as many blocks as the SMs hold (a small call saves the query)
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kern, threads, smem)) != cudaSuccess) return e;
    if (fit < 1) return cudaErrorInvalidConfiguration;
    if (blocks > static_cast<int64_t>(sms) * fit) blocks = static_cast<int64_t>(sms) * fit;
  }
  kern<<<static_cast<unsigned>(blocks), threads, smem, stream>>>(a);
  return cudaGetLastError();
}

// A warp takes rows of up to 1536 columns (48 values of a row, weight and bias in a thread's
// registers), a block longer ones.  Stages and rows of a step by what was fastest; the rates
// are of plain calls over 170 M elements, bf16 and fp32, in GB/s:
//   128 columns: 16 threads a row 6140, 8 threads (half the shuffles, fewer rows in flight) 5150;
//   512: one row a step and three stages 6160 and 5320, two rows and four (two) 5140 and 5310;
//   1024: a warp and two rows (fp32: one) 6180 and 5620, a block a row 4970 and 5260;
//   1536: a warp 6090 and 5210, a block 4480 and 4430;
//   weight and bias read again for every row: 4580 and 5040 at 1024 columns, 4530 and 4430 at 1536;
//   2048 and more: two rows a step 5520 and 5910, one 3840 and 4440 (4096: 5370 and 5440, 3600 and
//   4030).  Above 4096 columns two fp32 rows with a residual do not fit in shared memory.
// Rows that go through spans have fewer threads a row up to 512 columns: their rows' ends and
// barriers bind, and 8 threads a row move 2820 and 4340 at 121 columns, 16 2420 and 3450 (at 20 columns
// two threads 2160 and 3930, four 1520 and 2840).
template <typename T, bool VEC>
cudaError_t pick_fwd(const NormFwdArgs& a, cudaStream_t stream) {
  constexpr bool k16 = sizeof(T) == 2;
  const int n8 = (a.cols + 7) >> 3;
  if (n8 <= 1) return launch_fwd<T, VEC, 1, 1, 2, k16 ? 4 : 2>(a, stream);
  if constexpr (VEC) {
    if (n8 <= 4) return launch_fwd<T, VEC, 4, 1, 2, 3>(a, stream);
    if (n8 <= 8) return launch_fwd<T, VEC, 8, 1, k16 ? 2 : 4, 3>(a, stream);
    if (n8 <= 16) return launch_fwd<T, VEC, 16, 1, k16 ? 4 : 2, k16 ? 2 : 3>(a, stream);
    if (n8 <= 32) return launch_fwd<T, VEC, k16 ? 16 : 32, k16 ? 2 : 1, k16 ? 1 : 2, 3>(a, stream);
    if (n8 <= 64) return launch_fwd<T, VEC, 32, 2, 1, 3>(a, stream);
  } else {
    constexpr int S = k16 ? 4 : 2;
    if (n8 <= 4) return launch_fwd<T, VEC, 2, 2, 2, S>(a, stream);
    if (n8 <= 8) return launch_fwd<T, VEC, 4, 2, 2, S>(a, stream);
    if (n8 <= 16) return launch_fwd<T, VEC, 8, 2, 2, S>(a, stream);
    if (n8 <= 32) return launch_fwd<T, VEC, 16, 2, 2, S>(a, stream);
    if (n8 <= 64) return launch_fwd<T, VEC, 32, 2, 2, S>(a, stream);
  }
  if (n8 <= 128) return launch_fwd<T, VEC, 32, 4, k16 ? 2 : 1, 2>(a, stream);
  if (n8 <= 192) return launch_fwd<T, VEC, 32, 6, 1, k16 ? 3 : 2>(a, stream);
  if (k16 || n8 <= 512) return launch_fwd<T, VEC, 0, 2, 2, 2>(a, stream);
  return launch_fwd<T, VEC, 0, 2, 1, 2>(a, stream);
}

// Dropout, rows of a multiple of eight columns: chunk i of the flat array is counter block i.
// Four chunks a thread, all loaded first: 115 200 x 1536 bf16 in 119 us, 5950 GB/s (a copy takes
// 111 us); two chunks 134 us, eight 120 us.
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

// Dropout, any number of columns: a thread takes eight consecutive elements of the flat array
// (16-byte aligned) at a time, four times, its warp 32 times as many side by side.  They lie in
// two counter blocks in most places: that of their first element, which the thread evaluates, and
// the next, which is the next thread's; what is not there (row ends, the warp's last thread)
// is evaluated too.  Bound by the generator and the places' arithmetic: 72 754 x 1153 bf16 2580
// GB/s, fp32 4240; with every block evaluated by each thread that needs it 2120 and 3760, and 4 to
// 15 % more than here below 100 columns.
template <typename T>
__global__ void __launch_bounds__(256) dropout_any_kernel(const T* __restrict__ x, T* __restrict__ y, int64_t total,
                                                          int32_t cols, const NormDropout drop) {
  constexpr int U = 4;
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int64_t first = ((static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * (32 * U) + lane) * 8;
  Chunk<T> c[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t e0 = first + u * 256;
    if (e0 + 8 <= total) c[u].load(x + e0);
    else if (e0 < total) c[u].load_n(x + e0, static_cast<int>(total - e0));
  }
  if (drop.thr > 0) {
    const PhiloxKey key = philox_key(drop.rng);
    const uint32_t n8 = static_cast<uint32_t>((cols + 7) >> 3);
    int64_t row[U];
    int32_t col[U];
    uint32_t word[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t e0 = first + u * 256;
      if (total <= 0x7fffffff) {   // then e0 fits 32 bits unsigned
        const uint32_t r = static_cast<uint32_t>(e0) / static_cast<uint32_t>(cols);
        row[u] = r;
        col[u] = static_cast<int32_t>(static_cast<uint32_t>(e0) - r * static_cast<uint32_t>(cols));
      } else {
        row[u] = e0 / cols;
        col[u] = static_cast<int32_t>(e0 - row[u] * cols);
      }
      word[u] = philox_keep(philox_block(static_cast<uint64_t>(row[u]) * n8 + (col[u] >> 3), key), drop.thr);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // the next thread's block: its number (low half, which tells neighbours apart) and bits
      const uint32_t own = static_cast<uint32_t>(static_cast<uint64_t>(row[u]) * n8 + (col[u] >> 3));
      uint32_t next = __shfl_down_sync(0xffffffffu, own, 1), bits = __shfl_down_sync(0xffffffffu, word[u], 1);
      const int v = u + 1 < U ? u + 1 : u;
      const uint32_t own0 = __shfl_sync(0xffffffffu, static_cast<uint32_t>(static_cast<uint64_t>(row[v]) * n8 + (col[v] >> 3)), 0);
      const uint32_t word0 = __shfl_sync(0xffffffffu, word[v], 0);
      if (lane == 31) {
        next = own0;   // of the same step again where there is none after it: no later block, so it never matches
        bits = word0;
      }
      const int64_t e0 = first + u * 256;
      const int n = total - e0 < 8 ? static_cast<int>(total - e0) : 8;
      uint32_t keep = 0;
      int64_t r = row[u];
      int32_t k = col[u];
      for (int j = 0; j < n;) {
        const uint64_t block = static_cast<uint64_t>(r) * n8 + (k >> 3);
        uint32_t w = word[u];
        if (j > 0) w = static_cast<uint32_t>(block) == next ? bits : philox_keep(philox_block(block, key), drop.thr);
        const int at = k & 7;
        const int take = min(min(8 - at, cols - k), n - j);
        keep |= ((w >> at) & ((1u << take) - 1u)) << j;
        j += take;
        k += take;
        if (k == cols) {
          k = 0;
          ++r;
        }
      }
      float f[8];
      c[u].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (keep >> e) & 1u ? f[e] * drop.scale : 0.f;
      c[u].put(f);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t e0 = first + u * 256;
    if (e0 + 8 <= total) c[u].store(y + e0);
    else if (e0 < total) c[u].store_n(y + e0, static_cast<int>(total - e0));
  }
}

template <typename T>
cudaError_t dropout_t(const void* x, void* y, int64_t rows, int32_t cols, const NormDropout& drop, cudaStream_t stream) {
  const int64_t total = rows * cols;
  const bool flat = (cols & 7) == 0;
  constexpr int64_t per = 256 * 4 * 8;
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
