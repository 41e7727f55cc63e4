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
//
// Measured (a plain copy moves 6400 GB/s): 1 382 400 x 128 bf16 in 174 us, 6100 GB/s; 57 600 x
// 1536 bf16 with the gradient that reaches h, dropout and both outputs in 180 us, 4900 GB/s, bound
// by the generator's and the row's instructions at 12 warps an SM; fp32 4500 to 5900 GB/s; odd
// widths from 9 columns on 1000 to 4000 GB/s (36 377 x 1153 bf16 2190, fp32 3390), bound by their
// passes through shared memory and the barriers.
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

// Writes this block's part of the column sums: dw at partial[block], db at partial[blocks + block].
// A thread's sums are of chunks lane, lane + step, ... (every thread of the block calls it).
template <int TPR, int CH>
__device__ __forceinline__ void store_column_sums(const NormBwdArgs& a, const uint64_t (&dw)[CH][4], const uint64_t (&db)[CH][4],
                                                  int lane, int step) {
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
        for (int i = 0; i < 4; ++i) {
          float u[2];
          f32x2_split(pass ? db[k][i] : dw[k][i], u[0], u[1]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int o = 16; o >= TPR; o >>= 1) u[j] += __shfl_xor_sync(0xffffffffu, u[j], o);
            if ((static_cast<int>(threadIdx.x) & 31) < TPR) acc[warp][(lane + k * TPR) * 8 + 2 * i + j] = u[j];
          }
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
      for (int i = 0; i < 4; ++i) {
        float u[2], v[2];
        f32x2_split(dw[k][i], u[0], u[1]);
        f32x2_split(db[k][i], v[0], v[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (c0 + 2 * i + j < a.cols) {
            pw[c0 + 2 * i + j] = u[j];
            pb[c0 + 2 * i + j] = v[j];
          }
      }
    }
  }
}

// TPR threads share a row (0: the whole block); a thread holds CH chunks of R rows at a
// time, while the next STAGES - 1 steps of its warp (block) are on their way to shared memory.
template <typename T, int TPR, int CH, int R, int STAGES>
__global__ void __launch_bounds__(TPR > 0 ? 256 : 512) norm_bwd_kernel(const NormBwdArgs a) {
  constexpr bool kBlock = TPR == 0;
  constexpr int kGroups = kBlock ? 1 : 32 / (TPR > 0 ? TPR : 1);
  constexpr int kRows = kGroups * R;   // rows of a warp's (block's) step
  constexpr bool kOwnRows = kBlock || TPR >= 16;   // how a row goes out
  // block mode: partial row sums, a buffer per row in flight and per step parity
  __shared__ float2 red[2][R][32];
  extern __shared__ __align__(16) uint8_t bufs[];
  const int lane = kBlock ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x & 31) % (TPR > 0 ? TPR : 1);
  const int grp = kBlock ? 0 : static_cast<int>(threadIdx.x & 31) / (TPR > 0 ? TPR : 1);
  const int step = kBlock ? static_cast<int>(blockDim.x) : TPR;
  const int st = kBlock ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x & 31);
  const int snt = kBlock ? static_cast<int>(blockDim.x) : 32;
  const int64_t unit = kBlock ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t units = kBlock ? gridDim.x : static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  const int32_t n8 = (a.cols + 7) >> 3;
  const T* dy = static_cast<const T*>(a.dy);
  const T* h = static_cast<const T*>(a.h);
  const T* dh = static_cast<const T*>(a.dh);
  PhiloxKey key{};
  if (a.drop.thr > 0) key = philox_key(a.drop.rng);
  const uint32_t one = span_stage<T>(kRows, a.cols), stage = (dh != nullptr ? 3 : 2) * one;
  uint8_t* mine = bufs + (kBlock ? 0 : (threadIdx.x >> 5) * STAGES * stage);
  uint64_t w[CH][4], dw[CH][4], db[CH][4];   // pairs of columns
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int32_t ch = lane + k * step;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[k][i] = both(1.f);
      dw[k][i] = 0;
      db[k][i] = 0;
    }
    if (a.weight != nullptr && ch < n8)
      load_param2<T>(a.weight, a.wfp32, ch * 8, min(8, a.cols - ch * 8), w[k]);
  }
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  auto rows_at = [&](int64_t base) { return static_cast<int>(min(static_cast<int64_t>(kRows), a.rows - base)); };
  auto fetch = [&](int64_t base, int slot) {   // the step that starts at row `base`, if there is one
    if (base < a.rows) {
      const int n = rows_at(base) * a.cols;
      uint8_t* p = mine + slot * stage;
      span_load(p, dy + base * a.cols, n, st, snt);
      span_load(p + one, h + base * a.cols, n, st, snt);
      if (dh != nullptr) span_load(p + 2 * one, dh + base * a.cols, n, st, snt);
    }
    span_commit();
  };
  float mean[R], rstd[R];
  auto fetch_stats = [&](int64_t base) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = base + r * kGroups + grp;
      mean[r] = row < a.rows ? __ldg(a.mean + row) : 0.f;
      rstd[r] = row < a.rows ? __ldg(a.rstd + row) : 0.f;
    }
  };
  int64_t ahead = unit * kRows;
  fetch_stats(ahead);
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i, ahead += units * kRows) fetch(ahead, i);
  int par = 0, slot = 0;
  // every thread of a warp (block) makes the same number of steps: the sums synchronise
  for (int64_t base = unit * kRows; base < a.rows; base += units * kRows, ahead += units * kRows, par ^= 1) {
    fetch(ahead, slot == 0 ? STAGES - 1 : slot - 1);
    span_wait<STAGES - 1>();
    span_sync<kBlock>();
    const int live = rows_at(base);
    uint8_t* p = mine + slot * stage;
    const T *ey = span_elems(p, dy + base * a.cols), *ez = span_elems(p + one, h + base * a.cols);
    uint64_t g[R][CH][4], z[R][CH][4];
    float rs[R], c1[R], c2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t nm = both(-mean[r]), rs2 = both(rstd[r]);
      uint64_t s1[2] = {0, 0}, s2[2] = {0, 0};
      rs[r] = rstd[r];
      const int q = r * kGroups + grp;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c0 = (lane + k * step) * 8, e0 = q * a.cols + c0, n = q < live ? a.cols - c0 : 0;
        span_get<T, TPR == 1>(ey, e0, n, g[r][k]);
        span_get<T, TPR == 1>(ez, e0, n, z[r][k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t y = g[r][k][i];
          z[r][k][i] = mul_f32x2(add_f32x2(z[r][k][i], nm), rs2);
          dw[k][i] = fma_f32x2(y, z[r][k][i], dw[k][i]);
          db[k][i] = add_f32x2(db[k][i], y);
          g[r][k][i] = mul_f32x2(y, w[k][i]);
          s1[i & 1] = add_f32x2(s1[i & 1], g[r][k][i]);
          s2[i & 1] = fma_f32x2(g[r][k][i], z[r][k][i], s2[i & 1]);
        }
      }
      c1[r] = sum_f32x2(add_f32x2(s1[0], s1[1]));
      c2[r] = sum_f32x2(add_f32x2(s2[0], s2[1]));
    }
    fetch_stats(base + units * kRows);
#pragma unroll
    for (int r = 0; r < R; ++r) row_sum2<TPR>(c1[r], c2[r], red[par][r]);
    const T* ed = span_elems(p + 2 * one, dh + base * a.cols);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t n1 = both(-c1[r] * inv_n), n2 = both(-c2[r] * inv_n), rs2 = both(rs[r]);
#pragma unroll
      for (int k = 0; k < CH; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          g[r][k][i] = mul_f32x2(fma_f32x2(z[r][k][i], n2, add_f32x2(g[r][k][i], n1)), rs2);
        if (dh != nullptr) {
          const int q = r * kGroups + grp, c0 = (lane + k * step) * 8;
          uint64_t d2[4];
          span_get<T, TPR == 1>(ed, q * a.cols + c0, q < live ? a.cols - c0 : 0, d2);
#pragma unroll
          for (int i = 0; i < 4; ++i) g[r][k][i] = add_f32x2(g[r][k][i], d2[i]);
        }
      }
    }
    // dresidual as it is, dx through the mask
#pragma unroll
    for (int out = 0; out < 2; ++out) {
      T* dst = static_cast<T*>(out == 0 ? a.dres : a.dx);
      if (dst == nullptr) continue;
      span_sync<kBlock>();   // the slot's values are in registers (or stored): it carries the output
      // long rows lie on boundaries of their own (row_put), shorter ones as the span
      T* eo = span_elems(p, dst + base * a.cols);
      const uint32_t pitch = static_cast<uint32_t>(n8) * 8 * sizeof(T);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int q = r * kGroups + grp;
        if (q >= live) continue;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int32_t ch = lane + k * step;
          if (ch >= n8) continue;
          uint64_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = g[r][k][i];
          if (out == 1 && a.drop.thr > 0) drop_pairs(v, static_cast<uint64_t>(base + q) * n8 + ch, key, a.drop);
          if constexpr (kOwnRows) {
            row_put<T>(static_cast<uint32_t>(__cvta_generic_to_shared(p)) + q * pitch + ch * 8 * sizeof(T), v);
          } else {
            const int n = min(8, a.cols - ch * 8);
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
    span_sync<kBlock>();   // every thread is done with the slot: the next step's fetch fills it
    slot = slot + 1 == STAGES ? 0 : slot + 1;
  }
  span_wait<0>();
  store_column_sums<TPR, CH>(a, dw, db, lane, step);
}

// The same for rows of a multiple of eight columns (see Own).
// DROP: with dropout, whose generator takes registers that the other calls use for more warps.
template <typename T, bool DROP, int TPR, int CH, int R, int STAGES>
__global__ void __launch_bounds__(TPR > 0 ? 256 : CH * R == 4 ? 384 : 512, TPR > 0 && CH <= 2 ? 2 : 1) norm_bwd_vec_kernel(const NormBwdArgs a) {
  constexpr bool kBlock = TPR == 0;
  constexpr int kGroups = kBlock ? 1 : 32 / (TPR > 0 ? TPR : 1);
  constexpr int kRows = kGroups * R;   // rows of a warp's (block's) step
  constexpr int kParts = Own<T>::kParts;
  constexpr int kChunkBytes = 16 * kParts;
  __shared__ float2 red[2][R][32];
  extern __shared__ __align__(16) uint8_t bufs[];
  const int lane = kBlock ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x & 31) % (TPR > 0 ? TPR : 1);
  const int grp = kBlock ? 0 : static_cast<int>(threadIdx.x & 31) / (TPR > 0 ? TPR : 1);
  const int step = kBlock ? static_cast<int>(blockDim.x) : TPR;
  const uint32_t part = 16u * (kBlock ? blockDim.x : 256u);
  const int64_t unit = kBlock ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t units = kBlock ? gridDim.x : static_cast<int64_t>(gridDim.x) * 8;
  const int32_t n8 = a.cols >> 3;
  const bool has_dh = a.dh != nullptr;
  const uint32_t arr = static_cast<uint32_t>(R * CH * kParts) * part;   // one array of one stage
  const uint32_t stage = (has_dh ? 3 : 2) * arr;
  const uint32_t sm = static_cast<uint32_t>(__cvta_generic_to_shared(bufs)) + 16 * threadIdx.x;
  PhiloxKey key{};
  if (DROP) key = philox_key(a.drop.rng);
  uint64_t w[CH][4], dw[CH][4], db[CH][4];   // pairs of columns
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int32_t ch = lane + k * step;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[k][i] = both(1.f);
      dw[k][i] = 0;
      db[k][i] = 0;
    }
    if (a.weight != nullptr && ch < n8)
      read_param2<T>(static_cast<const char*>(a.weight) + ch * (a.wfp32 ? 32 : 8 * static_cast<int>(sizeof(T))), a.wfp32, w[k]);
  }
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  const int64_t row_bytes = static_cast<int64_t>(a.cols) * sizeof(T);
  const int64_t step_bytes = units * kRows * row_bytes, r_bytes = kGroups * row_bytes;
  const int k_bytes = step * kChunkBytes;
  const int64_t row0 = unit * kRows + grp, off0 = row0 * row_bytes + lane * kChunkBytes;   // see the forward
  const int64_t step_rows = units * kRows;
  const char *py = static_cast<const char*>(a.dy) + off0, *pz = static_cast<const char*>(a.h) + off0,
             *pd = static_cast<const char*>(a.dh) + off0;
  int64_t left_in = a.rows - row0;
  auto fetch = [&](uint32_t at) {
    const int left = static_cast<int>(left_in < 4096 ? left_in : 4096);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        // what does not exist reads as zero and adds nothing to any sum
        const bool ok = r * kGroups < left && lane + k * step < n8;
        const int64_t o = ok ? r * r_bytes + k * k_bytes : 0;
        const uint32_t d = at + static_cast<uint32_t>((r * CH + k) * kParts) * part;
        Own<T>::copy_or_zero(d, part, (ok ? py : static_cast<const char*>(a.dy)) + o, ok);
        Own<T>::copy_or_zero(d + arr, part, (ok ? pz : static_cast<const char*>(a.h)) + o, ok);
        if (has_dh) Own<T>::copy_or_zero(d + 2 * arr, part, (ok ? pd : static_cast<const char*>(a.dh)) + o, ok);
      }
    span_commit();
    left_in -= step_rows;
    py += step_bytes;
    pz += step_bytes;
    pd += step_bytes;
  };
  int64_t row = row0, left64 = left_in;
  char *po = static_cast<char*>(a.dres) + off0, *px = static_cast<char*>(a.dx) + off0;
  float mean[R], rstd[R];
  auto fetch_stats = [&](int64_t first) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t q = first + r * kGroups;
      mean[r] = q < a.rows ? __ldg(a.mean + q) : 0.f;
      rstd[r] = q < a.rows ? __ldg(a.rstd + q) : 0.f;
    }
  };
  fetch_stats(row);
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(sm + i * stage);
  uint32_t cur = 0;
  int par = 0;
  // every thread of a warp (block) makes the same number of steps: the sums synchronise
  for (int64_t base = unit * kRows; base < a.rows; base += step_rows, par ^= 1) {
    const int left = static_cast<int>(left64 < 4096 ? left64 : 4096);
    fetch(sm + (cur == 0 ? (STAGES - 1) * stage : cur - stage));
    span_wait<STAGES - 1>();
    uint64_t g[R][CH][4], z[R][CH][4];
    float rs[R], c1[R], c2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t nm = both(-mean[r]), rs2 = both(rstd[r]);
      uint64_t s1[2] = {0, 0}, s2[2] = {0, 0};
      rs[r] = rstd[r];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const uint32_t d = sm + cur + static_cast<uint32_t>((r * CH + k) * kParts) * part;
        Own<T>::read(d, part, g[r][k]);
        Own<T>::read(d + arr, part, z[r][k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t y = g[r][k][i];
          z[r][k][i] = mul_f32x2(add_f32x2(z[r][k][i], nm), rs2);
          dw[k][i] = fma_f32x2(y, z[r][k][i], dw[k][i]);
          db[k][i] = add_f32x2(db[k][i], y);
          g[r][k][i] = mul_f32x2(y, w[k][i]);
          s1[i & 1] = add_f32x2(s1[i & 1], g[r][k][i]);
          s2[i & 1] = fma_f32x2(g[r][k][i], z[r][k][i], s2[i & 1]);
        }
      }
      c1[r] = sum_f32x2(add_f32x2(s1[0], s1[1]));
      c2[r] = sum_f32x2(add_f32x2(s2[0], s2[1]));
    }
    fetch_stats(row + step_rows);
#pragma unroll
    for (int r = 0; r < R; ++r) row_sum2<TPR>(c1[r], c2[r], red[par][r]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t n1 = both(-c1[r] * inv_n), n2 = both(-c2[r] * inv_n), rs2 = both(rs[r]);
#pragma unroll
      for (int k = 0; k < CH; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          g[r][k][i] = mul_f32x2(fma_f32x2(z[r][k][i], n2, add_f32x2(g[r][k][i], n1)), rs2);
        if (has_dh) {
          uint64_t d2[4];
          Own<T>::read(sm + cur + 2 * arr + static_cast<uint32_t>((r * CH + k) * kParts) * part, part, d2);
#pragma unroll
          for (int i = 0; i < 4; ++i) g[r][k][i] = add_f32x2(g[r][k][i], d2[i]);
        }
        if (r * kGroups < left && lane + k * step < n8) {
          if (a.dres != nullptr) Own<T>::write(po + r * r_bytes + k * k_bytes, g[r][k]);
          if (a.dx != nullptr) {
            if (DROP)
              drop_pairs(g[r][k], static_cast<uint64_t>(row + r * kGroups) * n8 + (lane + k * step), key, a.drop);
            Own<T>::write(px + r * r_bytes + k * k_bytes, g[r][k]);
          }
        }
      }
    }
    cur = cur + stage == STAGES * stage ? 0 : cur + stage;
    left64 -= step_rows;
    row += step_rows;
    po += step_bytes;
    px += step_bytes;
  }
  span_wait<0>();
  store_column_sums<TPR, CH>(a, dw, db, lane, step);
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

// Launch shape of the first kernel: threads that share a row (0: the block), chunks of a
// thread, rows of a block's step, threads of a block, blocks.  It depends on the sizes, the type
// and whether dh is given, and so do the parts and the sums' order.  No more blocks than an SM
// holds, by registers here (128 a thread, 168 where a thread has two chunks of two rows) and by shared
// memory in launch_bwd: fp32 warps with their stages of two or three arrays often fill an SM with one
// block, and a grid of two waves took 1 to 4 % longer (937 500 x 64 with dh 163 and 158 us).
// Rates of plain calls over
// 170 M elements and of calls with every option over 85 M, in GB/s:
//   1024 columns: a warp a row, one block an SM: bf16 6000 and 5880, fp32 5700 and 4930; a block a
//   row: 5390 and 4800, 5980 and 4510;
//   bf16 blocks: two chunks and two rows 6100 and 4870 at 1536 columns, 5160 and 4590 at 4096; one
//   chunk and two rows 5220 and 4870, 5210 and 4750;
//   fp32 blocks: one chunk and two rows 6230 and 5490 at 1536 columns, 5230 and 4650 at 4096; two
//   chunks of one row 5440 and 5740, 5860 and 5430; two and two 4090 and 3540 at 1536;
//   odd widths, blocks: two rows 2190 and 3390 at 1153 columns, 2380 and 3310 at 2001; four 2080 and
//   3230, 2210 and 2450;
//   above 4096 columns: one block an SM 4570 and fp32 5690 at 5120 columns, two 4380 and 5440.
struct BwdShape {
  int tpr, ch, rows, threads;
  int64_t blocks;
};

BwdShape bwd_shape(int64_t rows, int32_t cols, bool fp32) {
  const int n8 = (cols + 7) >> 3;
  const bool vec = (cols & 7) == 0;
  BwdShape s{};
  s.tpr = n8 <= 1 ? 1 : n8 <= 4 ? 2 : n8 <= 8 ? 4 : n8 <= 16 ? 8 : n8 <= 32 ? 16 : n8 <= (vec ? 128 : 64) ? 32 : 0;
  int per_sm;
  int64_t block_rows;
  if (s.tpr > 0) {
    s.ch = n8 <= 1 ? 1 : n8 <= 64 ? 2 : 4;
    s.rows = 1;
    s.threads = 256;
    block_rows = static_cast<int64_t>(256 / s.tpr);
    per_sm = s.ch <= 2 ? 2 : 1;
  } else {
    if (n8 > 512) {
      s.ch = 2;
      s.rows = 1;
    } else if (!vec) {
      s.ch = 1;
      s.rows = 2;
    } else {
      s.ch = fp32 && n8 <= 256 ? 1 : 2;
      s.rows = fp32 && n8 > 256 ? 1 : 2;
    }
    s.threads = ((n8 + s.ch - 1) / s.ch + 31) / 32 * 32;
    block_rows = s.rows;
    per_sm = n8 > 512 ? 1 : (s.ch * s.rows == 4 && vec ? 384 : 512) / s.threads;
    if (per_sm < 1) per_sm = 1;
  }
  const int64_t need = (rows + block_rows - 1) / block_rows;
  s.blocks = need < 148 * per_sm ? need : 148 * per_sm;
  return s;
}

template <typename T, bool VEC, int TPR, int CH, int R, int STAGES>
cudaError_t launch_bwd(const NormBwdArgs& a, BwdShape& s, cudaStream_t stream) {
  void (*kern)(NormBwdArgs);
  if constexpr (VEC)
    kern = a.drop.thr > 0 ? norm_bwd_vec_kernel<T, true, TPR, CH, R, STAGES>
                          : norm_bwd_vec_kernel<T, false, TPR, CH, R, STAGES>;
  else
    kern = norm_bwd_kernel<T, TPR, CH, R, STAGES>;
  constexpr int rows = (TPR > 0 ? 32 / (TPR > 0 ? TPR : 1) : 1) * R;
  const int units = TPR > 0 ? s.threads / 32 : 1;
  const int stage = VEC ? R * CH * s.threads * 8 * static_cast<int>(sizeof(T))
                        : units * static_cast<int>(span_stage<T>(rows, a.cols));
  const int smem = STAGES * (a.dh != nullptr ? 3 : 2) * stage + (VEC ? 0 : kSpanSlack);
  constexpr int fixed = 2 * R * 32 * 8 + (TPR > 0 ? 8 * 32 * CH * 8 * 4 : 0);   // red and acc
  const int fit = kSmemSm / (smem + fixed + kSmemBlock);
  if (s.blocks > 148 * fit) s.blocks = 148 * fit;
  const cudaError_t e = allow_smem(kern, fixed);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(s.blocks), s.threads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t bwd_t(const NormBwdArgs& a, cudaStream_t stream) {
  BwdShape s = bwd_shape(a.rows, a.cols, sizeof(T) == 4);
  if (a.rows > 0) {
    cudaError_t e;
    switch (s.tpr) {
      case 1: e = launch_bwd<T, VEC, 1, 1, 1, 4>(a, s, stream); break;
      case 2: e = launch_bwd<T, VEC, 2, 2, 1, 4>(a, s, stream); break;
      case 4: e = launch_bwd<T, VEC, 4, 2, 1, 4>(a, s, stream); break;
      // three stages: 6080 and 5130 plain, 5290 and 5910 with every option; four: 5900 and 5870, 5020 and 4450
      case 8: e = launch_bwd<T, VEC, 8, 2, 1, 3>(a, s, stream); break;
      case 16: e = launch_bwd<T, VEC, 16, 2, 1, 4>(a, s, stream); break;
      case 32:
        if constexpr (VEC) {
          if (s.ch == 4) {
            e = launch_bwd<T, VEC, 32, 4, 1, 2>(a, s, stream);
            break;
          }
        }
        e = launch_bwd<T, VEC, 32, 2, 1, 4>(a, s, stream);
        break;
      default:
        if (s.ch == 2 && s.rows == 1) {
          e = launch_bwd<T, VEC, 0, 2, 1, 2>(a, s, stream);
        } else if constexpr (!VEC || sizeof(T) == 4) {
          e = launch_bwd<T, VEC, 0, 1, 2, 2>(a, s, stream);
        } else {
          e = launch_bwd<T, VEC, 0, 2, 2, 2>(a, s, stream);
        }
    }
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

int norm_bwd_parts(int64_t rows, int32_t cols) {
  const int64_t a = bwd_shape(rows, cols, false).blocks, b = bwd_shape(rows, cols, true).blocks;
  return static_cast<int>(a > b ? a : b);
}

cudaError_t launch_norm_bwd(int dtype, const NormBwdArgs& a, cudaStream_t stream) {
  const bool vec = (a.cols & 7) == 0;
  switch (dtype) {
    case 0: return vec ? bwd_t<__nv_bfloat16, true>(a, stream) : bwd_t<__nv_bfloat16, false>(a, stream);
    case 1: return vec ? bwd_t<__half, true>(a, stream) : bwd_t<__half, false>(a, stream);
    default: return vec ? bwd_t<float, true>(a, stream) : bwd_t<float, false>(a, stream);
  }
}

}  // namespace sta
