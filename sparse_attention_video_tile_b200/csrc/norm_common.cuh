// norm_common.cuh - loads, stores and sums shared by the layer norm and dropout kernels.
//
// A row is cut into chunks of eight columns, the unit of one generator block; a
// thread holds CH chunks of a row in registers as fp32.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "norm.h"
#include "packed.cuh"
#include "philox.cuh"
#include "ptx.cuh"

namespace sta {
namespace norm {

using ptx::add_f32x2;
using ptx::f32x2;
using ptx::f32x2_split;
using ptx::fma_f32x2;
using ptx::mul_f32x2;

__device__ __forceinline__ uint64_t both(float v) { return f32x2(v, v); }
__device__ __forceinline__ float sum_f32x2(uint64_t v) {
  float a, b;
  f32x2_split(v, a, b);
  return a + b;
}

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
// one rounding, to nearest even
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ uint4 ld_once(const void* p) {   // read once: no place in L1
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Eight columns as they lie in memory: 16 bytes (bf16, fp16) or 32 (fp32).
template <typename T>
struct Chunk {
  static constexpr int kWords = static_cast<int>(sizeof(T)) * 2;   // 32-bit words
  uint32_t w[kWords];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // aligned: the eight columns exist and lie on a 16-byte boundary
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 v = ld_once(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  }
  // any alignment; columns n .. 7 read as zero
  __device__ __forceinline__ void load_n(const T* p, int n) {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : from_f<T>(0.f);
    set(e);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  __device__ __forceinline__ void store_n(T* p, int n) const {
    T e[8];
    get_t(e);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = e[i];
  }
  __device__ __forceinline__ void get_t(T (&e)[8]) const;
  __device__ __forceinline__ void set(const T (&e)[8]);
  // to fp32, and from fp32 with one rounding (two at a time: the packed conversions run at
  // several times the rate of single ones, which bounded these kernels otherwise)
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        f[2 * i] = __uint_as_float(w[2 * i]);
        f[2 * i + 1] = __uint_as_float(w[2 * i + 1]);
      } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    }
  }
  // pairs of columns: the arithmetic runs on packed fp32 (half the instructions, which
  // bound these kernels where memory does not)
  __device__ __forceinline__ void get2(uint64_t (&f)[4]) const {
    float v[8];
    get(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f32x2(v[2 * i], v[2 * i + 1]);
  }
  __device__ __forceinline__ void put2(const uint64_t (&f)[4]) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f32x2_split(f[i], v[2 * i], v[2 * i + 1]);
    put(v);
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[2 * i] = __float_as_uint(f[2 * i]);
        w[2 * i + 1] = __float_as_uint(f[2 * i + 1]);
      } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      } else {
        const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ uint32_t bits16(T v) {
  return *reinterpret_cast<const uint16_t*>(&v);
}
template <typename T>
__device__ __forceinline__ T from_bits16(uint32_t b) {
  const uint16_t s = static_cast<uint16_t>(b);
  return *reinterpret_cast<const T*>(&s);
}
template <typename T>
__device__ __forceinline__ void Chunk<T>::get_t(T (&e)[8]) const {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[2 * i] = from_bits16<T>(w[i] & 0xFFFFu);
      e[2 * i + 1] = from_bits16<T>(w[i] >> 16);
    }
  }
}
template <typename T>
__device__ __forceinline__ void Chunk<T>::set(const T (&e)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bits16(e[2 * i]) | (bits16(e[2 * i + 1]) << 16);
  }
}

// Consecutive rows are one span of memory.  A span is copied to shared memory ahead of its
// use, in 16-byte asynchronous copies that need no registers, and (rows whose length is no
// multiple of eight start anywhere) back from there: in aligned blocks, at the same offset
// inside a block on both sides; the copy back goes element by element in a block that the
// span does not fill.  Element i of a span whose global address is g lies at buf + (g mod 16) + i size.
template <typename T>
__host__ __device__ constexpr uint32_t span_bytes(uint32_t n) {
  return (n * static_cast<uint32_t>(sizeof(T)) + 15) / 16 * 16 + 16;
}
// A stage of one array: the span of `rows` rows, or the rows on boundaries of their own (row_put).
template <typename T>
__host__ __device__ constexpr uint32_t span_stage(uint32_t rows, uint32_t cols) {
  const uint32_t a = span_bytes<T>(rows * cols), b = rows * ((cols + 7) / 8 * 8) * static_cast<uint32_t>(sizeof(T));
  return a > b ? a : b;
}
template <typename T>
__device__ __forceinline__ T* span_elems(uint8_t* buf, const T* g) {
  return reinterpret_cast<T*>(buf + (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(g)) & 15u));
}
// Starts the copy of n elements from g, by threads t, t + nt, ... (commit and wait by the caller).
template <typename T>
__device__ __forceinline__ void span_load(uint8_t* buf, const T* g, int n, int t, int nt) {
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(g)) & 15u;
  const uint32_t end = off + static_cast<uint32_t>(n) * sizeof(T);
  const uint8_t* base = reinterpret_cast<const uint8_t*>(g) - off;
  const uint32_t sbuf = static_cast<uint32_t>(__cvta_generic_to_shared(buf));
  for (uint32_t b = static_cast<uint32_t>(t) * 16; b < end; b += static_cast<uint32_t>(nt) * 16) {
    // what lies before the span in its first block belongs to the same array, whose start is aligned;
    // nothing is read behind the span
    const uint32_t size = end - b < 16u ? end - b : 16u;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sbuf + b), "l"(base + b), "r"(size) : "memory");
  }
}
__device__ __forceinline__ void span_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void span_wait() {   // all but this thread's last N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <typename T>
__device__ __forceinline__ void span_store(const uint8_t* buf, T* g, int n, int t, int nt) {
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(g)) & 15u;
  const uint32_t end = off + static_cast<uint32_t>(n) * sizeof(T);
  uint8_t* base = reinterpret_cast<uint8_t*>(g) - off;
  for (uint32_t b = static_cast<uint32_t>(t) * 16; b < end; b += static_cast<uint32_t>(nt) * 16) {
    if (b >= off && b + 16 <= end) {
      *reinterpret_cast<uint4*>(base + b) = *reinterpret_cast<const uint4*>(buf + b);
    } else {
      const uint32_t lo = b < off ? off : b, hi = b + 16 < end ? b + 16 : end;
      for (uint32_t x = lo; x < hi; x += sizeof(T)) *reinterpret_cast<T*>(base + x) = *reinterpret_cast<const T*>(buf + x);
    }
  }
}
// 16 bytes of shared memory, at an address of a multiple of 16.
__device__ __forceinline__ uint4 smem_read16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}
__device__ __forceinline__ void smem_write16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// N words from shared address `at`, a multiple of the element size (2 or 4): whole 16-byte blocks
// are read, and the words moved into place in registers.  Element by element the accesses
// conflict four ways (16 bytes a lane) or eight (32): forward at 4001 columns bf16 2350 GB/s
// this way and 2010 that way, backward at 257 fp32 2260 and 2030.  Reads up to 16 bytes past the
// last word's block.
template <int N, bool HALVES>
__device__ __forceinline__ void smem_words(uint32_t at, uint32_t (&o)[N]) {
  const uint32_t off = at & 15u;
  uint32_t w[N + 4];
#pragma unroll
  for (int i = 0; i < N / 4 + 1; ++i) {
    const uint4 v = smem_read16(at - off + 16 * i);
    w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < N + 2; ++i) w[i] = off & 8u ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < N + 1; ++i) w[i] = off & 4u ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = HALVES ? __funnelshift_r(w[i], w[i + 1], (off & 2u) * 8) : w[i];
}
// Bytes of shared memory that such reads may touch past the last stage.
constexpr int kSpanSlack = 64;
// Eight elements of a span from e0 on, as pairs of fp32; those from n on read as zero.  Rows of
// less than eight columns are read by elements, 8 % faster there.
template <typename T, bool SHORT>
__device__ __forceinline__ void span_get(const T* e, int e0, int n, uint64_t (&f)[4]) {
  if constexpr (SHORT) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = f32x2(2 * i < n ? to_f<T>(e[e0 + 2 * i]) : 0.f, 2 * i + 1 < n ? to_f<T>(e[e0 + 2 * i + 1]) : 0.f);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = 0;
  if (n <= 0) return;
  Chunk<T> c;
  smem_words<Chunk<T>::kWords, sizeof(T) == 2>(static_cast<uint32_t>(__cvta_generic_to_shared(e + e0)), c.w);
  c.get2(f);
  if (n >= 8) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float u, v;
    f32x2_split(f[i], u, v);
    f[i] = f32x2(2 * i < n ? u : 0.f, 2 * i + 1 < n ? v : 0.f);
  }
}
// Output rows: each lies on a 16-byte boundary of shared memory (pitch n8 chunks), its chunks
// written whole, and goes out in the 16-byte blocks of its place in memory, element by
// element only at its two ends.  Long rows only: forward at 1153 columns 2000 GB/s (as a span
// 1710; fp32 3300 and 2520), at 121 2630 (2820; fp32 2730 and 4390); backward at 257 columns 1390
// (1260; fp32 2440 and 2260), at 57 2120 (2400; fp32 2270 and 2670).
template <typename T>
__device__ __forceinline__ void row_put(uint32_t at, const uint64_t (&f)[4]) {
  Chunk<T> c;
  c.put2(f);
#pragma unroll
  for (int i = 0; i < Chunk<T>::kWords / 4; ++i) smem_write16(at + 16 * i, c.w[4 * i], c.w[4 * i + 1], c.w[4 * i + 2], c.w[4 * i + 3]);
}
template <typename T>
__device__ __forceinline__ void row_store(const uint8_t* buf, T* g, int cols, int t, int nt) {
  constexpr int kSize = static_cast<int>(sizeof(T));
  const int bytes = cols * kSize;
  const int head = min((16 - static_cast<int>(reinterpret_cast<uintptr_t>(g) & 15u)) & 15, bytes), full = (bytes - head) >> 4;
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(buf)) + head;
  uint8_t* base = reinterpret_cast<uint8_t*>(g) + head;
  for (int j = t; j < full; j += nt) {
    uint32_t o[4];
    smem_words<4, sizeof(T) == 2>(at + 16 * j, o);
    *reinterpret_cast<uint4*>(base + 16 * j) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  const T* e = reinterpret_cast<const T*>(buf);
  for (int x = t; x < head / kSize; x += nt) g[x] = e[x];
  for (int x = (head + 16 * full) / kSize + t; x < cols; x += nt) g[x] = e[x];
}
// Pairs through the dropout mask.  Dropped values are replaced, not multiplied by zero: an
// infinity or NaN there stays out.
__device__ __forceinline__ void drop_pairs(uint64_t (&f)[4], uint64_t block, const PhiloxKey& key, const NormDropout& d) {
  const uint32_t keep = philox_keep(philox_block(block, key), d.thr);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float u, v;
    f32x2_split(f[i], u, v);
    f[i] = f32x2((keep >> (2 * i)) & 1u ? u * d.scale : 0.f, (keep >> (2 * i + 1)) & 1u ? v * d.scale : 0.f);
  }
}

// Rows of a multiple of eight columns: every chunk is aligned, and a thread copies the
// chunks it will use itself, ahead of their use, into places of its own in shared memory
// (16 bytes of each thread side by side).  No other thread reads them, so waiting for its
// own copies is all a thread needs.
// 16 bytes where `ok`; otherwise zeros (src is then any valid address and is not read).
// L1: through the L1 cache, for chunks of two parts (fp32).  Each of the two copies then
// touches half of every 32-byte sector, and the second finds the sector in L1; past L1 both
// fetch it from L2 (backward at 163 840 x 512 fp32: 4060 GB/s past L1, 5950 through it).
template <bool L1>
__device__ __forceinline__ void own_copy_or_zero(uint32_t dst, const void* src, bool ok) {
  if constexpr (L1)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16u : 0u) : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16u : 0u) : "memory");
}
// A chunk is kParts 16-byte parts; part p of chunk i of a stage lies at (i kParts + p) 16 threads + 16 thread.
template <typename T>
struct Own {
  static constexpr int kParts = static_cast<int>(sizeof(T)) / 2;
  static __device__ __forceinline__ void copy_or_zero(uint32_t at, uint32_t part, const char* src, bool ok) {
#pragma unroll
    for (int p = 0; p < kParts; ++p) own_copy_or_zero<(kParts > 1)>(at + p * part, src + 16 * p, ok);
  }
  static __device__ __forceinline__ void read(uint32_t at, uint32_t part, uint64_t (&f)[4]) {
    Chunk<T> c;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const uint4 v = smem_read16(at + p * part);
      c.w[4 * p] = v.x; c.w[4 * p + 1] = v.y; c.w[4 * p + 2] = v.z; c.w[4 * p + 3] = v.w;
    }
    c.get2(f);
  }
  static __device__ __forceinline__ void write(char* dst, const uint64_t (&f)[4]) {
    Chunk<T> c;
    c.put2(f);
    c.store(reinterpret_cast<T*>(dst));
  }
};

// Allows a kernel all the dynamic shared memory that a block can have beside its static arrays
// (at most `fixed` bytes).  The attribute belongs to the process, so every call sets the same
// value, whatever it will use itself: with the call's own size, a call from another thread
// could lower it between this thread's setting and its launch, which was then refused.
constexpr int kSmemOptin = 227 * 1024;   // sm_100: a block's static and dynamic bytes
constexpr int kSmemSm = 228 * 1024, kSmemBlock = 1024;   // an SM's, and what it takes of them for a block
template <typename F>
inline cudaError_t allow_smem(F* kern, int fixed) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOptin - fixed);
}

// Barrier of the threads that share a span: a warp, or the block.
template <bool BLOCK>
__device__ __forceinline__ void span_sync() {
  if (BLOCK) __syncthreads(); else __syncwarp();
}

// The eight parameters at p, an address in an array of `fp32` or T elements.
template <typename T>
__device__ __forceinline__ void read_param2(const char* p, bool fp32, uint64_t (&f)[4]) {
  if (fp32) {
    const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2*>(p)), b = __ldg(reinterpret_cast<const ulonglong2*>(p) + 1);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
  } else {
    Chunk<T> k;
#pragma unroll
    for (int i = 0; i < Chunk<T>::kWords / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
      k.w[4 * i] = v.x; k.w[4 * i + 1] = v.y; k.w[4 * i + 2] = v.z; k.w[4 * i + 3] = v.w;
    }
    k.get2(f);
  }
}
// Parameters c .. c + 7 of the weight or bias, n of which exist (the rest read as zero).
template <typename T>
__device__ __forceinline__ void load_param2(const void* p, bool fp32, int32_t c, int n, uint64_t (&f)[4]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = i < n ? (fp32 ? static_cast<const float*>(p)[c + i] : to_f<T>(static_cast<const T*>(p)[c + i])) : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f32x2(v[2 * i], v[2 * i + 1]);
}

// Sum over the TPR threads that share a row (TPR = 0: the whole block, through `red`,
// which holds 32 floats; every thread of the block calls it).  One barrier: successive
// calls take two buffers in turn, so that a buffer is written again only after the other
// call's barrier.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  if constexpr (TPR > 0) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = static_cast<int>(blockDim.x) >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = static_cast<int>(threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  }
}

}  // namespace norm
}  // namespace sta
