// norm_common.cuh - loads, stores and sums shared by the layer norm and dropout kernels.
//
// A row is cut into chunks of eight columns, the unit of one generator block; a
// thread holds CH chunks of a row in registers as fp32.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "norm.h"
#include "philox.cuh"

namespace sta {
namespace norm {

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
  __device__ __forceinline__ void get(float (&f)[8]) const {
    T e[8];
    get_t(e);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_f<T>(e[i]);
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f<T>(f[i]);
    set(e);
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

// Columns c .. c + 7 of the weight or bias as fp32 (n of them exist; the rest read as zero).
template <typename T, bool VEC>
__device__ __forceinline__ void load_param(const void* p, bool fp32, int32_t c, int n, float (&f)[8]) {
  if constexpr (VEC) {
    if (fp32) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + c);
      const float4 a = __ldg(q), b = __ldg(q + 1);
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
      Chunk<T> k;
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(p) + c);
#pragma unroll
      for (int i = 0; i < Chunk<T>::kWords / 4; ++i) {
        const uint4 v = __ldg(q + i);
        k.w[4 * i] = v.x; k.w[4 * i + 1] = v.y; k.w[4 * i + 2] = v.z; k.w[4 * i + 3] = v.w;
      }
      k.get(f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = i < n ? (fp32 ? static_cast<const float*>(p)[c + i] : to_f<T>(static_cast<const T*>(p)[c + i])) : 0.f;
  }
}

// Sum over the TPR threads that share a row (TPR = 0: the whole block, through `red`,
// which holds 32 floats; every thread of the block calls it).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  if constexpr (TPR > 0) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  } else {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = static_cast<int>(blockDim.x) >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = static_cast<int>(threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    return s;
  }
}

}  // namespace norm
}  // namespace sta
