// diff_common.cuh - window walk, tensor maps and row addressing shared by the
// differential attention kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "diff.h"
#include "ptx.cuh"

namespace sta {
namespace diff {

using namespace ptx;

// Orders generic-proxy writes of shared memory before the async proxy's (MMA) reads.
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Three-input maximum that keeps a NaN.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// slabs with real tokens of the tiles at temporal index t
__device__ __forceinline__ int32_t slabs_at(const DiffGeo& g, int32_t t) { return t == g.nT - 1 ? g.slabs_last : g.slabs; }

// One unit of work: a 128-row block (slab s of tile (t, h, w)) of one (batch, head), and
// the box of tiles it is multiplied with.
struct Item {
  int32_t b, head, bh;
  int32_t t, h, w, s;            // own tile and slab
  int32_t bt0, bh0, bw0;         // box of tiles: start
  int32_t ent, enh, enw;         // box of tiles: extent
  int32_t n;                     // 128-row blocks with real tokens in the box
};

// Box of key tiles that query tile `a` attends: s = clamp(a - w / 2, 0, n - w), extent w.
__device__ __forceinline__ void key_range(int32_t a, int32_t w, int32_t n, int32_t& s, int32_t& e) {
  s = min(max(a - w / 2, 0), n - w);
  e = w;
}
// Box of query tiles that attend key tile `c`: the start above never decreases with a, so
// they are consecutive.  The first is 0 where the first window covers c, else the a whose
// window ends at c; the last is n - 1 where the last window covers c, else the a whose
// window starts at c.
__device__ __forceinline__ void query_range(int32_t c, int32_t w, int32_t n, int32_t& s, int32_t& e) {
  s = c < w ? 0 : c - w + 1 + w / 2;
  const int32_t last = c >= n - w ? n - 1 : c + w / 2;
  e = last - s + 1;
}

// Item `idx` (0 .. batch * heads * blocks - 1); KEYS: own block is a key block and the
// box holds query tiles.  Neighbouring items are neighbouring blocks of one head.
template <bool KEYS>
__device__ __forceinline__ Item get_item(const DiffGeo& g, int32_t idx) {
  Item it;
  const int32_t ob = idx / g.blocks, blk = idx - ob * g.blocks;
  it.b = ob % g.batch;
  it.head = g.order[ob / g.batch];
  it.bh = it.b * g.heads + it.head;
  const int32_t plane = g.nH * g.nW, full = (g.nT - 1) * plane * g.slabs;
  int32_t tile;
  if (blk < full) {
    tile = blk / g.slabs;
    it.s = blk - tile * g.slabs;
  } else {
    const int32_t r = blk - full;
    tile = r / g.slabs_last;
    it.s = r - tile * g.slabs_last;
    tile += (g.nT - 1) * plane;
  }
  it.t = tile / plane;
  it.h = (tile / g.nW) % g.nH;
  it.w = tile % g.nW;
  const int32_t wt = g.win[it.head][0], wh = g.win[it.head][1], ww = g.win[it.head][2];
  if (KEYS) {
    query_range(it.t, wt, g.nT, it.bt0, it.ent);
    query_range(it.h, wh, g.nH, it.bh0, it.enh);
    query_range(it.w, ww, g.nW, it.bw0, it.enw);
  } else {
    key_range(it.t, wt, g.nT, it.bt0, it.ent);
    key_range(it.h, wh, g.nH, it.bh0, it.enh);
    key_range(it.w, ww, g.nW, it.bw0, it.enw);
  }
  const int32_t lost = it.bt0 + it.ent == g.nT ? g.slabs - g.slabs_last : 0;
  it.n = it.enh * it.enw * (it.ent * g.slabs - lost);
  return it;
}

// A 128-row block of the padded latent.
struct Block {
  int32_t t, h, w, s;
};
__device__ __forceinline__ Block own_block(const Item& it) { return Block{it.t, it.h, it.w, it.s}; }
__device__ __forceinline__ Block first_block(const Item& it) { return Block{it.bt0, it.bh0, it.bw0, 0}; }
__device__ __forceinline__ void next_block(const DiffGeo& g, const Item& it, Block& b) {
  if (++b.s < slabs_at(g, b.t)) return;
  b.s = 0;
  if (++b.w < it.bw0 + it.enw) return;
  b.w = it.bw0;
  if (++b.h < it.bh0 + it.enh) return;
  b.h = it.bh0;
  ++b.t;
}
// First row of a block in the tiled order of the padded latent.
__device__ __forceinline__ int32_t tiled_row(const DiffGeo& g, const Block& b) {
  return ((b.t * g.nH + b.h) * g.nW + b.w) * g.ntile + b.s * kBlockRows;
}
// Whether the block holds pad tokens.
__device__ __forceinline__ bool has_pads(const DiffGeo& g, const Block& b) {
  return b.t * g.tt + (b.s + 1) * g.bt > g.T || (b.h + 1) * g.th > g.H || (b.w + 1) * g.tw > g.W;
}

// Place of a thread's row (0 .. 127) inside a slab.
struct Local {
  int32_t t, h, w;
};
__device__ __forceinline__ Local local_of(const DiffGeo& g, int32_t row) {
  const int32_t plane = g.th * g.tw;
  return Local{row / plane, (row % plane) / g.tw, row % g.tw};
}
// Raster token of a row of a block, or -1 for a pad.
__device__ __forceinline__ int32_t token_of(const DiffGeo& g, const Block& b, const Local& l) {
  const int32_t t = b.t * g.tt + b.s * g.bt + l.t, h = b.h * g.th + l.h, w = b.w * g.tw + l.w;
  return (t < g.T && h < g.H && w < g.W) ? (t * g.H + h) * g.W + w : -1;
}
// Row number of a token in the caller's tensor (of d elements each).
__device__ __forceinline__ int64_t row_of(const DiffGeo& g, int32_t b, int32_t head, int32_t token) {
  return g.token_major ? (static_cast<int64_t>(b) * g.L + token) * g.heads + head
                       : (static_cast<int64_t>(b) * g.heads + head) * g.L + token;
}
// Bit i of word c: key 32 c + i of the block is a real token (called by a whole warp).
__device__ __forceinline__ uint32_t real_word(const DiffGeo& g, const Block& b, int c) {
  return __ballot_sync(0xffffffffu, token_of(g, b, local_of(g, 32 * c + static_cast<int>(threadIdx.x & 31))) >= 0);
}

// Loads a block of D columns as 64-column boxes: 3-D boxes of a tiled copy, or 5-D boxes
// (one slab) of the raster tensor, whose coordinates past the grid read as zeros.
template <int D>
__device__ __forceinline__ void load_block(const DiffGeo& g, uint32_t dst, const CUtensorMap* m, uint32_t bar, const Item& it,
                                           const Block& b, bool tiled) {
#pragma unroll
  for (int x = 0; x < D / 64; ++x) {
    if (tiled)
      tma_load_3d(dst + x * (kBlockRows * 128), m, bar, x * 64, tiled_row(g, b), it.bh);
    else
      tma_load_5d(dst + x * (kBlockRows * 128), m, bar, (g.token_major ? it.head * D : 0) + x * 64, b.w * g.tw, b.h * g.th,
                  b.t * g.tt + b.s * g.bt, g.token_major ? it.b : it.bh);
  }
}

// Byte offset (>> 4) of K16 slice k16 in a 128-row K-major block of 64-column boxes.
__device__ __forceinline__ uint64_t koff(int k16) {
  return static_cast<uint64_t>(((k16 >> 2) * 16384 + (k16 & 3) * 32) >> 4);
}

// ---------------------------------------------------------------- host side

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Tiled copy [BH, Lpad, d]: box of 128 rows x 64 columns, 128-byte swizzle.
inline bool map_tiled(CUtensorMap* m, const void* base, const DiffGeo& g, int d) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(g.Lpad),
                        static_cast<cuuint64_t>(g.batch) * g.heads};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(g.Lpad) * d * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(kBlockRows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Raster tensor [B, heads, T, H, W, d] or [B, T, H, W, heads, d]: box of one slab x 64
// columns, 128-byte swizzle, so that the rows land in tile-local raster order.  Five
// dimensions serve both: (batch, head) is one of them, or the heads lie along the columns.
inline bool map_raster(CUtensorMap* m, const void* base, const DiffGeo& g, int d) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t cols = static_cast<cuuint64_t>(d) * (g.token_major ? g.heads : 1);
  const cuuint64_t row = cols * 2;
  cuuint64_t dims[5] = {cols, static_cast<cuuint64_t>(g.W), static_cast<cuuint64_t>(g.H), static_cast<cuuint64_t>(g.T),
                        static_cast<cuuint64_t>(g.batch) * (g.token_major ? 1 : g.heads)};
  cuuint64_t strides[4] = {row, row * g.W, row * g.W * g.H, row * g.W * g.H * g.T};
  cuuint32_t box[5] = {64, static_cast<cuuint32_t>(g.tw), static_cast<cuuint32_t>(g.th), static_cast<cuuint32_t>(g.bt), 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline cudaError_t sm_count(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace diff
}  // namespace sta
