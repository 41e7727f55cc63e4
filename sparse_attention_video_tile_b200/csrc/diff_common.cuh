// diff_common.cuh - window walk, tensor maps and row addressing shared by the
// differential attention kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "diff.h"
#include "packed.cuh"
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

// TMEM tiles of 16 lanes x 8 columns of 32 bits, spread over a warp like a matrix
// fragment: thread t holds columns 2 (t mod 4) and the next of rows t / 4 (first two
// registers of a tile) and t / 4 + 8.  Eight threads share a column pair, so a value that
// belongs to a column is needed by 4 of a thread's rows at once.
template <int OFF, int N>
__device__ __forceinline__ void tmem_ld_frag8(uint32_t taddr, uint32_t (&r)[N]) {   // 64 columns
  static_assert(OFF + 32 <= N, "register window out of range");
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[OFF + 0]), "=r"(r[OFF + 1]), "=r"(r[OFF + 2]), "=r"(r[OFF + 3]), "=r"(r[OFF + 4]), "=r"(r[OFF + 5]),
        "=r"(r[OFF + 6]), "=r"(r[OFF + 7]), "=r"(r[OFF + 8]), "=r"(r[OFF + 9]), "=r"(r[OFF + 10]), "=r"(r[OFF + 11]),
        "=r"(r[OFF + 12]), "=r"(r[OFF + 13]), "=r"(r[OFF + 14]), "=r"(r[OFF + 15]), "=r"(r[OFF + 16]),
        "=r"(r[OFF + 17]), "=r"(r[OFF + 18]), "=r"(r[OFF + 19]), "=r"(r[OFF + 20]), "=r"(r[OFF + 21]),
        "=r"(r[OFF + 22]), "=r"(r[OFF + 23]), "=r"(r[OFF + 24]), "=r"(r[OFF + 25]), "=r"(r[OFF + 26]),
        "=r"(r[OFF + 27]), "=r"(r[OFF + 28]), "=r"(r[OFF + 29]), "=r"(r[OFF + 30]), "=r"(r[OFF + 31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_frag4(uint32_t taddr, uint32_t (&r)[16]) {   // 32 columns
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// The same tiles with each column pair packed to one 32-bit column (4 columns a tile): one
// register for row t / 4, one for t / 4 + 8.
__device__ __forceinline__ void tmem_st_frag4(uint32_t taddr, const uint32_t (&r)[8]) {   // 16 columns
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

__device__ __forceinline__ uint64_t lds64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
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

// Item of this CTA's turn: the grid is walked forth and back, so that the CTA with the
// longest item of one turn has the shortest of the next (items come by decreasing window).
__device__ __forceinline__ int32_t item_at(int32_t turn) {
  const int32_t n = static_cast<int32_t>(gridDim.x), i = static_cast<int32_t>(blockIdx.x);
  return turn * n + ((turn & 1) ? n - 1 - i : i);
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
// Which keys of a block are real tokens, 32 at a time: lane i knows the places of keys
// 32 c + i inside a slab (8 bits each of t, h, w).
struct KeyPlaces {
  uint32_t at[4];
  __device__ __forceinline__ void init(const DiffGeo& g) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const Local l = local_of(g, 32 * c + static_cast<int>(threadIdx.x & 31));
      at[c] = static_cast<uint32_t>(l.t | (l.h << 8) | (l.w << 16));
    }
  }
  // bit i: key 32 c + i of the block is real (called by a whole warp)
  __device__ __forceinline__ uint32_t real(const DiffGeo& g, const Block& b, int c) const {
    const uint32_t p = at[c];
    return __ballot_sync(0xffffffffu, b.t * g.tt + b.s * g.bt + static_cast<int>(p & 255u) < g.T &&
                                          b.h * g.th + static_cast<int>((p >> 8) & 255u) < g.H &&
                                          b.w * g.tw + static_cast<int>(p >> 16) < g.W);
  }
};

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

// Calls f(Const<0>), f(Const<1>), ... f(Const<N - 1>): an unrolled loop whose index is a constant.
template <int I>
struct Const {
  static constexpr int value = I;
};
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(Const<I>{});
    static_for<N, I + 1>(f);
  }
}

// Shared-memory matrix descriptors (128-byte swizzle, 1024 bytes between 8-row groups)
// differ in their low word only: address >> 4, and the leading byte offset >> 4 above it.
// An issuing thread keeps one low word per operand; the offset of a K16 slice is added
// inside the instruction's own asm.  (As 64-bit values made outside, the slices of every
// operand are hoisted out of the block loop and spill: the dK, dV kernel then waited for
// local loads between its MMAs.)
constexpr uint32_t kDescHi = 0x40004040u;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
constexpr uint32_t kLboK = 16;                  // K-major operands
constexpr uint32_t kLboMn = kBlockRows * 128;   // MN-major: 64-column boxes

// Offset (>> 4) of K16 slice k16 in a 128-row K-major block of 64-column boxes.
constexpr uint32_t koff(int k16) { return static_cast<uint32_t>(((k16 >> 2) * 16384 + (k16 & 3) * 32) >> 4); }
// ... of K16 slice k16 (16 rows) of an MN-major block
constexpr uint32_t mnoff(int k16) { return static_cast<uint32_t>(k16 * (2048 >> 4)); }

template <uint32_t AO, uint32_t BO>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 u, v;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "add.u32 x, %1, %5;\n\t"
      "add.u32 y, %2, %6;\n\t"
      "mov.b64 u, {x, %7};\n\t"
      "mov.b64 v, {y, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], u, v, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(AO), "n"(BO), "n"(kDescHi)
      : "memory");
}
// A from tensor memory, AO columns further
template <uint32_t AO, uint32_t BO>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 v;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "add.u32 x, %1, %5;\n\t"
      "add.u32 y, %2, %6;\n\t"
      "mov.b64 v, {y, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], v, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(AO), "n"(BO), "n"(kDescHi)
      : "memory");
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
