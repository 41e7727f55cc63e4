// diff.h - geometry and launchers of differential attention (diff_fwd.cu, diff_bwd.cu).
//
// The windows travel in the kernels' parameters and every role of a kernel walks
// them itself, so a call needs no schedule in device memory: nothing is cached,
// uploaded or evicted, and a captured graph holds all it needs.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "internal.h"

namespace sta {

constexpr int kDiffMaxHeads = 256;

// Tile grid, windows and tensor layout, passed by value to the kernels.
struct DiffGeo {
  int32_t T, H, W;             // grid in tokens
  int32_t tt, th, tw;          // tile in tokens
  int32_t nT, nH, nW;          // tile grid of the padded latent
  int32_t bt;                  // frames of a 128-row slab
  int32_t ntile;               // rows of a tile
  int32_t slabs, slabs_last;   // 128-row slabs of a tile that hold real tokens; in the last tile row in t
  int32_t blocks;              // 128-row blocks with real rows, per (batch, head)
  int32_t batch, heads;
  int32_t L;                   // real tokens
  int64_t Lpad;                // rows of the tiled order of the padded latent
  int32_t padded;              // some tile has pad tokens
  int32_t token_major;
  uint8_t order[kDiffMaxHeads];      // heads by decreasing window, so that long items start first
  int16_t win[kDiffMaxHeads][3];     // windows clamped to the tile grid
};

struct DiffFwdArgs {
  const void *q, *k, *v;
  const float* lam;
  void *out, *out2;
  float* lse;
  int32_t d;
  float scale;
};

struct DiffBwdArgs {
  const void *q, *k, *v, *out, *out2, *dout;
  const float *lam, *lse;
  void *dq, *dk, *dv;
  float* dlam;
  float* vec;                  // [4][batch * heads][Lpad]: both maps' lse (log2 units), D_1, D_2
  float* dlam_part;            // [batch * heads * blocks][4]
  void* tiled;                 // q, k, v and dout in tiled order
  int32_t d;
  float scale;
};

cudaError_t launch_diff_fwd(const DiffGeo& g, const DiffFwdArgs& a, int32_t* err, uint64_t limit_ns, cudaStream_t stream);
cudaError_t launch_diff_bwd(const DiffGeo& g, const DiffBwdArgs& a, int32_t* err, uint64_t limit_ns, cudaStream_t stream);

}  // namespace sta
