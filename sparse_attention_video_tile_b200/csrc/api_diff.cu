// api_diff.cu - the C entry points of differential attention (include/sta.h):
// argument checks, the geometry that the kernels take by value, workspace layout.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "checks.h"
#include "diff.h"

namespace sta {
namespace {

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

// Checks sizes and windows and fills the geometry.  batch = 0 or heads = 0 passes with
// blocks = 0 work.
sta_status make_diff_geo(int32_t batch, int32_t heads, int32_t d, int32_t token_major, sta_dim3 grid, sta_dim3 tile,
                         const sta_dim3* win, DiffGeo* g) {
  if (d != 64 && d != 128) return STA_ERR_HEADDIM;
  if (batch < 0 || heads < 0 || heads > kDiffMaxHeads) return STA_ERR_ARG;
  if (token_major != 0 && token_major != 1) return STA_ERR_ARG;
  if (heads > 0 && !win) return STA_ERR_NULL;
  // keeps every product below inside 64 bits
  for (int32_t x : {grid.t, grid.h, grid.w})
    if (x > (1 << 20)) return STA_ERR_SHAPE;
  for (int32_t x : {tile.t, tile.h, tile.w})
    if (x > (1 << 14)) return STA_ERR_SHAPE;
  Geometry o;
  const sta_status s = make_geometry_padded(grid, tile, &o);
  if (s != STA_OK) return s;
  if (!raster_tile_ok(tile.t, tile.h, tile.w)) return STA_ERR_SHAPE;
  *g = DiffGeo{};
  g->T = o.T; g->H = o.H; g->W = o.W;
  g->tt = o.tt; g->th = o.th; g->tw = o.tw;
  g->nT = o.nT; g->nH = o.nH; g->nW = o.nW;
  g->bt = kBlockRows / (o.th * o.tw);
  g->ntile = o.ntile;
  const int32_t last = o.T - (o.nT - 1) * o.tt;   // frames of the last tile row
  g->slabs = o.nT > 1 ? o.tt / g->bt : (last + g->bt - 1) / g->bt;
  g->slabs_last = (last + g->bt - 1) / g->bt;
  const int64_t plane = static_cast<int64_t>(o.nH) * o.nW;
  const int64_t blocks = plane * ((o.nT - 1) * static_cast<int64_t>(g->slabs) + g->slabs_last);
  const int64_t bh = static_cast<int64_t>(batch) * heads;
  if (blocks * std::max<int64_t>(bh, 1) > 0x3fffffff || o.Lpad > 0x3fffffff) return STA_ERR_SHAPE;
  // row and element numbers of a tensor stay inside 40 bits
  if (bh * o.Lpad > (int64_t(1) << 40) / d) return STA_ERR_SHAPE;
  g->blocks = static_cast<int32_t>(blocks);
  g->batch = batch;
  g->heads = heads;
  g->L = static_cast<int32_t>(o.L);
  g->Lpad = o.Lpad;
  g->padded = o.padded ? 1 : 0;
  g->token_major = token_major;
  int64_t cost[kDiffMaxHeads];
  for (int32_t h = 0; h < heads; ++h) {
    if (win[h].t < 1 || win[h].h < 1 || win[h].w < 1) return STA_ERR_WINDOW;
    const int32_t w[3] = {std::min(win[h].t, o.nT), std::min(win[h].h, o.nH), std::min(win[h].w, o.nW)};
    cost[h] = 1;
    for (int i = 0; i < 3; ++i) {
      if (w[i] > 32767) return STA_ERR_SHAPE;
      g->win[h][i] = static_cast<int16_t>(w[i]);
      cost[h] *= w[i];
    }
    g->order[h] = static_cast<uint8_t>(h);
  }
  // insertion sort, stable: long items first
  for (int32_t i = 1; i < heads; ++i)
    for (int32_t j = i; j > 0 && cost[g->order[j]] > cost[g->order[j - 1]]; --j) std::swap(g->order[j], g->order[j - 1]);
  return STA_OK;
}

int64_t copy_bytes(const DiffGeo& g, int32_t d) {
  return round256(static_cast<int64_t>(g.batch) * g.heads * g.Lpad * d * 2);
}

// Backward workspace: tiled q, k, v, dout; four row vectors; parts of dlambda.
struct BwdLayout {
  int64_t vec, part, total;
};
BwdLayout bwd_layout(const DiffGeo& g, int32_t d) {
  const int64_t bh = static_cast<int64_t>(g.batch) * g.heads;
  BwdLayout l;
  l.vec = 4 * copy_bytes(g, d);
  l.part = l.vec + round256(4 * bh * g.Lpad * 4);
  l.total = l.part + round256(bh * g.blocks * 4 * 4);
  return l;
}

bool scale_ok(float scale) {
  const float s = scale * 1.4426950408889634f;
  return scale > 0.f && std::isfinite(s) && s >= FLT_MIN;
}

}  // namespace
}  // namespace sta

using namespace sta;

extern "C" {

int64_t sta_diff_attention_bwd_workspace(int32_t batch, int32_t heads, int32_t d, sta_dim3 grid, sta_dim3 tile,
                                         const sta_dim3* window_per_head) {
  DiffGeo g;
  return make_diff_geo(batch, heads, d, 0, grid, tile, window_per_head, &g) == STA_OK ? bwd_layout(g, d).total : -1;
}

sta_status sta_diff_attention_fwd(const void* q, const void* k, const void* v, const float* lambda, void* out,
                                  void* out2, float* lse, int32_t batch, int32_t heads, int32_t d,
                                  int32_t token_major, sta_dim3 grid, sta_dim3 tile,
                                  const sta_dim3* window_per_head, float scale, void* stream) {
  DiffGeo g;
  sta_status s = make_diff_geo(batch, heads, d, token_major, grid, tile, window_per_head, &g);
  if (s != STA_OK) return s;
  if (!scale_ok(scale)) return STA_ERR_ARG;
  const int64_t bh = static_cast<int64_t>(batch) * heads;
  if (bh == 0) return STA_OK;
  if (!q || !k || !v || !lambda || !out) return STA_ERR_NULL;
  for (const void* p : {q, k, v, static_cast<const void*>(out), static_cast<const void*>(out2)})
    if (!aligned_to(p, 16)) return STA_ERR_ALIGN;
  if (!aligned_to(lse, 4) || !aligned_to(lambda, 4)) return STA_ERR_ALIGN;
  const int64_t n = bh * g.L * d * 2;
  const Range r[] = {{out, n}, {out2, n}, {lse, 2 * bh * g.L * 4}, {q, n}, {k, n}, {v, n}, {lambda, heads * 4}};
  if (any_overlap(r, 3, 7)) return STA_ERR_ALIAS;
  int dev = 0;
  int32_t* err = nullptr;
  if ((s = check_device(&dev)) != STA_OK || (s = status_word(dev, &err)) != STA_OK) return s;
  DiffFwdArgs a{};
  a.q = q; a.k = k; a.v = v; a.lam = lambda;
  a.out = out; a.out2 = out2; a.lse = lse;
  a.d = d;
  a.scale = scale;
  const cudaError_t e = launch_diff_fwd(g, a, err, kWaitLimitNs, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? STA_OK : cuda_fail(e);
}

sta_status sta_diff_attention_bwd(const void* q, const void* k, const void* v, const float* lambda, const void* out,
                                  const void* out2, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                                  float* dlambda, int32_t batch, int32_t heads, int32_t d, int32_t token_major,
                                  sta_dim3 grid, sta_dim3 tile, const sta_dim3* window_per_head, float scale,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
  DiffGeo g;
  sta_status s = make_diff_geo(batch, heads, d, token_major, grid, tile, window_per_head, &g);
  if (s != STA_OK) return s;
  if (!scale_ok(scale)) return STA_ERR_ARG;
  if (heads == 0) return STA_OK;
  if (!dlambda) return STA_ERR_NULL;
  const int64_t bh = static_cast<int64_t>(batch) * heads;
  if (bh > 0 && (!q || !k || !v || !lambda || !out || !out2 || !lse || !dout || !dq || !dk || !dv || !workspace))
    return STA_ERR_NULL;
  for (const void* p : {q, k, v, out, out2, dout, static_cast<const void*>(dq), static_cast<const void*>(dk),
                        static_cast<const void*>(dv), static_cast<const void*>(workspace)})
    if (!aligned_to(p, 16)) return STA_ERR_ALIGN;
  for (const float* p : {lambda, lse, static_cast<const float*>(dlambda)})
    if (!aligned_to(p, 4)) return STA_ERR_ALIGN;
  const BwdLayout l = bwd_layout(g, d);
  if (bh > 0 && workspace_bytes < l.total) return STA_ERR_SCRATCH;
  const int64_t n = bh * g.L * d * 2;
  const Range r[] = {{dq, n}, {dk, n}, {dv, n}, {dlambda, heads * 4}, {workspace, bh > 0 ? l.total : 0}, {q, n}, {k, n},
                     {v, n}, {out, n}, {out2, n}, {dout, n}, {lambda, heads * 4}, {lse, 2 * bh * g.L * 4}};
  if (any_overlap(r, 5, 13)) return STA_ERR_ALIAS;
  int dev = 0;
  int32_t* err = nullptr;
  if ((s = check_device(&dev)) != STA_OK || (s = status_word(dev, &err)) != STA_OK) return s;
  if (bh == 0) {   // no rows: the sum is zero
    const cudaError_t e = cudaMemsetAsync(dlambda, 0, static_cast<size_t>(heads) * 4, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? STA_OK : cuda_fail(e);
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  DiffBwdArgs a{};
  a.q = q; a.k = k; a.v = v; a.out = out; a.out2 = out2; a.dout = dout;
  a.lam = lambda; a.lse = lse;
  a.dq = dq; a.dk = dk; a.dv = dv; a.dlam = dlambda;
  a.tiled = ws;
  a.vec = reinterpret_cast<float*>(ws + l.vec);
  a.dlam_part = reinterpret_cast<float*>(ws + l.part);
  a.d = d;
  a.scale = scale;
  const cudaError_t e = launch_diff_bwd(g, a, err, kWaitLimitNs, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? STA_OK : cuda_fail(e);
}

}  // extern "C"
