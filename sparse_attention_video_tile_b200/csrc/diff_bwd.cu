// diff_bwd.cu - differential attention over tile windows, backward, for sm_100a.
//
//   P_m = exp(scale S_m - lse_m),  dP = dO V^T (one product for both maps),
//   dS_1 = P_1 (dP - D_1),  dS_2 = -lambda P_2 (dP - D_2),  D_m = dO . (P_m V),
//   dQ_m = scale dS_m K_m,  dK_m = scale dS_m^T Q_m,  dV = (P_1 - lambda P_2)^T dO,
//   dlambda = - sum over rows of sum_j P_2 dP.
//
// Three launches:
//   * prep (HBM bound): q, k, v, dO copied into the tiled order of the padded latent,
//     and per row -lse_m in log2 units and -D_m, with D_2 = dO . O_2 and
//     D_1 = dO . out + lambda D_2 from the stored outputs.  These are bf16 (fp32 rows would be
//     four times the forward's writes), so D_m is off by half steps of out and out2, and
//     D_1's error grows with |lambda|, which D_1 itself does not.  Pad rows get P = 0
//     (-lse = -inf) and D = 0, so that they add nothing anywhere;
//   * dQ over query blocks and the key blocks of their windows;
//   * dK, dV over key blocks and the query blocks that attend them; its first blocks also
//     add dlambda's parts, which the dQ kernel left per item.
// Per 128 x 128 block the tensor cores do 1860 clocks of work in the dQ kernel (S_1,
// S_2, dP, dQ_1, dQ_2; d = 128) and 2370 in the other (S_1, S_2, dP, dV, dK_1, dK_2), at 64
// per M128 N128 K16 and 52 per M128 N64 K16, and both rebuild 2 x 128 x 128 exponentials
// (2048 clocks of MUFU).
// One pass that also added dQ through L2 would save S, dP and the exponentials of one
// kernel.  It has 64 KB of fp32 reductions per block: 28.7 GB at 6 heads of 115 200 tokens and
// windows of 27 tiles of 384, 10.9 ms at the 2.63 TB/s that reductions reach, against the two
// kernels' 13.7 ms.  That rate leaves room for it; it was not built.  Against it: the dK, dV kernel has
// no TMEM columns and no shared memory for a third accumulator, and dQ would depend on the
// order of the reductions.
#include "diff_common.cuh"

namespace sta {
namespace {

using namespace diff;

constexpr int kThreads = 384;    // warps 0-7 elementwise + epilogue, 8 and 11 loads, 9 and 10 MMA issue
constexpr int kRegsElem = 224;
constexpr int kRegsOther = 56;
static_assert(256 * kRegsElem + 128 * kRegsOther <= kThreads * 168, "register split above the launch allocation");
constexpr float kLog2e = 1.4426950408889634f;

struct BwdParams {
  DiffGeo g;
  const float* lam;
  const float* vec;        // [4][BH][Lpad]: -lse_1, -lse_2 (log2 units), -D_1, -D_2
  __nv_bfloat16 *o0, *o1;  // dq; or dk and dv
  float* part;             // [item][4] sums of P_2 dP: the dQ kernel writes them, the dK, dV kernel adds them
  float* dlam;
  int32_t n_items;
  float scale, scale_log2;
  int32_t* err;
  uint64_t limit_ns;
};

__device__ __forceinline__ const float* vec_at(const BwdParams& p, int i, const Item& it) {
  return p.vec + (static_cast<int64_t>(i) * p.g.batch * p.g.heads + it.bh) * p.g.Lpad;
}

// Half a row of an accumulator (N columns from TMEM address t), times mul, as bf16.
template <int N>
__device__ __forceinline__ void store_half(uint32_t t, __nv_bfloat16* dst, float mul, bool live) {
#pragma unroll
  for (int c = 0; c < N / 32; ++c) {
    uint32_t o[32];
    tmem_ld32(t + 32 * c, o);
    tmem_wait_ld();
    if (live) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = pack_bf16x2(__uint_as_float(o[8 * q + 2 * i]) * mul, __uint_as_float(o[8 * q + 2 * i + 1]) * mul);
        reinterpret_cast<uint4*>(dst)[4 * c + q] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// ---------------------------------------------------------------- prep
//
// Ten arrays of the tensors' size cross memory once: 6 heads of 115 200 tokens, d = 128, in
// 0.26 ms, the copy rate; d = 64 0.13 ms.

template <int D>
__global__ void __launch_bounds__(256) diff_prep_kernel(const uint4* __restrict__ q, const uint4* __restrict__ k,
                                                        const uint4* __restrict__ v, const uint4* __restrict__ dout,
                                                        const uint4* __restrict__ out, const uint4* __restrict__ out2,
                                                        const float* __restrict__ lam, const float* __restrict__ lse,
                                                        uint4* __restrict__ tiled, float* __restrict__ vec,
                                                        const __grid_constant__ DiffGeo g) {
  constexpr int C = D / 8;   // threads of a row, 16 bytes each
  const int64_t bhs = static_cast<int64_t>(g.batch) * g.heads, rows = bhs * g.Lpad;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / C) + threadIdx.x / C;
  const int c = static_cast<int>(threadIdx.x) % C;
  float d1 = 0.f, d2 = 0.f;
  int32_t token = -1, bh = 0;
  if (r < rows) {
    bh = static_cast<int32_t>(r / g.Lpad);
    const int32_t x = static_cast<int32_t>(r - bh * g.Lpad);
    const int32_t tile = x / g.ntile, i = x - tile * g.ntile, plane = g.th * g.tw;
    const Block b{tile / (g.nH * g.nW), (tile / g.nW) % g.nH, tile % g.nW, 0};
    token = token_of(g, b, Local{i / plane, (i % plane) / g.tw, i % g.tw});
    uint4 a[4] = {};
    if (token >= 0) {
      const int64_t at = row_of(g, bh / g.heads, bh % g.heads, token) * C + c;
      a[0] = __ldg(q + at);
      a[1] = __ldg(k + at);
      a[2] = __ldg(v + at);
      a[3] = __ldg(dout + at);
      const uint4 o1 = __ldg(out + at), o2 = __ldg(out2 + at);
      const uint32_t x0[4] = {a[3].x, a[3].y, a[3].z, a[3].w}, x1[4] = {o1.x, o1.y, o1.z, o1.w},
                     x2[4] = {o2.x, o2.y, o2.z, o2.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x0[u]));
        const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x1[u]));
        const float2 z = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x2[u]));
        d1 = fmaf(f.y, y.y, fmaf(f.x, y.x, d1));
        d2 = fmaf(f.y, z.y, fmaf(f.x, z.x, d2));
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) tiled[(u * rows + r) * C + c] = a[u];
  }
#pragma unroll
  for (int o = C / 2; o > 0; o >>= 1) {
    d1 += __shfl_xor_sync(0xffffffffu, d1, o);
    d2 += __shfl_xor_sync(0xffffffffu, d2, o);
  }
  if (r < rows && c < 4) {
    float val = 0.f;
    if (c < 2)
      val = token >= 0 ? -kLog2e * __ldg(lse + (c * bhs + bh) * g.L + token) : -INFINITY;
    else if (token >= 0)
      val = c == 2 ? -fmaf(__ldg(lam + bh % g.heads), d2, d1) : -d2;
    vec[c * rows + r] = val;
  }
}

// dlambda[head] = - sum of the dQ items' parts, in a fixed order, by all threads of a block
// (`red`: kThreads / 32 floats of shared memory).
__device__ __forceinline__ void sum_dlambda(const DiffGeo& g, const float* part, float* dlam, float* red) {
  const int64_t n = static_cast<int64_t>(g.batch) * g.blocks * 4;   // a head's items lie together
  for (int32_t i = static_cast<int32_t>(blockIdx.x); i < g.heads; i += static_cast<int32_t>(gridDim.x)) {
    const float* p = part + n * i;
    float s = 0.f;
    for (int64_t x = threadIdx.x; x < n; x += kThreads) s += p[x];
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      s = 0.f;
      for (int x = 0; x < kThreads / 32; ++x) s += red[x];
      dlam[g.order[i]] = -s;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- dQ
//
// Warps 0-3 do map 1, warps 4-7 map 2; a thread holds its row's 128 scores.  TMEM: one
// score buffer that the maps use in turn (0-127), dP (128-255), dS_1 and dS_2 as bf16
// in columns of their own (256-383), dQ_1 and dQ_2 (384-511).  Scores are free again
// once they are in registers and dP once both maps have read it, so the next block's
// S and dP run under this block's exponentials.  Bound by that chain of the elementwise
// warps, 3547 clocks a block (ncu, active cycles; 1.69 GHz).  Measured, 6 heads of 115 200
// tokens, windows of 27 tiles of 384:
// 5.84 ms at d = 128, 5.28 at d = 64 (5.42 with two stages of K and V instead of four).

template <int D>
struct Dq {
  static constexpr int kBlk = kBlockRows * D * 2;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kQ = 0, kDo = kBlk, kK = 2 * kBlk, kV = kK + kStages * kBlk;
  static constexpr int kBar = kV + kStages * kBlk;
  static constexpr int kFixFull = kBar, kFixEmpty = kFixFull + 8;
  static constexpr int kKFull = kFixEmpty + 8, kKEmpty = kKFull + 8 * kStages;
  static constexpr int kVFull = kKEmpty + 8 * kStages, kVEmpty = kVFull + 8 * kStages;
  static constexpr int kSFull = kVEmpty + 8 * kStages, kSFree = kSFull + 16;   // [map]
  static constexpr int kDsFull = kSFree + 16, kDsDone = kDsFull + 16;          // [map]
  static constexpr int kPFull = kDsDone + 16, kPFree = kPFull + 8;             // dP
  static constexpr int kOFull = kPFree + 8, kDrain = kOFull + 8;
  static constexpr int kSlot = kDrain + 16, kAbort = kSlot + 4;
  static constexpr int kBytes = kAbort + 4 + 1024;
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
};

// PAD: some tile has pad tokens; the elementwise warps then walk the blocks and mask their keys.
template <int D, bool PAD>
__global__ void __launch_bounds__(kThreads, 1)
    diff_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                   const __grid_constant__ BwdParams p) {
  using S = Dq<D>;
  constexpr int KS = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kAbort);
  if (threadIdx.x == 0) {
    mbar_init(sb + S::kFixFull, 1);
    mbar_init(sb + S::kFixEmpty, 1);
    for (int i = 0; i < KS; ++i) {
      mbar_init(sb + S::kKFull + 8 * i, 1);
      mbar_init(sb + S::kKEmpty + 8 * i, 1);
      mbar_init(sb + S::kVFull + 8 * i, 1);
      mbar_init(sb + S::kVEmpty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sb + S::kSFull + 8 * i, 1);
      mbar_init(sb + S::kSFree + 8 * i, 4);
      mbar_init(sb + S::kDsFull + 8 * i, 4);
      mbar_init(sb + S::kDsDone + 8 * i, 1);
      mbar_init(sb + S::kDrain + 8 * i, 1);
    }
    mbar_init(sb + S::kPFull, 1);
    mbar_init(sb + S::kPFree, 8);
    mbar_init(sb + S::kOFull, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 9) {
    tmem_alloc(sb + S::kSlot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<uint32_t*>(smem + S::kSlot);
  const WaitCtx wc{abort_flag, p.err, p.limit_ns};
  const DiffGeo& g = p.g;

  if (warp >= 8) {
    setmaxnreg_dec<kRegsOther>();
    if (lane == 0 && warp == 8) {
      // ---------------------------------------------------------- Q, dO and K loads
      uint32_t seq = 0, k = 0;
      bool ok = true;
      for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn)) {
        const Item it = get_item<false>(g, idx);
        ok = mbar_wait(sb + S::kFixEmpty, (k & 1) ^ 1, wc, 0x31);
        if (!ok) break;
        ++k;
        mbar_arrive_expect_tx(sb + S::kFixFull, 2 * S::kBlk);
        load_block<D>(g, sb + S::kQ, &tm_q, sb + S::kFixFull, it, own_block(it), true);
        load_block<D>(g, sb + S::kDo, &tm_do, sb + S::kFixFull, it, own_block(it), true);
        Block b = first_block(it);
        for (int32_t j = 0; j < it.n; ++j, ++seq, next_block(g, it, b)) {
          const uint32_t st = seq % KS;
          ok = mbar_wait(sb + S::kKEmpty + 8 * st, ((seq / KS) & 1) ^ 1, wc, 0x32);
          if (!ok) break;
          mbar_arrive_expect_tx(sb + S::kKFull + 8 * st, S::kBlk);
          load_block<D>(g, sb + S::kK + st * S::kBlk, &tm_k, sb + S::kKFull + 8 * st, it, b, true);
        }
      }
      if (k > 0) mbar_wait_drain(sb + S::kFixFull, (k - 1) & 1, p.limit_ns);
      for (uint32_t i = 0; i < KS && i < seq; ++i) {
        const uint32_t last = seq - 1 - ((seq - 1 - i) % KS);
        mbar_wait_drain(sb + S::kKFull + 8 * i, (last / KS) & 1, p.limit_ns);
      }
    } else if (lane == 0 && warp == 11) {
      // ---------------------------------------------------------- V loads
      uint32_t seq = 0;
      bool ok = true;
      for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn)) {
        const Item it = get_item<false>(g, idx);
        Block b = first_block(it);
        for (int32_t j = 0; j < it.n; ++j, ++seq, next_block(g, it, b)) {
          const uint32_t st = seq % KS;
          ok = mbar_wait(sb + S::kVEmpty + 8 * st, ((seq / KS) & 1) ^ 1, wc, 0x33);
          if (!ok) break;
          mbar_arrive_expect_tx(sb + S::kVFull + 8 * st, S::kBlk);
          load_block<D>(g, sb + S::kV + st * S::kBlk, &tm_v, sb + S::kVFull + 8 * st, it, b, true);
        }
      }
      for (uint32_t i = 0; i < KS && i < seq; ++i) {
        const uint32_t last = seq - 1 - ((seq - 1 - i) % KS);
        mbar_wait_drain(sb + S::kVFull + 8 * i, (last / KS) & 1, p.limit_ns);
      }
    } else if (lane == 0 && warp == 10) {
      // ---------------------------------------------------------- S_1, S_2, dP
      constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
      const uint32_t dq = desc_lo(sb + S::kQ, kLboK), ddo = desc_lo(sb + S::kDo, kLboK);
      const uint32_t dk0 = desc_lo(sb + S::kK, kLboK), dv0 = desc_lo(sb + S::kV, kLboK);
      uint32_t seq = 0, k = 0;
      bool ok = true;
      for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn), ++k) {
        const Item it = get_item<false>(g, idx);
        ok = mbar_wait(sb + S::kFixFull, k & 1, wc, 0x34);
        for (int32_t j = 0; ok && j < it.n; ++j, ++seq) {
          const uint32_t st = seq % KS, ph = (seq / KS) & 1;
          ok = mbar_wait(sb + S::kKFull + 8 * st, ph, wc, 0x35);
          const uint32_t dk = dk0 + st * (S::kBlk >> 4), dv = dv0 + st * (S::kBlk >> 4);
          static_for<2>([&](auto M) {
            constexpr int m = decltype(M)::value;
            // the buffer's scores (map 2 of the last block, then map 1 of this one) are in registers
            if (ok && (m == 1 || seq > 0))
              ok = mbar_wait(sb + S::kSFree + 8 * (1 - m), (m == 1 ? seq : seq - 1) & 1, wc, 0x36);
            if (!ok) return;
            tc_fence_after();
            static_for<D / 32>([&](auto I) {
              constexpr uint32_t o = koff(m * (D / 32) + decltype(I)::value);
              mma_ss<o, o>(tmem, dq, dk, idesc, decltype(I)::value > 0);
            });
            umma_commit(sb + S::kSFull + 8 * m);
          });
          ok = ok && mbar_wait(sb + S::kVFull + 8 * st, ph, wc, 0x37) &&
               (seq == 0 || mbar_wait(sb + S::kPFree, (seq - 1) & 1, wc, 0x38));
          if (!ok) break;
          tc_fence_after();
          static_for<D / 16>([&](auto I) {
            constexpr uint32_t o = koff(decltype(I)::value);
            mma_ss<o, o>(tmem + 128, ddo, dv, idesc, decltype(I)::value > 0);
          });
          umma_commit(sb + S::kVEmpty + 8 * st);
          if (j + 1 == it.n) umma_commit(sb + S::kFixEmpty);
          umma_commit(sb + S::kPFull);
        }
      }
      umma_commit(sb + S::kDrain);
      mbar_wait_drain(sb + S::kDrain, 0, p.limit_ns);
    } else if (lane == 0 && warp == 9) {
      // ---------------------------------------------------------- dQ_m += dS_m K_m
      // B is the 64-column box that holds K_m; at d = 64 both maps share the only box and
      // the other map's half of the product is left unread.
      constexpr uint32_t idesc = idesc_bf16_f32(128, 64, false, true);
      const uint32_t dk0 = desc_lo(sb + S::kK, kLboMn);
      uint32_t seq = 0;
      bool ok = true;
      for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn)) {
        const Item it = get_item<false>(g, idx);
        for (int32_t j = 0; ok && j < it.n; ++j, ++seq) {
          const uint32_t st = seq % KS;
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            // dS_m follows S_m, so K has landed; the map's warps store an item's first dS after
            // they have read the last item's dQ_m
            ok = ok && mbar_wait(sb + S::kDsFull + 8 * m, seq & 1, wc, 0x39);
            if (!ok) break;
            tc_fence_after();
            const uint32_t dk = dk0 + st * (S::kBlk >> 4) + (D == 128 ? m * (16384 >> 4) : 0);
            static_for<8>([&](auto I) {
              constexpr int i = decltype(I)::value;
              mma_ts<8 * i, mnoff(i)>(tmem + 384 + 64 * m, tmem + 256 + 64 * m, dk, idesc, (j > 0 || i > 0));
            });
            umma_commit(sb + S::kDsDone + 8 * m);
          }
          if (!ok) break;
          umma_commit(sb + S::kKEmpty + 8 * st);
          if (j + 1 == it.n) umma_commit(sb + S::kOFull);
        }
      }
      umma_commit(sb + S::kDrain + 8);
      mbar_wait_drain(sb + S::kDrain + 8, 0, p.limit_ns);
    }
    __syncwarp();
  } else {
    setmaxnreg_inc<kRegsElem>();
    const int m = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t tDs = tl + 256 + 64 * m;
    const Local loc = local_of(g, row);
    KeyPlaces places;
    if constexpr (PAD) places.init(g);
    uint32_t seq = 0, k = 0;
    bool ok = true;
    for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn), ++k) {
      const Item it = get_item<false>(g, idx);
      Block b = first_block(it);
      const int32_t trow = tiled_row(g, own_block(it)) + row;
      const float nlse = __ldg(vec_at(p, m, it) + trow), nd = __ldg(vec_at(p, 2 + m, it) + trow);
      const float wgt = m == 0 ? 1.0f : -__ldg(p.lam + it.head);
      const uint64_t sl2x2 = f32x2(p.scale_log2, p.scale_log2), nlse2 = f32x2(nlse, nlse), nd2 = f32x2(nd, nd),
                     w2 = f32x2(wgt, wgt);
      uint64_t corr[2] = {0, 0};   // sums of P (dP - D)
      for (int32_t j = 0; j < it.n; ++j, ++seq) {
        ok = __all_sync(0xffffffffu, mbar_wait(sb + S::kSFull + 8 * m, seq & 1, wc, 0x3a));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[128];
        tmem_ld32_at<0>(tl, s);
        tmem_ld32_at<32>(tl + 32, s);
        tmem_ld32_at<64>(tl + 64, s);
        tmem_ld32_at<96>(tl + 96, s);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + S::kSFree + 8 * m);
#pragma unroll
        for (int i = 0; i < 128; i += 2) {
          float x0, x1;
          f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), sl2x2, nlse2), x0, x1);
          s[i] = __float_as_uint(ex2_approx(x0));
          s[i + 1] = __float_as_uint(ex2_approx(x1));
        }
        if constexpr (PAD) {
          if (has_pads(g, b)) {   // pad keys: exp(0 - lse) of a row with low scores could overflow
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t w = places.real(g, b, c);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((w >> i) & 1u)) s[32 * c + i] = 0;
            }
          }
          next_block(g, it, b);
        }
        ok = __all_sync(0xffffffffu, mbar_wait(sb + S::kPFull, seq & 1, wc, 0x3b) &&
                                         (seq == 0 || mbar_wait(sb + S::kDsDone + 8 * m, (seq - 1) & 1, wc, 0x3c)));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t dp[32], ds[16];
          tmem_ld32(tl + 128 + 32 * c, dp);
          tmem_wait_ld();
          if (c == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sb + S::kPFree);
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const uint64_t t = add_f32x2(f32x2(__uint_as_float(dp[i]), __uint_as_float(dp[i + 1])), nd2);
            const uint64_t e = mul_f32x2(f32x2(__uint_as_float(s[32 * c + i]), __uint_as_float(s[32 * c + i + 1])), t);
            corr[(i >> 1) & 1] = add_f32x2(corr[(i >> 1) & 1], e);
            float e0, e1;
            f32x2_split(mul_f32x2(e, w2), e0, e1);
            ds[i >> 1] = pack_bf16x2(e0, e1);
          }
          tmem_st16(tDs + 16 * c, ds);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + S::kDsFull + 8 * m);
      }
      if (!ok) break;
      const int32_t token = token_of(g, own_block(it), loc);
      if (m == 1) {
        // sum_j P_2 dP of the row = D_2 + sum_j P_2 (dP - D_2)
        float a0, a1;
        f32x2_split(add_f32x2(corr[0], corr[1]), a0, a1);
        float r = token >= 0 ? (a0 + a1) - nd : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
        if (lane == 0) p.part[static_cast<int64_t>(idx) * 4 + quad] = r;
      }
      ok = __all_sync(0xffffffffu, mbar_wait(sb + S::kOFull, k & 1, wc, 0x3d));
      if (!ok) break;
      tc_fence_after();
      store_half<D / 2>(tl + 384 + 64 * m + (D == 64 ? 32 * m : 0),
                        p.o0 + row_of(g, it.b, it.head, token >= 0 ? token : 0) * D + m * (D / 2), p.scale, token >= 0);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- dK, dV
//
// S_m^T = K_m Q_m^T, dP^T = V dO^T: TMEM lane = key row, columns = queries.  Warps w and
// w + 4 take columns 0-63 and 64-127 of lane quadrant w for both maps, since dV needs
// P_1 - lambda P_2 of an element in one place.  TMEM: one score buffer that the maps
// use in turn (0-127), dP^T (128-255), dV (256-383), dK_1, dK_2 (384-511).  That leaves
// no columns for three bf16 operands of 64: P^T and dS_1^T go over the dP^T columns that
// their warp has read, dS_2^T through shared memory (K-major, 128-byte swizzle).
// -lse and -D of a query block are loaded apart from Q and dO, each into one buffer: -lse
// is free after the exponentials, -D after dS, and each is needed again half a block later.
// Bound by the elementwise warps: exponentials of both maps, then dP, the three operands and
// their stores, 4571 clocks a block (ncu, active cycles; 1.59 GHz), under which the products
// run.  Measured at the sizes above:
// 7.85 ms at d = 128, 7.4 at d = 64; 10.1 with a row per thread, 8.1 to 9.2 with 2 to 4 of 8
// exponentials on the FMA pipe.

template <int D>
struct Dkv {
  static constexpr int kBlk = kBlockRows * D * 2;
  static constexpr int kQs = D == 64 ? 4 : 3;              // stages of Q
  static constexpr int kOs = D == 64 ? 4 : 1;              // stages of dO
  static constexpr int kK = 0, kV = kBlk, kQ = 2 * kBlk, kDo = kQ + kQs * kBlk;
  static constexpr int kDs = kDo + kOs * kBlk;             // dS_2^T: two boxes of 128 rows x 64 columns
  static constexpr int kLse = kDs + 32768;                 // float [map][query]
  static constexpr int kD = kLse + 1024;                   // float [map][query]
  static constexpr int kBar = kD + 1024;
  static constexpr int kFixFull = kBar, kFixEmpty = kFixFull + 8;
  static constexpr int kQFull = kFixEmpty + 8, kQEmpty = kQFull + 8 * kQs;
  static constexpr int kDoFull = kQEmpty + 8 * kQs, kDoEmpty = kDoFull + 8 * kOs;
  static constexpr int kLFull = kDoEmpty + 8 * kOs, kLEmpty = kLFull + 8;
  static constexpr int kDFull = kLEmpty + 8, kDEmpty = kDFull + 8;
  static constexpr int kSFull = kDEmpty + 8, kSFree = kSFull + 16;    // [map]
  static constexpr int kPFull = kSFree + 16;               // dP^T written
  static constexpr int kDsFull = kPFull + 8, kDsDone = kDsFull + 8;   // P^T, dS^T stored; dK_2's product done
  static constexpr int kOFull = kDsDone + 8, kDrain = kOFull + 8;
  static constexpr int kSlot = kDrain + 8, kAbort = kSlot + 4;
  static constexpr int kBytes = kAbort + 4;                // the base is 1024-byte aligned (checked)
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    diff_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ BwdParams p) {
  using S = Dkv<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  if ((sb & 1023u) != 0) {   // no room for a pad: report instead of computing with a wrong swizzle
    if (threadIdx.x == 0) atomicCAS(p.err, 0, 0x200 | 0x40);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  sum_dlambda(p.g, p.part, p.dlam, reinterpret_cast<float*>(smem));   // before any load into shared memory
  fence_proxy_async();   // the loads (async proxy) write where the sums lay (generic proxy): after the barrier below
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kAbort);
  if (threadIdx.x == 0) {
    mbar_init(sb + S::kFixFull, 1);
    mbar_init(sb + S::kFixEmpty, 1);
    for (int i = 0; i < S::kQs; ++i) {
      mbar_init(sb + S::kQFull + 8 * i, 1);
      mbar_init(sb + S::kQEmpty + 8 * i, 1);
    }
    for (int i = 0; i < S::kOs; ++i) {
      mbar_init(sb + S::kDoFull + 8 * i, 1);
      mbar_init(sb + S::kDoEmpty + 8 * i, 1);
    }
    mbar_init(sb + S::kLFull, 1);
    mbar_init(sb + S::kLEmpty, 8);
    mbar_init(sb + S::kDFull, 1);
    mbar_init(sb + S::kDEmpty, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(sb + S::kSFull + 8 * i, 1);
      mbar_init(sb + S::kSFree + 8 * i, 8);
    }
    mbar_init(sb + S::kPFull, 1);
    mbar_init(sb + S::kDsFull, 8);
    mbar_init(sb + S::kDsDone, 1);
    mbar_init(sb + S::kOFull, 1);
    mbar_init(sb + S::kDrain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 9) {
    tmem_alloc(sb + S::kSlot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<uint32_t*>(smem + S::kSlot);
  const WaitCtx wc{abort_flag, p.err, p.limit_ns};
  const DiffGeo& g = p.g;

  if (warp >= 8) {
    setmaxnreg_dec<kRegsOther>();
    if (lane == 0 && warp == 8) {
      // ---------------------------------------------------------- K, V of the item; Q of its blocks
      uint32_t seq = 0, k = 0;
      bool ok = true;
      for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn)) {
        const Item it = get_item<true>(g, idx);
        ok = mbar_wait(sb + S::kFixEmpty, (k & 1) ^ 1, wc, 0x41);
        if (!ok) break;
        ++k;
        mbar_arrive_expect_tx(sb + S::kFixFull, 2 * S::kBlk);
        load_block<D>(g, sb + S::kK, &tm_k, sb + S::kFixFull, it, own_block(it), true);
        load_block<D>(g, sb + S::kV, &tm_v, sb + S::kFixFull, it, own_block(it), true);
        Block b = first_block(it);
        for (int32_t j = 0; j < it.n; ++j, ++seq, next_block(g, it, b)) {
          const uint32_t st = seq % S::kQs;
          ok = mbar_wait(sb + S::kQEmpty + 8 * st, ((seq / S::kQs) & 1) ^ 1, wc, 0x42);
          if (!ok) break;
          mbar_arrive_expect_tx(sb + S::kQFull + 8 * st, S::kBlk);
          load_block<D>(g, sb + S::kQ + st * S::kBlk, &tm_q, sb + S::kQFull + 8 * st, it, b, true);
        }
      }
      if (k > 0) mbar_wait_drain(sb + S::kFixFull, (k - 1) & 1, p.limit_ns);
      for (uint32_t i = 0; i < S::kQs && i < seq; ++i) {
        const uint32_t last = seq - 1 - ((seq - 1 - i) % S::kQs);
        mbar_wait_drain(sb + S::kQFull + 8 * i, (last / S::kQs) & 1, p.limit_ns);
      }
    } else if (lane == 0 && warp == 10) {
      // ---------------------------------------------------------- dO of the blocks
      uint32_t seq = 0;
      bool ok = true;
      for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn)) {
        const Item it = get_item<true>(g, idx);
        Block b = first_block(it);
        for (int32_t j = 0; j < it.n; ++j, ++seq, next_block(g, it, b)) {
          const uint32_t st = seq % S::kOs;
          ok = mbar_wait(sb + S::kDoEmpty + 8 * st, ((seq / S::kOs) & 1) ^ 1, wc, 0x4f);
          if (!ok) break;
          mbar_arrive_expect_tx(sb + S::kDoFull + 8 * st, S::kBlk);
          load_block<D>(g, sb + S::kDo + st * S::kBlk, &tm_do, sb + S::kDoFull + 8 * st, it, b, true);
        }
      }
      for (uint32_t i = 0; i < S::kOs && i < seq; ++i) {
        const uint32_t last = seq - 1 - ((seq - 1 - i) % S::kOs);
        mbar_wait_drain(sb + S::kDoFull + 8 * i, (last / S::kOs) & 1, p.limit_ns);
      }
    } else if (lane == 0 && warp == 11) {
      // ---------------------------------------------------------- -lse and -D of the blocks
      uint32_t seq = 0;
      bool ok = true, half = false;   // half: this block's lse was loaded, its D not
      for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn)) {
        const Item it = get_item<true>(g, idx);
        Block b = first_block(it);
        for (int32_t j = 0; j < it.n; ++j, ++seq, next_block(g, it, b)) {
          const int32_t row = tiled_row(g, b);
          ok = mbar_wait(sb + S::kLEmpty, (seq & 1) ^ 1, wc, 0x43);
          if (!ok) break;
          mbar_arrive_expect_tx(sb + S::kLFull, 1024);
          bulk_load(sb + S::kLse, vec_at(p, 0, it) + row, 512, sb + S::kLFull);
          bulk_load(sb + S::kLse + 512, vec_at(p, 1, it) + row, 512, sb + S::kLFull);
          ok = mbar_wait(sb + S::kDEmpty, (seq & 1) ^ 1, wc, 0x44);
          if (!ok) {
            half = true;
            break;
          }
          mbar_arrive_expect_tx(sb + S::kDFull, 1024);
          bulk_load(sb + S::kD, vec_at(p, 2, it) + row, 512, sb + S::kDFull);
          bulk_load(sb + S::kD + 512, vec_at(p, 3, it) + row, 512, sb + S::kDFull);
        }
      }
      if (seq + (half ? 1 : 0) > 0) mbar_wait_drain(sb + S::kLFull, (seq + (half ? 1 : 0) - 1) & 1, p.limit_ns);
      if (seq > 0) mbar_wait_drain(sb + S::kDFull, (seq - 1) & 1, p.limit_ns);
    } else if (lane == 0 && warp == 9) {
      // ---------------------------------------------------------- MMAs, all from one thread
      // Steady state per block i: S_1 of i + 1 | dV of i | S_2 of i + 1 | dK_1 of i | dP of i + 1 |
      // dK_2 of i.  MMAs of one thread execute in order, so dP may overwrite the columns that dV
      // and dK_1 read.  S_2 of i + 1 sits between the accumulations: the warps have loaded S_1
      // by then and work on its exponentials.  dK_2 reads shared memory and comes last: its
      // operand is overwritten only at the end of the next block's elementwise step.
      constexpr uint32_t id_ss = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t id_dv = idesc_bf16_f32(128, D, false, true);
      constexpr uint32_t id_dk = idesc_bf16_f32(128, 64, false, true);
      const uint32_t dk = desc_lo(sb + S::kK, kLboK), dv = desc_lo(sb + S::kV, kLboK), dds = desc_lo(sb + S::kDs, kLboK);
      const uint32_t dq = desc_lo(sb + S::kQ, kLboK), ddo = desc_lo(sb + S::kDo, kLboK);
      constexpr uint32_t kMn = ((kLboMn - kLboK) >> 4) << 16;   // K-major to MN-major low word
      auto q_full = [&](uint32_t i) { return mbar_wait(sb + S::kQFull + 8 * (i % S::kQs), (i / S::kQs) & 1, wc, 0x45); };
      auto do_full = [&](uint32_t i) { return mbar_wait(sb + S::kDoFull + 8 * (i % S::kOs), (i / S::kOs) & 1, wc, 0x50); };
      auto q_at = [&](uint32_t i) -> uint32_t { return dq + (i % S::kQs) * (S::kBlk >> 4); };
      auto do_at = [&](uint32_t i) -> uint32_t { return ddo + (i % S::kOs) * (S::kBlk >> 4); };
      auto issue_s = [&](uint32_t i, auto M) {
        constexpr int m = decltype(M)::value;
        const uint32_t q = q_at(i);
        static_for<D / 32>([&](auto X) {
          constexpr uint32_t o = koff(m * (D / 32) + decltype(X)::value);
          mma_ss<o, o>(tmem, dk, q, id_ss, decltype(X)::value > 0);
        });
        umma_commit(sb + S::kSFull + 8 * m);
      };
      auto issue_dp = [&](uint32_t i) {
        const uint32_t d = do_at(i);
        static_for<D / 16>([&](auto X) {
          constexpr uint32_t o = koff(decltype(X)::value);
          mma_ss<o, o>(tmem + 128, dv, d, id_ss, decltype(X)::value > 0);
        });
        umma_commit(sb + S::kPFull);
      };
      uint32_t i = 0;   // block of the CTA's stream
      uint32_t k = 0;
      bool ok = true;
      for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn), ++k) {
        const Item it = get_item<true>(g, idx);
        ok = mbar_wait(sb + S::kFixFull, k & 1, wc, 0x46) && q_full(i) && do_full(i) &&
             (i == 0 || mbar_wait(sb + S::kSFree + 8, (i - 1) & 1, wc, 0x47));
        if (!ok) break;
        tc_fence_after();
        issue_s(i, Const<0>{});
        issue_dp(i);
        ok = mbar_wait(sb + S::kSFree, i & 1, wc, 0x48);
        if (!ok) break;
        tc_fence_after();
        issue_s(i, Const<1>{});
        if (it.n == 1) umma_commit(sb + S::kFixEmpty);
        for (int32_t j = 0; j < it.n; ++j, ++i) {
          const bool more = j + 1 < it.n;
          if (more) {
            ok = q_full(i + 1) && mbar_wait(sb + S::kSFree + 8, i & 1, wc, 0x47);
            if (!ok) break;
            tc_fence_after();
            issue_s(i + 1, Const<0>{});
          }
          ok = mbar_wait(sb + S::kDsFull, i & 1, wc, 0x49);
          if (!ok) break;
          tc_fence_after();
          const uint32_t dqm = q_at(i) + kMn, dom = do_at(i) + kMn;
          // P^T and dS_1^T of 16 queries x: 8 columns each of the dP region
          static_for<8>([&](auto X) {
            constexpr int x = decltype(X)::value;
            mma_ts<(x >> 2) * 64 + ((x >> 1) & 1) * 32 + (x & 1) * 8, mnoff(x)>(tmem + 256, tmem + 128, dom, id_dv,
                                                                               (j > 0 || x > 0));
          });
          umma_commit(sb + S::kDoEmpty + 8 * (i % S::kOs));   // dP of block i was issued before
          if (more) {
            ok = mbar_wait(sb + S::kSFree, (i + 1) & 1, wc, 0x48);
            if (!ok) break;
            tc_fence_after();
            issue_s(i + 1, Const<1>{});
          }
          static_for<8>([&](auto X) {
            constexpr int x = decltype(X)::value;
            mma_ts<(x >> 2) * 64 + ((x >> 1) & 1) * 32 + 16 + (x & 1) * 8, mnoff(x)>(tmem + 384, tmem + 128, dqm, id_dk,
                                                                                    (j > 0 || x > 0));
          });
          if (more) {
            ok = do_full(i + 1);
            if (!ok) break;
            tc_fence_after();
            issue_dp(i + 1);
            if (j + 2 == it.n) umma_commit(sb + S::kFixEmpty);
          }
          static_for<8>([&](auto X) {
            constexpr int x = decltype(X)::value;
            mma_ss<koff(x), (D == 128 ? (16384 >> 4) : 0) + mnoff(x)>(tmem + 448, dds, dqm, id_dk, (j > 0 || x > 0));
          });
          umma_commit(sb + S::kDsDone);
          umma_commit(sb + S::kQEmpty + 8 * (i % S::kQs));
          if (!more) umma_commit(sb + S::kOFull);
        }
      }
      umma_commit(sb + S::kDrain);
      mbar_wait_drain(sb + S::kDrain, 0, p.limit_ns);
    }
    __syncwarp();
  } else {
    setmaxnreg_inc<kRegsElem>();
    const int hh = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t tS = tl + 64 * hh, tP = tl + 128 + 64 * hh;
    // Scores are read as 16 x 8 fragments (two lane halves L, eight tiles j): this thread has the
    // queries 8 j + 2 (lane mod 4) and the next, of 4 key rows, so -lse and -D are read once for
    // 4 rows.  (With a row per thread every thread read them for all 64 queries: 1200 of the
    // block's clocks of shared memory bandwidth, which the MMAs' operands need.)
    const uint32_t ds_at = sb + S::kDs + hh * 16384 + (quad * 32 + (lane >> 2)) * 128 + (lane & 3) * 4;
    const uint32_t vec_lane = sb + S::kLse + 256 * hh + 8 * (lane & 3);   // this thread's queries of tile 0
    const uint64_t sl2x2 = f32x2(p.scale_log2, p.scale_log2);
    constexpr uint32_t kHalf = 16u << 16;   // TMEM address of lane 16
    uint32_t seq = 0, k = 0;
    bool ok = true;
    for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn), ++k) {
      // the loop keeps two numbers of the item: the block's P of both maps needs the registers
      int32_t n;
      uint64_t nlam2;
      {
        const Item it = get_item<true>(g, idx);
        const float nlam = -__ldg(p.lam + it.head);
        n = it.n;
        nlam2 = f32x2(nlam, nlam);
      }
      for (int32_t j = 0; j < n; ++j, ++seq) {
        uint64_t pr[2][32];   // P_1 and -lambda P_2: [16 L + 2 tile + row half], pairs of queries
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          ok = __all_sync(0xffffffffu, mbar_wait(sb + S::kSFull + 8 * m, seq & 1, wc, 0x4a) &&
                                           (m == 1 || mbar_wait(sb + S::kLFull, seq & 1, wc, 0x4b)));
          if (!ok) break;
          tc_fence_after();
          uint32_t s[64];
          tmem_ld_frag8<0>(tS, s);
          tmem_ld_frag8<32>(tS + kHalf, s);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(sb + S::kSFree + 8 * m);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const uint64_t nl = lds64(vec_lane + 512 * m + 32 * x);
#pragma unroll
            for (int L = 0; L < 2; ++L)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int r = 32 * L + 4 * x + 2 * y;
                float a, b;
                f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[r]), __uint_as_float(s[r + 1])), sl2x2, nl), a, b);
                const uint64_t e = f32x2(ex2_approx(a), ex2_approx(b));
                pr[m][r / 2] = m == 0 ? e : mul_f32x2(e, nlam2);
              }
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + S::kLEmpty);
        ok = __all_sync(0xffffffffu, mbar_wait(sb + S::kPFull, seq & 1, wc, 0x4c) &&
                                         mbar_wait(sb + S::kDFull, seq & 1, wc, 0x4d));
        if (!ok) break;
        tc_fence_after();
        uint32_t d2[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int L = 0; L < 2; ++L) {
            uint32_t dp[16], pk[8], d1[8];
            tmem_ld_frag4(tP + 32 * c + L * kHalf, dp);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint64_t n1 = lds64(vec_lane + 1024 + 32 * (4 * c + x)), n2 = lds64(vec_lane + 1536 + 32 * (4 * c + x));
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int q = 16 * L + 2 * (4 * c + x) + y;
                const uint64_t g2 = f32x2(__uint_as_float(dp[4 * x + 2 * y]), __uint_as_float(dp[4 * x + 2 * y + 1]));
                const uint64_t p1 = pr[0][q], p2 = pr[1][q];
                float a, b;
                f32x2_split(add_f32x2(p1, p2), a, b);
                pk[2 * x + y] = pack_bf16x2(a, b);
                f32x2_split(mul_f32x2(p1, add_f32x2(g2, n1)), a, b);
                d1[2 * x + y] = pack_bf16x2(a, b);
                f32x2_split(mul_f32x2(p2, add_f32x2(g2, n2)), a, b);
                d2[q] = pack_bf16x2(a, b);
              }
            }
            tmem_st_frag4(tP + 32 * c + L * kHalf, pk);
            tmem_st_frag4(tP + 32 * c + 16 + L * kHalf, d1);
          }
        }
        // the last block's dK_2 has read dS_2^T; a tile's 8 queries are one 16-byte chunk of a row,
        // at its swizzled place (rows 8 apart share the swizzle)
        if (seq > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(sb + S::kDsDone, (seq - 1) & 1, wc, 0x4e));
          if (!ok) break;
        }
#pragma unroll
        for (int L = 0; L < 2; ++L)
#pragma unroll
          for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              sts32(ds_at + (16 * L + 8 * y) * 128 + ((x ^ (lane >> 2)) << 4), d2[16 * L + 2 * x + y]);
        tmem_wait_st();
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(sb + S::kDEmpty);
          mbar_arrive(sb + S::kDsFull);
        }
      }
      if (!ok) break;
      ok = __all_sync(0xffffffffu, mbar_wait(sb + S::kOFull, k & 1, wc, 0x4f));
      if (!ok) break;
      tc_fence_after();
      const Item it = get_item<true>(g, idx);
      const int32_t token = token_of(g, own_block(it), local_of(g, row));
      const int64_t at = row_of(g, it.b, it.head, token >= 0 ? token : 0) * D + hh * (D / 2);
      store_half<D / 2>(tl + 384 + 64 * hh + (D == 64 ? 32 * hh : 0), p.o0 + at, p.scale, token >= 0);
      store_half<D / 2>(tl + 256 + hh * (D / 2), p.o1 + at, 1.0f, token >= 0);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_t(const DiffGeo& g, const DiffBwdArgs& a, int32_t* err, uint64_t limit_ns, cudaStream_t stream) {
  const int64_t bh = static_cast<int64_t>(g.batch) * g.heads, rows = bh * g.Lpad;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  constexpr int per = 256 / (D / 8);
  const int64_t blocks = (rows + per - 1) / per;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  // before the tensor maps: these calls make the device's context current in a thread that
  // has not used the device yet (autograd's), which the driver's encode call needs
  auto dq = g.padded ? diff_dq_kernel<D, true> : diff_dq_kernel<D, false>;
  if ((e = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, Dq<D>::kBytes)) != cudaSuccess) return e;
  auto dkv = diff_dkv_kernel<D>;
  if ((e = cudaFuncSetAttribute(dkv, cudaFuncAttributeMaxDynamicSharedMemorySize, Dkv<D>::kBytes)) != cudaSuccess) return e;
  __nv_bfloat16* t = static_cast<__nv_bfloat16*>(a.tiled);
  CUtensorMap tm[4];
  for (int i = 0; i < 4; ++i)
    if (!map_tiled(&tm[i], t + i * rows * D, g, D)) return cudaErrorInvalidValue;
  using V = const uint4*;
  diff_prep_kernel<D><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
      static_cast<V>(a.q), static_cast<V>(a.k), static_cast<V>(a.v), static_cast<V>(a.dout), static_cast<V>(a.out),
      static_cast<V>(a.out2), a.lam, a.lse, static_cast<uint4*>(a.tiled), a.vec, g);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  BwdParams p;
  p.g = g;
  p.lam = a.lam;
  p.vec = a.vec;
  p.part = a.dlam_part;
  p.dlam = a.dlam;
  p.n_items = static_cast<int32_t>(bh * g.blocks);
  p.scale = a.scale;
  p.scale_log2 = a.scale * kLog2e;
  p.err = err;
  p.limit_ns = limit_ns;
  const int grid = p.n_items < sms ? p.n_items : sms;
  p.o0 = static_cast<__nv_bfloat16*>(a.dq);
  p.o1 = nullptr;
  dq<<<grid, kThreads, Dq<D>::kBytes, stream>>>(tm[0], tm[1], tm[2], tm[3], p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  p.o0 = static_cast<__nv_bfloat16*>(a.dk);
  p.o1 = static_cast<__nv_bfloat16*>(a.dv);
  dkv<<<grid, kThreads, Dkv<D>::kBytes, stream>>>(tm[0], tm[1], tm[2], tm[3], p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_bwd(const DiffGeo& g, const DiffBwdArgs& a, int32_t* err, uint64_t limit_ns, cudaStream_t stream) {
  return a.d == 128 ? launch_t<128>(g, a, err, limit_ns, stream) : launch_t<64>(g, a, err, limit_ns, stream);
}

}  // namespace sta
