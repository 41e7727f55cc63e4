// diff_bwd.cu - differential attention over tile windows, backward, for sm_100a.
//
//   P_m = exp(scale S_m - lse_m),  dP = dO V^T (one product for both maps),
//   dS_1 = P_1 (dP - D_1),  dS_2 = -lambda P_2 (dP - D_2),  D_m = dO . (P_m V),
//   dQ_m = scale dS_m K_m,  dK_m = scale dS_m^T Q_m,  dV = (P_1 - lambda P_2)^T dO,
//   dlambda = - sum over rows of sum_j P_2 dP.
//
// Four launches:
//   * prep (HBM bound): q, k, v, dO copied into the tiled order of the padded latent,
//     and per row -lse_m in log2 units and -D_m, with D_2 = dO . O_2 and
//     D_1 = dO . out + lambda D_2 from the stored outputs.  Pad rows get P = 0
//     (-lse = -inf) and D = 0, so that they add nothing anywhere;
//   * dQ over query blocks and the key blocks of their windows;
//   * dK, dV over key blocks and the query blocks that attend them;
//   * the sum of dlambda's parts.
// Per 128 x 128 block the tensor cores do 1536 clocks of work in the dQ kernel (S_1,
// S_2, dP, dQ_1, dQ_2) and 2048 in the other (S_1, S_2, dP, dV, dK_1, dK_2), at 64 per
// M128 N128 K16, and both rebuild 2 x 128 x 128 exponentials (2048 clocks of MUFU).
// A pass that also added dQ through L2 would save S, dP and the exponentials of one
// kernel, but needs 64 KB of fp32 reductions per block, which this L2 does not keep up with.
#include "diff_common.cuh"

namespace sta {
namespace {

using namespace diff;

constexpr int kThreads = 384;    // warps 0-7 elementwise + epilogue, 8 and 11 loads, 9 and 10 MMA issue
constexpr int kRegsElem = 224;
constexpr int kRegsOther = 56;
static_assert(256 * kRegsElem + 128 * kRegsOther <= kThreads * 168, "register split above the launch allocation");
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

struct BwdParams {
  DiffGeo g;
  const float* lam;
  const float* vec;        // [4][BH][Lpad]: -lse_1, -lse_2 (log2 units), -D_1, -D_2
  __nv_bfloat16 *o0, *o1;  // dq; or dk and dv
  float* part;             // dQ kernel: [item][4] sums of P_2 dP
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

// dlambda[head] = - sum of the dQ items' parts, in a fixed order.
__global__ void __launch_bounds__(256) diff_dlam_kernel(const float* __restrict__ part, float* __restrict__ dlam,
                                                        const __grid_constant__ DiffGeo g) {
  __shared__ float red[8];
  const int64_t n = static_cast<int64_t>(g.batch) * g.blocks * 4;   // the head's items lie together
  const float* p = part + n * blockIdx.x;
  float s = 0.f;
  for (int64_t i = threadIdx.x; i < n; i += 256) s += p[i];
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.f;
    for (int i = 0; i < 8; ++i) s += red[i];
    dlam[g.order[blockIdx.x]] = -s;
  }
}

// ---------------------------------------------------------------- dQ
//
// Warps 0-3 do map 1, warps 4-7 map 2; a thread holds its row's 128 scores.  TMEM: one
// score buffer that the maps use in turn (0-127), dP (128-255), dS_1 and dS_2 as bf16
// in columns of their own (256-383), dQ_1 and dQ_2 (384-511).  Scores are free again
// once they are in registers and dP once both maps have read it, so the next block's
// S and dP run under this block's exponentials.

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

template <int D>
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
  const int32_t stride = static_cast<int32_t>(gridDim.x), first = static_cast<int32_t>(blockIdx.x);

  if (warp >= 8) {
    setmaxnreg_dec<kRegsOther>();
    if (lane == 0 && warp == 8) {
      // ---------------------------------------------------------- Q, dO and K loads
      uint32_t seq = 0, k = 0;
      bool ok = true;
      for (int32_t idx = first; ok && idx < p.n_items; idx += stride) {
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
      for (int32_t idx = first; ok && idx < p.n_items; idx += stride) {
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
      const uint64_t dq = sdesc_sw128(sb + S::kQ, 16, 1024), ddo = sdesc_sw128(sb + S::kDo, 16, 1024);
      const uint64_t dk0 = sdesc_sw128(sb + S::kK, 16, 1024), dv0 = sdesc_sw128(sb + S::kV, 16, 1024);
      uint32_t seq = 0, k = 0;
      bool ok = true;
      for (int32_t idx = first; ok && idx < p.n_items; idx += stride, ++k) {
        const Item it = get_item<false>(g, idx);
        ok = mbar_wait(sb + S::kFixFull, k & 1, wc, 0x34);
        for (int32_t j = 0; ok && j < it.n; ++j, ++seq) {
          const uint32_t st = seq % KS, ph = (seq / KS) & 1;
          ok = mbar_wait(sb + S::kKFull + 8 * st, ph, wc, 0x35);
          const uint64_t dk = dk0 + st * (S::kBlk >> 4), dv = dv0 + st * (S::kBlk >> 4);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            // the buffer's scores (map 2 of the last block, then map 1 of this one) are in registers
            if (ok && (m == 1 || seq > 0))
              ok = mbar_wait(sb + S::kSFree + 8 * (1 - m), (m == 1 ? seq : seq - 1) & 1, wc, 0x36);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              umma_ss(tmem, dq + koff(m * (D / 32) + i), dk + koff(m * (D / 32) + i), idesc, i > 0);
            umma_commit(sb + S::kSFull + 8 * m);
          }
          ok = ok && mbar_wait(sb + S::kVFull + 8 * st, ph, wc, 0x37) &&
               (seq == 0 || mbar_wait(sb + S::kPFree, (seq - 1) & 1, wc, 0x38));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < D / 16; ++i) umma_ss(tmem + 128, ddo + koff(i), dv + koff(i), idesc, i > 0);
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
      const uint64_t dk0 = sdesc_sw128(sb + S::kK, kBlockRows * 128, 1024);
      uint32_t seq = 0;
      bool ok = true;
      for (int32_t idx = first; ok && idx < p.n_items; idx += stride) {
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
            const uint64_t dk = dk0 + st * (S::kBlk >> 4) + (D == 128 ? m * (16384 >> 4) : 0);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              umma_ts(tmem + 384 + 64 * m, tmem + 256 + 64 * m + 8 * i, dk + static_cast<uint64_t>(i * (2048 >> 4)), idesc,
                      (j > 0 || i > 0));
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
    uint32_t seq = 0, k = 0;
    bool ok = true;
    for (int32_t idx = first; ok && idx < p.n_items; idx += stride, ++k) {
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
        if (g.padded) {
          if (has_pads(g, b)) {   // pad keys: exp(0 - lse) of a row with low scores could overflow
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t w = real_word(g, b, c);
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

template <int D>
struct Dkv {
  static constexpr int kBlk = kBlockRows * D * 2;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kStage = 2 * kBlk;                  // Q and dO
  static constexpr int kK = 0, kV = kBlk, kRing = 2 * kBlk;
  static constexpr int kDs = kRing + kStages * kStage;     // dS_2^T: two boxes of 128 rows x 64 columns
  static constexpr int kLse = kDs + 32768;                 // float [map][query]
  static constexpr int kD = kLse + 1024;                   // float [map][query]
  static constexpr int kBar = kD + 1024;
  static constexpr int kFixFull = kBar, kFixEmpty = kFixFull + 8;
  static constexpr int kFull = kFixEmpty + 8, kEmpty = kFull + 8 * kStages;
  static constexpr int kLFull = kEmpty + 8 * kStages, kLEmpty = kLFull + 8;
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
  constexpr int KS = S::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  if ((sb & 1023u) != 0) {   // no room for a pad: report instead of computing with a wrong swizzle
    if (threadIdx.x == 0) atomicCAS(p.err, 0, 0x200 | 0x40);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kAbort);
  if (threadIdx.x == 0) {
    mbar_init(sb + S::kFixFull, 1);
    mbar_init(sb + S::kFixEmpty, 1);
    for (int i = 0; i < KS; ++i) {
      mbar_init(sb + S::kFull + 8 * i, 1);
      mbar_init(sb + S::kEmpty + 8 * i, 1);
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
  const int32_t stride = static_cast<int32_t>(gridDim.x), first = static_cast<int32_t>(blockIdx.x);

  if (warp >= 8) {
    setmaxnreg_dec<kRegsOther>();
    if (lane == 0 && warp == 8) {
      // ---------------------------------------------------------- K, V of the item; Q, dO of its blocks
      uint32_t seq = 0, k = 0;
      bool ok = true;
      for (int32_t idx = first; ok && idx < p.n_items; idx += stride) {
        const Item it = get_item<true>(g, idx);
        ok = mbar_wait(sb + S::kFixEmpty, (k & 1) ^ 1, wc, 0x41);
        if (!ok) break;
        ++k;
        mbar_arrive_expect_tx(sb + S::kFixFull, 2 * S::kBlk);
        load_block<D>(g, sb + S::kK, &tm_k, sb + S::kFixFull, it, own_block(it), true);
        load_block<D>(g, sb + S::kV, &tm_v, sb + S::kFixFull, it, own_block(it), true);
        Block b = first_block(it);
        for (int32_t j = 0; j < it.n; ++j, ++seq, next_block(g, it, b)) {
          const uint32_t st = seq % KS, full = sb + S::kFull + 8 * st, base = sb + S::kRing + st * S::kStage;
          ok = mbar_wait(sb + S::kEmpty + 8 * st, ((seq / KS) & 1) ^ 1, wc, 0x42);
          if (!ok) break;
          mbar_arrive_expect_tx(full, 2 * S::kBlk);
          load_block<D>(g, base, &tm_q, full, it, b, true);
          load_block<D>(g, base + S::kBlk, &tm_do, full, it, b, true);
        }
      }
      if (k > 0) mbar_wait_drain(sb + S::kFixFull, (k - 1) & 1, p.limit_ns);
      for (uint32_t i = 0; i < KS && i < seq; ++i) {
        const uint32_t last = seq - 1 - ((seq - 1 - i) % KS);
        mbar_wait_drain(sb + S::kFull + 8 * i, (last / KS) & 1, p.limit_ns);
      }
    } else if (lane == 0 && warp == 11) {
      // ---------------------------------------------------------- -lse and -D of the blocks
      uint32_t seq = 0;
      bool ok = true, half = false;   // half: this block's lse was loaded, its D not
      for (int32_t idx = first; ok && idx < p.n_items; idx += stride) {
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
      // Steady state per block i: S_1 of i + 1 | dV, dK_1 of i | S_2 of i + 1 | dK_2 of i | dP of
      // i + 1.  MMAs of one thread execute in order, so dP may overwrite the columns that dV
      // and dK_1 read.  S_2 of i + 1 sits between the accumulations: the warps have loaded S_1
      // by then and work on its exponentials.
      constexpr uint32_t id_ss = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t id_dv = idesc_bf16_f32(128, D, false, true);
      constexpr uint32_t id_dk = idesc_bf16_f32(128, 64, false, true);
      const uint64_t dk = sdesc_sw128(sb + S::kK, 16, 1024), dv = sdesc_sw128(sb + S::kV, 16, 1024);
      const uint64_t dds = sdesc_sw128(sb + S::kDs, 16, 1024);
      const uint64_t dring = sdesc_sw128(sb + S::kRing, 16, 1024);                     // K-major
      const uint64_t dring_mn = sdesc_sw128(sb + S::kRing, kBlockRows * 128, 1024);    // MN-major
      auto ring_full = [&](uint32_t i) { return mbar_wait(sb + S::kFull + 8 * (i % KS), (i / KS) & 1, wc, 0x45); };
      auto stage = [&](uint32_t i) -> uint64_t { return (i % KS) * static_cast<uint64_t>(S::kStage >> 4); };
      auto issue_s = [&](uint32_t i, int m) {
#pragma unroll
        for (int x = 0; x < D / 32; ++x)
          umma_ss(tmem, dk + koff(m * (D / 32) + x), dring + stage(i) + koff(m * (D / 32) + x), id_ss, x > 0);
        umma_commit(sb + S::kSFull + 8 * m);
      };
      auto issue_dp = [&](uint32_t i) {
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          umma_ss(tmem + 128, dv + koff(x), dring + stage(i) + (S::kBlk >> 4) + koff(x), id_ss, x > 0);
        umma_commit(sb + S::kPFull);
      };
      uint32_t i = 0;   // block of the CTA's stream
      uint32_t k = 0;
      bool ok = true;
      for (int32_t idx = first; ok && idx < p.n_items; idx += stride, ++k) {
        const Item it = get_item<true>(g, idx);
        ok = mbar_wait(sb + S::kFixFull, k & 1, wc, 0x46) && ring_full(i) &&
             (i == 0 || mbar_wait(sb + S::kSFree + 8, (i - 1) & 1, wc, 0x47));
        if (!ok) break;
        tc_fence_after();
        issue_s(i, 0);
        issue_dp(i);
        ok = mbar_wait(sb + S::kSFree, i & 1, wc, 0x48);
        if (!ok) break;
        tc_fence_after();
        issue_s(i, 1);
        if (it.n == 1) umma_commit(sb + S::kFixEmpty);
        for (int32_t j = 0; j < it.n; ++j, ++i) {
          const bool more = j + 1 < it.n;
          if (more) {
            ok = ring_full(i + 1) && mbar_wait(sb + S::kSFree + 8, i & 1, wc, 0x47);
            if (!ok) break;
            tc_fence_after();
            issue_s(i + 1, 0);
          }
          ok = mbar_wait(sb + S::kDsFull, i & 1, wc, 0x49);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dqm = dring_mn + stage(i), dom = dqm + (S::kBlk >> 4);
          // P^T and dS_1^T of 16 queries x: 8 columns each of the dP region
#pragma unroll
          for (int x = 0; x < 8; ++x)
            umma_ts(tmem + 256, tmem + 128 + (x >> 2) * 64 + ((x >> 1) & 1) * 32 + (x & 1) * 8,
                    dom + static_cast<uint64_t>(x * (2048 >> 4)), id_dv, (j > 0 || x > 0));
#pragma unroll
          for (int x = 0; x < 8; ++x)
            umma_ts(tmem + 384, tmem + 128 + (x >> 2) * 64 + ((x >> 1) & 1) * 32 + 16 + (x & 1) * 8,
                    dqm + static_cast<uint64_t>(x * (2048 >> 4)), id_dk, (j > 0 || x > 0));
          if (more) {
            ok = mbar_wait(sb + S::kSFree, (i + 1) & 1, wc, 0x48);
            if (!ok) break;
            tc_fence_after();
            issue_s(i + 1, 1);
          }
#pragma unroll
          for (int x = 0; x < 8; ++x)
            umma_ss(tmem + 448, dds + koff(x), dqm + (D == 128 ? (16384 >> 4) : 0) + static_cast<uint64_t>(x * (2048 >> 4)),
                    id_dk, (j > 0 || x > 0));
          umma_commit(sb + S::kDsDone);
          umma_commit(sb + S::kEmpty + 8 * (i % KS));
          if (more) {
            issue_dp(i + 1);
            if (j + 2 == it.n) umma_commit(sb + S::kFixEmpty);
          } else {
            umma_commit(sb + S::kOFull);
          }
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
    const Local loc = local_of(g, row);
    uint8_t* ds_row = smem + S::kDs + hh * 16384 + row * 128;
    const ulonglong2* lse2 = reinterpret_cast<const ulonglong2*>(smem + S::kLse) + 16 * hh;   // two pairs of queries each
    const ulonglong2* dd2 = reinterpret_cast<const ulonglong2*>(smem + S::kD) + 16 * hh;
    const uint64_t sl2x2 = f32x2(p.scale_log2, p.scale_log2);
    uint32_t seq = 0, k = 0;
    bool ok = true;
    for (int32_t idx = first; ok && idx < p.n_items; idx += stride, ++k) {
      const Item it = get_item<true>(g, idx);
      const float nlam = -__ldg(p.lam + it.head);
      const uint64_t nlam2 = f32x2(nlam, nlam);
      for (int32_t j = 0; j < it.n; ++j, ++seq) {
        uint64_t pr[2][32];   // P_1 and -lambda P_2, pairs of queries
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          ok = __all_sync(0xffffffffu, mbar_wait(sb + S::kSFull + 8 * m, seq & 1, wc, 0x4a) &&
                                           (m == 1 || mbar_wait(sb + S::kLFull, seq & 1, wc, 0x4b)));
          if (!ok) break;
          tc_fence_after();
          uint32_t s[64];
          tmem_ld32_at<0>(tS, s);
          tmem_ld32_at<32>(tS + 32, s);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(sb + S::kSFree + 8 * m);
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const ulonglong2 nl = lse2[32 * m + x];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float a, b;
              f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[4 * x + 2 * y]), __uint_as_float(s[4 * x + 2 * y + 1])), sl2x2,
                                    y == 0 ? nl.x : nl.y),
                          a, b);
              const uint64_t e = f32x2(ex2_approx(a), ex2_approx(b));
              pr[m][2 * x + y] = m == 0 ? e : mul_f32x2(e, nlam2);
            }
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + S::kLEmpty);
        ok = __all_sync(0xffffffffu, mbar_wait(sb + S::kPFull, seq & 1, wc, 0x4c) && mbar_wait(sb + S::kDFull, seq & 1, wc, 0x4d) &&
                                         (seq == 0 || mbar_wait(sb + S::kDsDone, (seq - 1) & 1, wc, 0x4e)));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t dp[32], pk[16], d1[16], d2[16];
          tmem_ld32(tP + 32 * c, dp);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const ulonglong2 n1 = dd2[8 * c + x], n2 = dd2[32 + 8 * c + x];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int q = 2 * x + y;
              const uint64_t g2 = f32x2(__uint_as_float(dp[2 * q]), __uint_as_float(dp[2 * q + 1]));
              const uint64_t p1 = pr[0][16 * c + q], p2 = pr[1][16 * c + q];
              float a, b;
              f32x2_split(add_f32x2(p1, p2), a, b);
              pk[q] = pack_bf16x2(a, b);
              f32x2_split(mul_f32x2(p1, add_f32x2(g2, y == 0 ? n1.x : n1.y)), a, b);
              d1[q] = pack_bf16x2(a, b);
              f32x2_split(mul_f32x2(p2, add_f32x2(g2, y == 0 ? n2.x : n2.y)), a, b);
              d2[q] = pack_bf16x2(a, b);
            }
          }
          tmem_st16(tP + 32 * c, pk);
          tmem_st16(tP + 32 * c + 16, d1);
          // 16-byte chunk x (8 queries) of the row's 128 bytes, at its swizzled place
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4*>(ds_row + (((4 * c + x) ^ (row & 7)) << 4)) =
                make_uint4(d2[4 * x], d2[4 * x + 1], d2[4 * x + 2], d2[4 * x + 3]);
        }
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
      const int32_t token = token_of(g, own_block(it), loc);
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
  auto dq = diff_dq_kernel<D>;
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
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  diff_dlam_kernel<<<g.heads, 256, 0, stream>>>(a.dlam_part, a.dlam, g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_bwd(const DiffGeo& g, const DiffBwdArgs& a, int32_t* err, uint64_t limit_ns, cudaStream_t stream) {
  return a.d == 128 ? launch_t<128>(g, a, err, limit_ns, stream) : launch_t<64>(g, a, err, limit_ns, stream);
}

}  // namespace sta
