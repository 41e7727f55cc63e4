// diff_fwd.cu - differential attention over tile windows, forward, for sm_100a.
//
//   P_m = softmax(scale Q_m K_m^T) over the window, m = 1, 2 (the halves of a head's columns)
//   out = (P_1 - lambda P_2) V = O_1 / l_1 - lambda O_2 / l_2,   O_m = sum exp(.) V, l_m = sum exp(.)
//
// One pass: both maps' scores of a 128 x 128 block are made, exponentiated against
// their own running maxima and multiplied with V, which is loaded once for both; the
// difference is taken in the epilogue, when both sums are known.  A persistent CTA
// per SM walks the key blocks of its items (128 query rows of one head each):
//
//   * warps 0-3 are the softmax of map 1, warps 4-7 of map 2; TMEM lane = query row,
//     and a thread holds its row's 128 scores in registers, so the maximum is exact,
//     no row state is shared, and the score columns are free again after the load;
//   * warp 8 loads Q (two buffers) and K, warp 11 loads V (TMA, 128-byte swizzle,
//     rings of their own, so neither waits for the other's free stage);
//   * warp 10 issues S_m = Q_m K_m^T, warp 9 O_m += P_m V (P_m from TMEM).
//
// TMEM (d = 128): O_1, O_2 256 columns, P_1, P_2 64 each (bf16), one score buffer of
// 128 that the maps use in turn: S_1 of block g, S_2 of block g, S_1 of block g + 1.
// P has columns of its own instead of overwriting the scores, so the next scores need
// no finished product: the wait S -> softmax -> P V -> S is gone, and each map's
// softmax finds its next scores ready (d = 64 has a score buffer per map).
//
// The running maximum moves only when a row's block maximum is more than 20 (in log2)
// above it; then O_m and l_m are rescaled, and O_m / l_m does not depend on the
// reference.  p is at most 2^20, so O_m stays finite where |v| is below 2^107 divided by
// the keys of the window.  With 60 that bound was 2^67; 8 raises it to 2^119, but
// where scores spread by 11 in log2 it rescales so often that the kernel takes 8 to 14 %
// longer (20: 4 %; ordinary scores: the same time with all three).  Scores, sums and O are
// fp32; P is rounded to bf16 for the tensor cores (relative error 2^-8 at most per element, as
// in the other attention kernels; two bf16 parts would take 1024 more clocks of tensor work a
// block and TMEM columns that d = 128 lacks), l is summed from the unrounded p.
//
// Bound: one warp's serial chain per block (scores into registers, maximum, 128
// exponentials a thread, P out), 2626 clocks (active cycles counted by ncu over 1313.5 blocks
// an SM, d = 128), against 2048 of MUFU (78 %) and 1536 of tensor work (24 M128 N128 K16 of 64
// clocks, 58.5 %); the rest of the time is the clock under the power cap, 1.62 GHz.  Measured
// on 115 200 tokens, windows of 27 tiles of 384: d = 128, 24 heads 20.1 to 20.8 ms, 690 to 710
// TFLOP/s counting 4 d a pair (12 heads 10.0, 8.9 in short runs below the cap); d = 64, 12
// heads 8.8 ms.  Sixteen softmax warps with half rows take 10.85 and 9.5 ms at 12 heads, P
// stored in parts as it is made 11.6 and 9.8, 2 or 4 of 8 pairs of exponentials on the FMA
// pipe 10.6 and 12.1 (d = 128).
#include "diff_common.cuh"

namespace sta {
namespace {

using namespace diff;

constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 216;
constexpr int kRegsOther = 64;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "register split above the launch allocation");
constexpr int kKWarp = 8, kPvWarp = 9, kSWarp = 10, kVWarp = 11;
constexpr float kRaise = 20.0f;   // log2 units a block maximum may exceed the reference by
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Fwd {
  static constexpr int kBlk = kBlockRows * D * 2;
  static constexpr int kStages = 2;                   // of K and of V; d = 64: three or four take the same time
  static constexpr int kSBufs = D == 64 ? 2 : 1;
  static constexpr int kTO = 0;                       // O_m at kTO + m D
  static constexpr int kTP = 2 * D;                   // P_m at kTP + 64 m
  static constexpr int kTS = 2 * D + 128;             // score buffer b at kTS + 128 b
  static_assert(kTS + 128 * kSBufs <= 512, "TMEM columns");
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kBlk;
  static constexpr int kV = kK + kStages * kBlk;
  static constexpr int kLx = kV + kStages * kBlk;     // float [item parity][map][row]
  static constexpr int kBar = kLx + 2 * 2 * kBlockRows * 4;
  static constexpr int kQFull = kBar, kQEmpty = kQFull + 16;
  static constexpr int kKFull = kQEmpty + 16, kKEmpty = kKFull + 8 * kStages;
  static constexpr int kVFull = kKEmpty + 8 * kStages, kVEmpty = kVFull + 8 * kStages;
  static constexpr int kSFull = kVEmpty + 8 * kStages;   // [map] scores written
  static constexpr int kSFree = kSFull + 16;             // [map] scores in registers
  static constexpr int kPFull = kSFree + 16;             // [map] P written
  static constexpr int kPvDone = kPFull + 16;            // [map] P V completed
  static constexpr int kLxBar = kPvDone + 16;            // [lane quadrant] row sums written
  static constexpr int kOFull = kLxBar + 32, kOFree = kOFull + 8;
  static constexpr int kDrain = kOFree + 8;              // [2]
  static constexpr int kSlot = kDrain + 16, kAbort = kSlot + 4;
  static constexpr int kBytes = kAbort + 4 + 1024;       // + slack to align the base to 1024
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
};

struct FwdParams {
  DiffGeo g;
  const float* lam;
  __nv_bfloat16 *out, *out2;
  float* lse;
  int32_t n_items;
  float scale_log2;
  int32_t* err;
  uint64_t limit_ns;
};

// PAD: some tile has pad tokens; the softmax warps then walk the blocks and mask their keys.
// The state for that takes registers in the loop: one kernel for both kinds of grid ran 12
// heads of 30 x 48 x 80 without pads in 10.5 to 10.9 ms (d = 64: 9.4), this one in 10.0 (8.8).
template <int D, bool PAD>
__global__ void __launch_bounds__(kThreads, 1)
    diff_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ FwdParams p) {
  using S = Fwd<D>;
  constexpr int KS = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kAbort);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(sb + S::kQFull + 8 * i, 1);
      mbar_init(sb + S::kQEmpty + 8 * i, 1);
      mbar_init(sb + S::kSFull + 8 * i, 1);
      mbar_init(sb + S::kSFree + 8 * i, 4);
      mbar_init(sb + S::kPFull + 8 * i, 4);
      mbar_init(sb + S::kPvDone + 8 * i, 1);
      mbar_init(sb + S::kDrain + 8 * i, 1);
    }
    for (int i = 0; i < KS; ++i) {
      mbar_init(sb + S::kKFull + 8 * i, 1);
      mbar_init(sb + S::kKEmpty + 8 * i, 1);
      mbar_init(sb + S::kVFull + 8 * i, 1);
      mbar_init(sb + S::kVEmpty + 8 * i, 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(sb + S::kLxBar + 8 * i, 64);
    mbar_init(sb + S::kOFull, 1);
    mbar_init(sb + S::kOFree, 256);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kPvWarp) {
    tmem_alloc(sb + S::kSlot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<uint32_t*>(smem + S::kSlot);
  const WaitCtx wc{abort_flag, p.err, p.limit_ns};
  const DiffGeo& g = p.g;

  auto other_roles = [&]() {
    setmaxnreg_dec<kRegsOther>();
    if (lane == 0 && warp == kKWarp) {
      // ---------------------------------------------------------- Q and K loads
      uint32_t seq = 0, k = 0;
      bool ok = true;
      for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn), ++k) {
        const Item it = get_item<false>(g, idx);
        const uint32_t qb = k & 1;
        ok = mbar_wait(sb + S::kQEmpty + 8 * qb, ((k >> 1) & 1) ^ 1, wc, 0x21);
        if (!ok) break;
        mbar_arrive_expect_tx(sb + S::kQFull + 8 * qb, S::kBlk);
        load_block<D>(g, sb + S::kQ + qb * S::kBlk, &tm_q, sb + S::kQFull + 8 * qb, it, own_block(it), false);
        Block b = first_block(it);
        for (int32_t j = 0; j < it.n; ++j, ++seq, next_block(g, it, b)) {
          const uint32_t st = seq % KS;
          ok = mbar_wait(sb + S::kKEmpty + 8 * st, ((seq / KS) & 1) ^ 1, wc, 0x22);
          if (!ok) break;
          mbar_arrive_expect_tx(sb + S::kKFull + 8 * st, S::kBlk);
          load_block<D>(g, sb + S::kK + st * S::kBlk, &tm_k, sb + S::kKFull + 8 * st, it, b, false);
        }
        if (!ok) {   // this item's Q is in flight
          ++k;
          break;
        }
      }
      // every load issued has landed before the CTA may exit
      for (uint32_t i = 0; i < 2 && i < k; ++i) {
        const uint32_t last = k - 1 - ((k - 1 - i) & 1);
        mbar_wait_drain(sb + S::kQFull + 8 * i, (last >> 1) & 1, p.limit_ns);
      }
      for (uint32_t i = 0; i < KS && i < seq; ++i) {
        const uint32_t last = seq - 1 - ((seq - 1 - i) % KS);
        mbar_wait_drain(sb + S::kKFull + 8 * i, (last / KS) & 1, p.limit_ns);
      }
    } else if (lane == 0 && warp == kVWarp) {
      // ---------------------------------------------------------- V loads
      uint32_t seq = 0;
      bool ok = true;
      for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn)) {
        const Item it = get_item<false>(g, idx);
        Block b = first_block(it);
        for (int32_t j = 0; j < it.n; ++j, ++seq, next_block(g, it, b)) {
          const uint32_t st = seq % KS;
          ok = mbar_wait(sb + S::kVEmpty + 8 * st, ((seq / KS) & 1) ^ 1, wc, 0x23);
          if (!ok) break;
          mbar_arrive_expect_tx(sb + S::kVFull + 8 * st, S::kBlk);
          load_block<D>(g, sb + S::kV + st * S::kBlk, &tm_v, sb + S::kVFull + 8 * st, it, b, false);
        }
      }
      for (uint32_t i = 0; i < KS && i < seq; ++i) {
        const uint32_t last = seq - 1 - ((seq - 1 - i) % KS);
        mbar_wait_drain(sb + S::kVFull + 8 * i, (last / KS) & 1, p.limit_ns);
      }
    } else if (lane == 0 && warp == kSWarp) {
      // ---------------------------------------------------------- S_m = Q_m K_m^T
      constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
      const uint64_t dq0 = sdesc_sw128(sb + S::kQ, 16, 1024), dk0 = sdesc_sw128(sb + S::kK, 16, 1024);
      uint32_t seq = 0, k = 0;
      bool ok = true;
      for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn), ++k) {
        const Item it = get_item<false>(g, idx);
        const uint32_t qb = k & 1;
        ok = mbar_wait(sb + S::kQFull + 8 * qb, (k >> 1) & 1, wc, 0x24);
        for (int32_t j = 0; ok && j < it.n; ++j, ++seq) {
          const uint32_t st = seq % KS;
          ok = mbar_wait(sb + S::kKFull + 8 * st, (seq / KS) & 1, wc, 0x25);
          const uint64_t dq = dq0 + qb * (S::kBlk >> 4), dk = dk0 + st * (S::kBlk >> 4);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (!ok) break;
            // the buffer's last scores are in registers: with one buffer the other map's, just
            // issued (or the block before's), with two this map's of the block before
            const int of = S::kSBufs == 1 ? 1 - m : m;
            const uint32_t ph = (S::kSBufs == 1 && m == 1) ? seq : seq - 1;
            if (ph + 1 > 0) ok = mbar_wait(sb + S::kSFree + 8 * of, ph & 1, wc, 0x26);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              umma_ss(tmem + S::kTS + (S::kSBufs == 1 ? 0 : 128 * m), dq + koff(m * (D / 32) + i),
                      dk + koff(m * (D / 32) + i), idesc, i > 0);
            if (m == 1) {
              umma_commit(sb + S::kKEmpty + 8 * st);
              if (j + 1 == it.n) umma_commit(sb + S::kQEmpty + 8 * qb);
            }
            umma_commit(sb + S::kSFull + 8 * m);
          }
        }
      }
      umma_commit(sb + S::kDrain);
      mbar_wait_drain(sb + S::kDrain, 0, p.limit_ns);
    } else if (lane == 0 && warp == kPvWarp) {
      // ---------------------------------------------------------- O_m += P_m V
      constexpr uint32_t idesc = idesc_bf16_f32(128, D, false, true);
      const uint64_t dv0 = sdesc_sw128(sb + S::kV, kBlockRows * 128, 1024);
      uint32_t seq = 0, k = 0;
      bool ok = true;
      for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn), ++k) {
        const Item it = get_item<false>(g, idx);
        // the item's first products overwrite O: every softmax thread has read the last item's
        if (k > 0) ok = mbar_wait(sb + S::kOFree, (k - 1) & 1, wc, 0x27);
        for (int32_t j = 0; ok && j < it.n; ++j, ++seq) {
          const uint32_t st = seq % KS;
          ok = mbar_wait(sb + S::kVFull + 8 * st, (seq / KS) & 1, wc, 0x28);
          const uint64_t dv = dv0 + st * (S::kBlk >> 4);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            ok = ok && mbar_wait(sb + S::kPFull + 8 * m, seq & 1, wc, 0x29);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              umma_ts(tmem + S::kTO + m * D, tmem + S::kTP + 64 * m + 8 * i, dv + static_cast<uint64_t>(i * (2048 >> 4)),
                      idesc, (j > 0 || i > 0));
            umma_commit(sb + S::kPvDone + 8 * m);
          }
          if (!ok) break;
          umma_commit(sb + S::kVEmpty + 8 * st);
          if (j + 1 == it.n) umma_commit(sb + S::kOFull);
        }
      }
      umma_commit(sb + S::kDrain + 8);
      mbar_wait_drain(sb + S::kDrain + 8, 0, p.limit_ns);
    }
    __syncwarp();
  };
  auto softmax_role = [&]() {
    setmaxnreg_inc<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax + epilogue
    const int m = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t tS = tl + S::kTS + (S::kSBufs == 1 ? 0 : 128 * m);
    const uint32_t tP = tl + S::kTP + 64 * m, tO = tl + S::kTO + m * D;
    const Local loc = local_of(g, row);
    KeyPlaces places;
    if constexpr (PAD) places.init(g);
    const float sl2 = p.scale_log2;
    float* lx = reinterpret_cast<float*>(smem + S::kLx);
    uint32_t seq = 0, k = 0;
    bool ok = true;
    for (int32_t turn = 0, idx = item_at(0); ok && idx < p.n_items; idx = item_at(++turn), ++k) {
      const Item it = get_item<false>(g, idx);
      Block b = first_block(it);
      float mref = -INFINITY, l = 0.f;   // reference maximum (log2 units), sum against it
      for (int32_t j = 0; j < it.n; ++j, ++seq) {
        ok = __all_sync(0xffffffffu, mbar_wait(sb + S::kSFull + 8 * m, seq & 1, wc, 0x2a));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[128];
        tmem_ld32_at<0>(tS, s);
        tmem_ld32_at<32>(tS + 32, s);
        tmem_ld32_at<64>(tS + 64, s);
        tmem_ld32_at<96>(tS + 96, s);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + S::kSFree + 8 * m);
        if constexpr (PAD) {
          if (has_pads(g, b)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t w = places.real(g, b, c);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((w >> i) & 1u)) s[32 * c + i] = __float_as_uint(-INFINITY);
            }
          }
          next_block(g, it, b);
        }
        float a4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float a = max_nan(__uint_as_float(s[q]), __uint_as_float(s[q + 4]));
#pragma unroll
          for (int i = 8; i < 128; i += 8) a = max3_nan(a, __uint_as_float(s[q + i]), __uint_as_float(s[q + i + 4]));
          a4[q] = a;
        }
        // scale > 0, so the maximum of the scaled scores is the scaled maximum
        const float mx = max3_nan(max_nan(a4[0], a4[1]), a4[2], a4[3]) * sl2;
        const bool raise = !(mx <= mref + kRaise);   // also an item's first block, and a NaN
        float f = 1.0f;
        if (raise) {
          f = (mref == mx) ? 1.0f : ex2_approx(mref - mx);   // equal: both are -inf
          l *= f;
          mref = mx;
        }
        const float nm = (mref == -INFINITY) ? 0.f : -mref;
        const uint64_t sl2x2 = f32x2(sl2, sl2), nmx2 = f32x2(nm, nm);
        uint64_t ls[2] = {0, 0};
        uint32_t pk[64];
#pragma unroll
        for (int i = 0; i < 128; i += 2) {
          const uint64_t x2 = fma_f32x2(f32x2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), sl2x2, nmx2);
          float x0, x1;
          f32x2_split(x2, x0, x1);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          ls[(i >> 1) & 1] = add_f32x2(ls[(i >> 1) & 1], f32x2(p0, p1));
          pk[i >> 1] = pack_bf16x2(p0, p1);
        }
        float u0, u1;
        f32x2_split(add_f32x2(ls[0], ls[1]), u0, u1);
        l += u0 + u1;
        // the product of the block before has read P, and O holds it
        if (seq > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(sb + S::kPvDone + 8 * m, (seq - 1) & 1, wc, 0x2b));
          if (!ok) break;
          tc_fence_after();
        }
        if (j > 0 && __any_sync(0xffffffffu, raise)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32(tO + c * 32, o);
          }
        }
        tmem_st32_at<0>(tP, pk);
        tmem_st32_at<32>(tP + 32, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + S::kPFull + 8 * m);
      }
      if (!ok) break;
      // epilogue: this thread takes half m of the columns of both O_1 and O_2
      float* lk = lx + (k & 1) * 2 * kBlockRows;
      lk[m * kBlockRows + row] = l;
      mbar_arrive(sb + S::kLxBar + 8 * quad);
      ok = __all_sync(0xffffffffu, mbar_wait(sb + S::kLxBar + 8 * quad, k & 1, wc, 0x2c) &&
                                       mbar_wait(sb + S::kOFull, k & 1, wc, 0x2d));
      if (!ok) break;
      tc_fence_after();
      const float l1 = m == 0 ? l : lk[row], l2 = m == 0 ? lk[kBlockRows + row] : l;
      const float i1 = 1.0f / l1, i2 = 1.0f / l2, lam = p.lam[it.head];
      const int32_t token = token_of(g, own_block(it), loc);
      if (p.lse != nullptr && token >= 0)
        p.lse[(static_cast<int64_t>(m) * g.batch * g.heads + it.bh) * g.L + token] =
            (mref + log2f(l)) * 0.6931471805599453f;
      const int64_t at = row_of(g, it.b, it.head, token >= 0 ? token : 0) * D + m * (D / 2);
      uint4* d1 = reinterpret_cast<uint4*>(p.out + at);
      uint4* d2 = reinterpret_cast<uint4*>(p.out2 + at);
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        uint32_t o1[32], o2[32];
        tmem_ld32(tl + S::kTO + m * (D / 2) + 32 * c, o1);
        tmem_ld32(tl + S::kTO + D + m * (D / 2) + 32 * c, o2);
        tmem_wait_ld();
        if (token >= 0) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float y = __uint_as_float(o2[i]) * i2;
            o2[i] = __float_as_uint(y);
            o1[i] = __float_as_uint(fmaf(-lam, y, __uint_as_float(o1[i]) * i1));
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_bf16x2(__uint_as_float(o1[8 * q + 2 * i]), __uint_as_float(o1[8 * q + 2 * i + 1]));
            d1[4 * c + q] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (p.out2 != nullptr) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = pack_bf16x2(__uint_as_float(o2[8 * q + 2 * i]), __uint_as_float(o2[8 * q + 2 * i + 1]));
              d2[4 * c + q] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(sb + S::kOFree);
    }
  };
  // Same work either way: the placement decides how the compiler lays out the softmax loop.
  // Timed on B200: first is 3 % faster at d = 64 and 6 % with pads, last 10 % at d = 128.
  if constexpr (D == 64 || PAD) {
    if (warp < 8) softmax_role(); else other_roles();
  } else {
    if (warp >= 8) other_roles(); else softmax_role();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kPvWarp) tmem_dealloc(tmem, 512);
}

template <int D, bool PAD>
cudaError_t launch_t(const DiffGeo& g, const DiffFwdArgs& a, int32_t* err, uint64_t limit_ns, cudaStream_t stream) {
  using S = Fwd<D>;
  const int64_t bh = static_cast<int64_t>(g.batch) * g.heads;
  // before the tensor maps: makes the device's context current in a thread that has not
  // used the device yet, which the driver's encode call needs
  auto kern = diff_fwd_kernel<D, PAD>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != cudaSuccess) return e;
  CUtensorMap tq, tk, tv;
  if (!map_raster(&tq, a.q, g, D) || !map_raster(&tk, a.k, g, D) || !map_raster(&tv, a.v, g, D))
    return cudaErrorInvalidValue;
  int sms = 0;
  if ((e = sm_count(&sms)) != cudaSuccess) return e;
  FwdParams p;
  p.g = g;
  p.lam = a.lam;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.out2 = static_cast<__nv_bfloat16*>(a.out2);
  p.lse = a.lse;
  p.n_items = static_cast<int32_t>(bh * g.blocks);
  p.scale_log2 = a.scale * kLog2e;
  p.err = err;
  p.limit_ns = limit_ns;
  kern<<<p.n_items < sms ? p.n_items : sms, kThreads, S::kBytes, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_fwd(const DiffGeo& g, const DiffFwdArgs& a, int32_t* err, uint64_t limit_ns, cudaStream_t stream) {
  if (a.d == 128)
    return g.padded ? launch_t<128, true>(g, a, err, limit_ns, stream) : launch_t<128, false>(g, a, err, limit_ns, stream);
  return g.padded ? launch_t<64, true>(g, a, err, limit_ns, stream) : launch_t<64, false>(g, a, err, limit_ns, stream);
}

}  // namespace sta
