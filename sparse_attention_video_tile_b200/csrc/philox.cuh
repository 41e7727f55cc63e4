// philox.cuh - the counter-based generator behind dropout.
//
// Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011): a keyed bijection of a 128-bit counter.
// A dropout mask is a pure function of (seed, offset, row, column), so it is
// never stored: the backward pass evaluates it again.
//
// Element (r, c) of a [rows, cols] array takes 16-bit word c mod 8 (word 2i is the
// low half of 32-bit output i, word 2i + 1 its high half) of the block with counter
// (r * ceil(cols / 8) + c div 8, offset), 64 bits each, low words first, and key
// seed.  It is kept where that word is at least round(65536 p), so the drop
// probability is p to the nearest 2^-16, and kept values are multiplied by
// 65536 / (65536 - round(65536 p)), which keeps the expectation exact for the
// rounded probability.  Sixteen bits per element instead of 32: a block of ten
// rounds then serves eight elements, about ten integer instructions for each, which
// stays below the time that moving the element takes.
#pragma once

#include <cstdint>

namespace sta {

struct PhiloxKey {
  uint32_t seed_lo, seed_hi, off_lo, off_hi;
};

// rng: two 64-bit words on the device, seed and offset.
__device__ __forceinline__ PhiloxKey philox_key(const int64_t* rng) {
  const uint64_t s = static_cast<uint64_t>(rng[0]), o = static_cast<uint64_t>(rng[1]);
  return PhiloxKey{static_cast<uint32_t>(s), static_cast<uint32_t>(s >> 32), static_cast<uint32_t>(o),
                   static_cast<uint32_t>(o >> 32)};
}

// The 128 bits of counter block `n`.
__device__ __forceinline__ uint4 philox_block(uint64_t n, const PhiloxKey& k) {
  uint32_t c0 = static_cast<uint32_t>(n), c1 = static_cast<uint32_t>(n >> 32), c2 = k.off_lo, c3 = k.off_hi;
  uint32_t k0 = k.seed_lo, k1 = k.seed_hi;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c0, b = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    const uint32_t n0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0, n2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Bit j: element j of the block's eight is kept (thr = round(65536 p), 0 .. 65536).
__device__ __forceinline__ uint32_t philox_keep(const uint4& b, uint32_t thr) {
  uint32_t m = 0;
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m |= ((w[i] & 0xFFFFu) >= thr ? 1u : 0u) << (2 * i);
    m |= ((w[i] >> 16) >= thr ? 1u : 0u) << (2 * i + 1);
  }
  return m;
}

}  // namespace sta
