// Counter-based random bits for dropout: Philox4x32-10 (J. K. Salmon, M. A. Moraes, R. O. Dror,
// D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011), whose output depends only on
// a 64-bit key and a 128-bit counter, so a mask is recomputed wherever it is needed and never
// stored.
//
// Dropout's use of it: key = seed, counter = (column / 8, row, offset low, offset high), one call
// per group of eight consecutive columns of a row.  Element i of the group takes 16 bits of word
// i / 2, the low half for even i, and is kept where they are >= threshold = round(p 65536): p is
// resolved to 2^-16 and the kept values are scaled by the exact reciprocal of that probability.
// Sixteen bits an element instead of 32 halve the multiplications, which would otherwise bound
// the kernels before memory does (ten rounds of two 32 x 32 -> 64 products).
#pragma once

#include "common.h"

namespace moe {

struct DropArgs {
  const uint64_t* rng;  // device: {seed, offset}
  uint32_t threshold;   // keep where bits >= threshold (65536: keep none)
  float scale;          // 65536 / (65536 - threshold), 0 where nothing is kept
};

struct PhiloxKey {
  uint32_t k0, k1, c2, c3;
};

__device__ __forceinline__ PhiloxKey philox_key(const uint64_t* rng) {
  const uint64_t seed = rng[0], offset = rng[1];
  return PhiloxKey{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
}

__device__ __forceinline__ u32x4 philox10(const PhiloxKey& k, uint32_t c0, uint32_t c1) {
  uint32_t c2 = k.c2, c3 = k.c3, k0 = k.k0, k1 = k.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// Whether element i (0 .. 7) of the group whose words are w is kept.
__device__ __forceinline__ bool drop_keep(u32x4 w, int i, uint32_t threshold) {
  const uint32_t bits = (i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu;
  return bits >= threshold;
}

}  // namespace moe
