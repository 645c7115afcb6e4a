// Top-K of one token by one wave, and small helpers of the decode kernels.
#pragma once

#include "common.h"

namespace moe {

__device__ __forceinline__ uint32_t dec_order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float dec_key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// The K largest of E <= 64 EJ logits, logit(e) each: lane k receives the k-th expert and its logit.
template <int EJ, class Logit>
__device__ __forceinline__ void wave_select(Logit logit, int E, int K, int& my_e, float& my_v) {
  const int lane = threadIdx.x & 63;
  // lane i holds the order keys of experts i + 64 j (E <= 1024); each round takes the largest
  // key still in play (a DPP wave maximum) and, among the experts holding it, the lowest id
  // (ballots in ascending e): logit descending, then expert id ascending
  const int ej = (E + 63) >> 6;
  uint32_t key[EJ];
  uint32_t alive = 0;
#pragma unroll
  for (int j = 0; j < EJ; ++j) {
    const int e = lane + 64 * j;
    key[j] = e < E ? dec_order_key(logit(e)) : 0u;
    alive |= e < E ? (1u << j) : 0u;
  }
  my_e = 0;
  my_v = 0.0f;
  for (int k = 0; k < K; ++k) {
    uint32_t lm = 0;  // NaN keys are 0 too; ties at 0 are settled among live candidates
#pragma unroll
    for (int j = 0; j < EJ; ++j)
      if (j < ej && ((alive >> j) & 1u)) lm = key[j] > lm ? key[j] : lm;
    const uint32_t kmax = wave_max_u32(lm);
    int win = -1;
#pragma unroll
    for (int j = 0; j < EJ; ++j) {
      if (j >= ej) break;
      const uint64_t m = __builtin_amdgcn_ballot_w64(((alive >> j) & 1u) && key[j] == kmax);
      if (win < 0 && m != 0ull) win = 64 * j + (int)__builtin_ctzll(m);
    }
    win = __builtin_amdgcn_readfirstlane(win);
    if (lane == (win & 63)) alive &= ~(1u << (win >> 6));
    if (lane == k) {
      my_e = win;
      my_v = dec_key_value(kmax);
    }
  }
}

template <typename T>
__device__ __forceinline__ void dec_store4(T* p, f32x4 v) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t lo = (uint32_t)__builtin_bit_cast(uint16_t, from_f32<bf16>(v[0])) |
                        ((uint32_t)__builtin_bit_cast(uint16_t, from_f32<bf16>(v[1])) << 16);
    const uint32_t hi = (uint32_t)__builtin_bit_cast(uint16_t, from_f32<bf16>(v[2])) |
                        ((uint32_t)__builtin_bit_cast(uint16_t, from_f32<bf16>(v[3])) << 16);
    *reinterpret_cast<u32x2*>(p) = u32x2{lo, hi};
  } else {
    *reinterpret_cast<f32x4*>(p) = v;
  }
}

}  // namespace moe
