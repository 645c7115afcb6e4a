// Skinny products [weight rows x k] x [k x tokens] on 16 x 16 MFMA tiles, the weight rows streamed
// straight from memory into registers: shared by the single-launch decode kernel and the dense
// projection of a few rows.
#pragma once

#include "common.h"

namespace moe {

constexpr int DEC_U = 4;           // reduction steps per batch with one token group (two batches in flight)

// One reduction step of a 16x16 tile: every lane holds 16 bytes of its weight row (A, row
// lane % 16) and 16 bytes of its token's vector (B, column lane % 16), both at the same k offset
// (lane / 16) * V inside the step, so the products pair the same k on both sides.
template <typename T> struct DecMma;
template <> struct DecMma<bf16> {
  static constexpr int S = 32;  // k elements per step
  static constexpr int V = 8;   // k elements per lane per step
  __device__ static f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
template <> struct DecMma<float> {
  static constexpr int S = 16;
  static constexpr int V = 4;
  __device__ static f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    // four k = 4 products; product i takes element i of every lane's 4-element chunk
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
    return c;
  }
};

// Steps per batch: the register budget holds two batches of (1 + NG) 16-byte operands.
template <int NG> struct DecBatch { static constexpr int U = NG <= 2 ? DEC_U : DEC_U / 2; };

template <typename T, int NG>
struct DecStream {
  static constexpr int U = DecBatch<NG>::U;
  const T* w;       // lane's weight row at its k offset
  const T* x[NG];   // lane's token vectors at its k offset

  // steps st .. st + U - 1, constant offsets from one base per operand
  __device__ __forceinline__ void load(u32x4 (&wv)[U], u32x4 (&xv)[NG][U], int st) const {
    constexpr int S = DecMma<T>::S;
    const T* wp = w + st * S;
    const T* xp[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) xp[g] = x[g] + st * S;
#pragma unroll
    for (int u = 0; u < U; ++u) {  // in the order the MFMAs consume them
      wv[u] = ld16(wp + u * S);
#pragma unroll
      for (int g = 0; g < NG; ++g) xv[g][u] = ld16(xp[g] + u * S);
    }
  }
};

template <typename T, int NG, int U>
__device__ __forceinline__ void dec_mma(const u32x4 (&wv)[U], const u32x4 (&xv)[NG][U], f32x4 (&acc)[NG]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[g] = DecMma<T>::mma(wv[u], xv[g][u], acc[g]);
  }
}

// Steps [a, b) of one wave (a, b wave-uniform): whole batches with two register sets, the next
// batch's loads issued before the MFMAs of the current one, then the last (b - a) mod U steps
// as one short batch.
template <typename T, int NG>
__device__ __forceinline__ void dec_stream(const DecStream<T, NG>& ds, int a, int b, f32x4* acc) {
  constexpr int U = DecBatch<NG>::U;
  constexpr int S = DecMma<T>::S;
  f32x4 (&ac)[NG] = *reinterpret_cast<f32x4(*)[NG]>(acc);
  const int nfull = (b - a) / U;
  if (nfull > 0) {
    u32x4 w0[U], x0[NG][U], w1[U], x1[NG][U];
    ds.load(w0, x0, a);
    int i = 0;
    for (; i + 2 < nfull; i += 2) {  // steady state: loads unconditional, so the waits stay partial
      ds.load(w1, x1, a + (i + 1) * U);
      dec_mma<T, NG, U>(w0, x0, ac);
      ds.load(w0, x0, a + (i + 2) * U);
      dec_mma<T, NG, U>(w1, x1, ac);
    }
    if (i + 1 < nfull) {
      ds.load(w1, x1, a + (i + 1) * U);
      dec_mma<T, NG, U>(w0, x0, ac);
      dec_mma<T, NG, U>(w1, x1, ac);
    } else {
      dec_mma<T, NG, U>(w0, x0, ac);
    }
  }
  const int st = a + nfull * U, r = b - st;
  if (r > 0) {  // one more batch, all of its loads in flight together; steps past b repeat b - 1
    u32x4 wt[U], xt[NG][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int su = st + min(u, r - 1);
      wt[u] = ld16(ds.w + su * S);
#pragma unroll
      for (int g = 0; g < NG; ++g) xt[g][u] = ld16(ds.x[g] + su * S);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < r) {
#pragma unroll
        for (int g = 0; g < NG; ++g) ac[g] = DecMma<T>::mma(wt[u], xt[g][u], ac[g]);
      }
    }
  }
}

}  // namespace moe
