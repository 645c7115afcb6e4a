// 4-bit weights with group scales as the A operand of 16 x 16 x 32 MFMAs: shared by the dense projection
// of a few rows (w4.hip) and the single-launch decode kernel (decode.hip).
//
// A row of K codes lies in K / 2 bytes, the even element in the low half.  A lane loads 16 bytes, 32
// codes, of its weight row at a time; the four lanes of a row cover a block of 128.
//
// FP (E2M1 values times 2^(e - 127), one scale byte per 32): lane q's codes are scale group q of the
// block, and one conversion instruction makes two codes with their scale into two bf16 values, exactly.
// Step j of the block takes the lane's codes 8 j .. 8 j + 7, against the same elements of the tokens.
//
// INT (value (c - 8) s, s bf16 per group of G = 32, 64 or 128): four lane swaps transpose the block, so
// that step j holds elements 32 j .. 32 j + 31 of the row in the MFMA's own order and a group is G / 32
// whole steps.  A code is put into the mantissa of 1.0 (1 + c / 16, one shift and one and-or for two codes)
// and the excess of 1.5 is taken off by a second product of the tokens with -1.5, which is exact in
// bf16: both sums are exact products accumulated in fp32, and the group's scale multiplies their sum in
// fp32.  So no weight is rounded.  Two codes that share a register are four apart; the tokens'
// elements are put into the same order (0 4 1 5 2 6 3 7) by four byte permutations.
#pragma once

#include "common.h"

namespace moe {

enum { W4_INT = 0, W4_FP = 1 };

constexpr int W4_BLOCK = 128;  // elements of a row per block

// Whole blocks and the part of a last one (a multiple of 32 elements).
__host__ __device__ __forceinline__ int w4_blocks(int K) { return (K + W4_BLOCK - 1) / W4_BLOCK; }

__device__ __forceinline__ bf16x8 w4_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }
__device__ __forceinline__ f32x4 w4_mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w4_bf16x8(a), w4_bf16x8(b), c, 0, 0, 0);
}

// Word j of lane group i becomes word i of lane group j (lane groups: lane / 16).
__device__ __forceinline__ void w4_transpose(u32x4& c) {
  auto a = __builtin_amdgcn_permlane32_swap(c[0], c[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(c[1], c[3], false, false);
  auto x = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto y = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  c = u32x4{x[0], x[1], y[0], y[1]};
}

// Eight codes of a word as 1 + c / 16 in bf16, elements 0 4 1 5 2 6 3 7.
__device__ __forceinline__ u32x4 w4_unpack_int(uint32_t w) {
  constexpr uint32_t M = 0x00780078u, ONE = 0x3f803f80u;
  return u32x4{((w << 3) & M) | ONE, ((w >> 1) & M) | ONE, ((w >> 5) & M) | ONE, ((w >> 9) & M) | ONE};
}
__device__ __forceinline__ u32x4 w4_order_int(u32x4 x) {
  return u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
               __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}
__device__ __forceinline__ u32x4 w4_unpack_fp(uint32_t w, float s) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
}

// One wave's stream over blocks of RT tiles of 16 weight rows against NG groups of 16 tokens.
template <int FMT, int G, int NG, int RT, int U>  // U: blocks per batch of loads
struct W4Stream {
  static constexpr bool INT = FMT == W4_INT;
  static constexpr int GS = INT ? G / 32 : 1;                  // steps per group
  static constexpr int NS = INT ? W4_BLOCK / G : 1;            // scale words per block and tile
  static constexpr int XS = INT ? 32 : 8;                      // elements between a lane's steps in x

  const uint8_t* w[RT];  // lane's weight row, at byte 16 (lane / 16)
  const uint8_t* s[RT];  // INT: scales of rows 4 (lane / 16) .. + 3 of the tile; FP: scale byte (lane / 16) of the lane's row
  int64_t plane;         // bytes between scale planes (INT: per group; FP: per block)
  const bf16* x[NG];     // lane's token, at element 8 (lane / 16) (INT) or 32 (lane / 16) (FP)
  int K;

  struct Codes {
    u32x4 c[RT];
    u32x2 s[RT][NS];  // INT: four bf16; FP: one byte
  };
  // the codes and scales of a block's first `left` elements (a multiple of 32)
  __device__ __forceinline__ void load_codes(Codes& b, int blk, int left = W4_BLOCK) const {
    const int q = (threadIdx.x & 63) >> 4;
    const bool in = left == W4_BLOCK || 32 * q < left;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      // a lane whose 32 elements lie behind the row reads the block's first ones, against zeros
      b.c[r] = ld16(w[r] + (int64_t)blk * (W4_BLOCK / 2) - (in ? 0 : 16 * q));
      if constexpr (INT) {
#pragma unroll
        for (int g = 0; g < NS; ++g)
          if (left == W4_BLOCK || g * G < left) b.s[r][g] = *reinterpret_cast<const u32x2*>(s[r] + ((int64_t)blk * NS + g) * plane);
      } else {
        b.s[r][0][0] = in ? s[r][blk * plane] : 127;
      }
    }
  }
  __device__ __forceinline__ void load_x(u32x4 (&v)[NG][4], int blk) const {
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[g][j] = ld16(x[g] + blk * W4_BLOCK + j * XS);
  }
  // the first `steps` steps of a block
  __device__ __forceinline__ void mma(Codes& b, const u32x4 (&xv)[NG][4], int steps, f32x4 (&acc)[RT][NG]) const {
    if constexpr (INT) {
      constexpr uint32_t NEG = 0xbfc0bfc0u;  // -1.5, twice
      const u32x4 neg = {NEG, NEG, NEG, NEG};
      const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int r = 0; r < RT; ++r) w4_transpose(b.c[r]);
      f32x4 corr[NG], part[RT][NG];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= steps) break;
        const bool first = j % GS == 0;
        u32x4 a[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) a[r] = w4_unpack_int(b.c[r][j]);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const u32x4 xo = w4_order_int(xv[g][j]);
          corr[g] = w4_mfma(neg, xo, first ? zero : corr[g]);
#pragma unroll
          for (int r = 0; r < RT; ++r) part[r][g] = w4_mfma(a[r], xo, first ? zero : part[r][g]);
        }
        if (j % GS == GS - 1) {
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const u32x2 sv = b.s[r][j / GS];
            const float f[4] = {__uint_as_float(sv[0] << 16), __uint_as_float(sv[0] & 0xffff0000u), __uint_as_float(sv[1] << 16),
                                __uint_as_float(sv[1] & 0xffff0000u)};
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[r][g][i] = fmaf(f[i], part[r][g][i] + corr[g][i], acc[r][g][i]);
          }
        }
      }
    } else {
      (void)steps;  // (lanes behind the row have zeros in xv)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        // 2^(e - 127); e = 0 is below the normal range
        const uint32_t e = b.s[r][0][0];
        const float sc = __uint_as_float(e ? e << 23 : 0x00400000u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 a = w4_unpack_fp(b.c[r][j], sc);
#pragma unroll
          for (int g = 0; g < NG; ++g) acc[r][g] = w4_mfma(a, xv[g][j], acc[r][g]);
        }
      }
    }
  }
  // blocks [a, b) of the row's w4_blocks(K); the last one may be a part
  __device__ __forceinline__ void run(int a, int b, f32x4 (&acc)[RT][NG]) const {
    const int whole = min(b, K / W4_BLOCK);
    if (a < whole) {
      Codes c0[U], c1[U];
      u32x4 x0[U][NG][4];
      auto codes = [&](Codes (&c)[U], int blk) {
#pragma unroll
        for (int u = 0; u < U; ++u) load_codes(c[u], min(blk + u, whole - 1));
      };
      // a batch: its tokens are requested before the next batch's codes, since loads return in order
      auto batch = [&](Codes (&c)[U], Codes (&next)[U], int blk, bool more) {
#pragma unroll
        for (int u = 0; u < U; ++u) load_x(x0[u], min(blk + u, whole - 1));
        if (more) codes(next, blk + U);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (blk + u < whole) mma(c[u], x0[u], 4, acc);
      };
      codes(c0, a);
      int blk = a;
      for (; blk + 2 * U < whole; blk += 2 * U) {
        batch(c0, c1, blk, true);
        batch(c1, c0, blk + U, true);
      }
      batch(c0, c1, blk, blk + U < whole);
      if (blk + U < whole) batch(c1, c0, blk + U, false);
    }
    if (b > whole && b * W4_BLOCK > K && a < b) tail(b - 1, acc);
  }
  // the part of a last block: K - 128 blk = 32, 64 or 96 elements
  __device__ __forceinline__ void tail(int blk, f32x4 (&acc)[RT][NG]) const {
    const int q = (threadIdx.x & 63) >> 4, left = K - blk * W4_BLOCK;
    Codes c;
    u32x4 v[NG][4];
    load_codes(c, blk, left);
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = INT ? 32 * j < left : 32 * q < left;
        v[g][j] = in ? ld16(x[g] + blk * W4_BLOCK + j * XS) : zero;
      }
    mma(c, v, left / 32, acc);
  }
};

// What a sum over blocks is still to be multiplied by (INT: codes went in as c / 16).
template <int FMT> __device__ __forceinline__ constexpr float w4_factor() { return FMT == W4_INT ? 16.0f : 1.0f; }

}  // namespace moe
