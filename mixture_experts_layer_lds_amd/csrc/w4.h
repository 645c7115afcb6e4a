// 4-bit weights with group scales as the B operand of 16 x 16 x 32 MFMAs, the tokens being A: shared by the
// dense projection of a few rows (w4.hip) and the decode of the routed experts (decode_w4.hip).
//
// A row of K codes lies in K / 2 bytes, the even element in the low half.  A lane loads 16 bytes, 32
// codes, of its weight row at a time; the four lanes of a row cover a block of 128.
//
// FP (E2M1 values times 2^(e - 127), one scale byte per 32): lane group q's codes are scale group q of the
// block, and one conversion instruction makes two codes with their scale into two bf16 values, exactly.
// Step j of the block takes the lane's codes 8 j .. 8 j + 7, against the same elements of the tokens.
//
// INT (value (c - 8) s, s bf16 per group of G = 32, 64 or 128): a group has to be whole steps, since its
// scale multiplies their sum.  With G = 128 the block is one group and steps are as above; with less, four
// lane swaps transpose the block so that step j holds elements 32 j .. 32 j + 31.  c - 8 = 4 h + l with the digits
// h = -2 .. 1 and l = 0 .. 3, each of which is an E2M1 value (h / 2 and l / 2): six bit operations make both digits of
// eight codes, the same conversions as for FP make them bf16, and a product is two MFMAs.  All products are exact, sums
// fp32, the weights are never rounded, and a weight of zero adds nothing however large the token's element is.
// (Codes as 1 + c / 16 and a product of the tokens with -1.5 to take the excess off are eight operations and fewer
// MFMAs, 14.1 us for 13 x 14336 -> 4096 with groups of 128 where this takes 14.4 and level for one token, but every sum
// carries rounding errors of 24 |x| s, and overflows for large finite x.)  The digits are scaled by 2^-12, which the end
// takes back: 128 products of any finite x stay in range.
//
// With the weights as B a lane's results all belong to one weight row, so a group costs one scale conversion
// and NI multiply-adds a lane: 4 for up to 16 tokens, 1 for up to 4, which then lie in every fourth row of A.
#pragma once

#include "common.h"

namespace moe {

enum { W4_INT = 0, W4_FP = 1 };

constexpr int W4_BLOCK = 128;  // elements of a row per block

__host__ __device__ __forceinline__ int w4_blocks(int K) { return (K + W4_BLOCK - 1) / W4_BLOCK; }

// a: tokens, b: weights
__device__ __forceinline__ f32x4 w4_mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Between LDS accesses of a wave's lanes to one another's places.  The LDS takes a wave's accesses in their order, so
// nothing has to be waited for: this keeps the compiler from changing that order.
__device__ __forceinline__ void w4_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Word j of lane group i becomes word i of lane group j (lane groups: lane / 16).
__device__ __forceinline__ void w4_transpose(u32x4& c) {
  auto a = __builtin_amdgcn_permlane32_swap(c[0], c[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(c[1], c[3], false, false);
  auto x = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto y = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  c = u32x4{x[0], x[1], y[0], y[1]};
}

__device__ __forceinline__ u32x4 w4_unpack_fp(uint32_t w, float s) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
}

// The digits of eight INT codes as E2M1 codes: l / 2 (its code is l) and h / 2 (-1, -0.5, 0, 0.5 for the code's upper two
// bits 0 .. 3).
__device__ __forceinline__ uint32_t w4_low_digits(uint32_t w) { return w & 0x33333333u; }
__device__ __forceinline__ uint32_t w4_high_digits(uint32_t w) {
  const uint32_t t = w >> 2;  // the upper two bits of a code in the lower two of its place
  return (~w & 0x88888888u) | (~((w >> 1) | t) & 0x22222222u) | (t & 0x11111111u);
}
constexpr float W4_LOW = 0x1p-11f, W4_HIGH = 0x1p-9f;  // 2 and 8, times 2^-12
constexpr float W4_INT_UNIT = 0x1p12f;

// Where a stream's tokens come from: memory, each lane the elements that its products take (one token, which all
// lanes of a group read); LDS (W4Stage); memory by whole lines, which the wave turns in its own part of LDS.  The
// last is for groups of 16 tokens, where reading a lane's 16 bytes from a token each costs more in the caches than the
// bytes do: a tenth of the whole with 32 x 14336 -> 4096 and 13 x 2048 -> 7168.
enum { W4_XMEM = 0, W4_XLDS = 1, W4_XLINE = 2 };
constexpr int W4_XSLOT = 16 * 256;  // bytes of LDS per wave and group with W4_XLINE: [token][chunk ^ token]

// One wave's stream over blocks of RT tiles of 16 weight rows against NG groups of tokens.
// U: blocks per batch of loads.
template <int FMT, int G, int NG, int RT, int NI, int XMODE, int U>
struct W4Stream {
  static constexpr bool XLDS = XMODE == W4_XLDS, XLINE = XMODE == W4_XLINE;
  static constexpr bool INT = FMT == W4_INT;
  static constexpr bool TR = INT && G < W4_BLOCK;     // blocks are transposed
  static constexpr int GS = INT ? G / 32 : 1;         // steps per group
  static constexpr int NS = INT ? W4_BLOCK / G : 1;   // scales per block and lane
  static constexpr int XQ = TR ? 8 : 32, XS = TR ? 32 : 8;  // a lane's elements of step j: block + XQ (lane / 16) + XS j

  const uint8_t* w[RT];  // lane's weight row (lane % 16 of the tile), at byte 16 (lane / 16)
  const uint8_t* s[RT];  // INT: its scales' first bytes; FP: its scale byte of group lane / 16
  int64_t plane;         // bytes between scale planes (INT: per group; FP: per block)
  const bf16* x[NG];     // lane's token, at element XQ (lane / 16); XLDS: in LDS
  // XLINE: lane's chunk lane % 16 of tokens 4 i + lane / 16, and the wave's LDS (NG W4_XSLOT)
  const char* xb;
  uint32_t xo[NG][4];
  char* xs;
  int K;

  struct Codes {
    u32x4 c[RT];
    uint32_t s[RT][NS];
  };
  struct Batch {
    Codes c[U];
    u32x4 x[XLDS ? 1 : U][NG][4];
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
          if (left == W4_BLOCK || g * G < left)
            b.s[r][g] = *reinterpret_cast<const uint16_t*>(s[r] + ((int64_t)blk * NS + g) * plane);
      } else {
        b.s[r][0] = in ? s[r][blk * plane] : 127;
      }
    }
  }
  // the tokens' elements of a block; of its first `left` (a multiple of 32), zeros behind
  __device__ __forceinline__ void load_x(u32x4 (&v)[NG][4], int blk, int left = W4_BLOCK) const {
    const int lane = threadIdx.x & 63;
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = XLINE ? 8 * (lane & 15) : TR ? 32 * j : 32 * (lane >> 4);
        const bool in = left == W4_BLOCK || at < left;
        if constexpr (XLINE) v[g][j] = in ? ld16(xb + (xo[g][j] + (uint32_t)blk * (2 * W4_BLOCK))) : zero;
        else v[g][j] = in ? ld16(x[g] + blk * W4_BLOCK + j * XS) : zero;
      }
  }
  // XLINE: a block's elements from the order of memory to LDS, where the lanes have read the last block's, and the
  // lane's of a step from there
  __device__ __forceinline__ void put(const u32x4 (&v)[NG][4]) const {
    const int lane = threadIdx.x & 63;
    w4_lds_order();
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * i + (lane >> 4);
        st16(xs + g * W4_XSLOT + t * 256 + 16 * ((lane & 15) ^ t), v[g][i]);
      }
    w4_lds_order();
  }
  __device__ __forceinline__ u32x4 get(int g, int j) const {
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    return ld16(xs + g * W4_XSLOT + r16 * 256 + 16 * ((TR ? 4 * j + q : 4 * q + j) ^ r16));
  }
  // the first `steps` steps of a block
  __device__ __forceinline__ void mma(Codes& b, u32x4 (&xv)[NG][4], int steps, f32x4 (&acc)[RT][NG]) const {
    if constexpr (XLINE) put(xv);
    if constexpr (INT) {
      if constexpr (TR) {
#pragma unroll
        for (int r = 0; r < RT; ++r) w4_transpose(b.c[r]);
      }
#pragma unroll
      for (int h = 0; h < NS; ++h) {
        if (h * GS >= steps) break;
        u32x4 xi[NG][GS];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int j = 0; j < GS; ++j) xi[g][j] = XLINE ? get(g, h * GS + j) : xv[g][h * GS + j];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          f32x4 part[NG];
#pragma unroll
          for (int g = 0; g < NG; ++g) part[g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int j = 0; j < GS; ++j) {
            const uint32_t w8 = b.c[r][h * GS + j];
            const u32x4 lo = w4_unpack_fp(w4_low_digits(w8), W4_LOW), hi = w4_unpack_fp(w4_high_digits(w8), W4_HIGH);
#pragma unroll
            for (int g = 0; g < NG; ++g) part[g] = w4_mfma(xi[g][j], lo, part[g]);
#pragma unroll
            for (int g = 0; g < NG; ++g) part[g] = w4_mfma(xi[g][j], hi, part[g]);
          }
          const float f = __uint_as_float(b.s[r][h] << 16);
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int i = 0; i < NI; ++i) acc[r][g][i] = fmaf(f, part[g][i], acc[r][g][i]);
        }
      }
    } else {
      (void)steps;  // (lanes behind the row have zeros in xv)
      if constexpr (XLINE) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int j = 0; j < 4; ++j) xv[g][j] = get(g, j);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        // 2^(e - 127); e = 0 is below the normal range
        const uint32_t e = b.s[r][0];
        const float sc = __uint_as_float(e ? e << 23 : 0x00400000u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 c = w4_unpack_fp(b.c[r][j], sc);
#pragma unroll
          for (int g = 0; g < NG; ++g) acc[r][g] = w4_mfma(xv[g][j], c, acc[r][g]);
        }
      }
    }
  }

  __device__ __forceinline__ void load(Batch& t, int blk, int last) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = min(blk + u, last);
      load_codes(t.c[u], k);
      if constexpr (!XLDS) load_x(t.x[u], k);
    }
  }
  __device__ __forceinline__ void mma(Batch& t, int blk, int live, f32x4 (&acc)[RT][NG]) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= live) break;
      if constexpr (XLDS) load_x(t.x[0], blk + u);
      mma(t.c[u], t.x[XLDS ? 0 : u], 4, acc);
    }
  }
  // Blocks [a, b) of the row's w4_blocks(K); the last one may be a part.  Batches of U blocks, the next
  // batch's loads issued before the current one's products; blocks past the last whole one repeat it and
  // are not used.
  // ready() is called once, when the first codes have been requested: what it does to the tokens' place in LDS
  // costs no time of its own.
  template <class Ready>
  __device__ __forceinline__ void run(int a, int b, f32x4 (&acc)[RT][NG], Ready ready) const {
    const int whole = min(b, K / W4_BLOCK);
    if (a >= whole) ready();
    if (a < whole) {
      Batch t0, t1;
      load(t0, a, whole - 1);
      ready();
      int st = a;
      for (; st + 2 * U < whole; st += 2 * U) {  // steady state: both batches whole
        load(t1, st + U, whole - 1);
        mma(t0, st, U, acc);
        load(t0, st + 2 * U, whole - 1);
        mma(t1, st + U, U, acc);
      }
      if (st + U < whole) {
        load(t1, st + U, whole - 1);
        mma(t0, st, U, acc);
        mma(t1, st + U, whole - st - U, acc);
      } else {
        mma(t0, st, whole - st, acc);
      }
    }
    if (b > whole && a < b) tail(b - 1, acc);
    if constexpr (INT) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int g = 0; g < NG; ++g) acc[r][g] *= W4_INT_UNIT;
    }
  }
  __device__ __forceinline__ void run(int a, int b, f32x4 (&acc)[RT][NG]) const { run(a, b, acc, [] {}); }
  // the part of a last block: K - 128 blk = 32, 64 or 96 elements
  __device__ __forceinline__ void tail(int blk, f32x4 (&acc)[RT][NG]) const {
    const int left = K - blk * W4_BLOCK;
    Codes c;
    u32x4 v[NG][4];
    load_codes(c, blk, left);
    load_x(v, blk, left);
    mma(c, v, left / 32, acc);
  }
};

// Copies elements [k0, k1) (multiples of 32) of a token to LDS, for the calling wave's own use.  The first 64 x 8 R
// elements pass through registers, so that other loads can be issued between request() and write().
template <int R>
struct W4Stage {
  u32x4 v[R];
  const bf16* x;
  bf16* lds;
  int k0, k1;
  __device__ __forceinline__ void request(const bf16* x_, bf16* lds_, int a, int b) {
    x = x_;
    lds = lds_;
    k0 = a + (threadIdx.x & 63) * 8;
    k1 = b;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (k0 + 512 * i < k1) v[i] = ld16(x + k0 + 512 * i);
  }
  __device__ __forceinline__ void write() const {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (k0 + 512 * i < k1) st16(lds + k0 + 512 * i, v[i]);
    for (int k = k0 + 512 * R; k < k1; k += 512) st16(lds + k, ld16(x + k));
    w4_lds_order();
  }
};

// A wave's results of one tile and token group to LDS as [token][16 rows] floats: 16 tokens, or 4 with NI = 1.
template <int NI> constexpr int w4_tokens() { return NI == 1 ? 4 : 16; }
template <int NI>
__device__ __forceinline__ void w4_put(float* p, f32x4 v) {
  const int r16 = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int i = 0; i < NI; ++i) p[(NI * q + i) * 16 + r16] = v[i];
}
// With NI = 1, a lane's token: of A's 16 rows every fourth counts.
__device__ __forceinline__ int w4_token() { return (threadIdx.x & 15) >> 2; }

}  // namespace moe
