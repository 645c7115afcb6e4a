// 4-bit weights with group scales (w4.h has the formats): quantisation, expansion, and the dense
// projection on them, out = residual + act(X W^T + bias) with bf16 X.
//
// Few rows: the codes are streamed from memory straight into registers (k_w4_rows).  Some hundred: tiles with X in
// LDS (k_w4_tile).  More: W expanded to bf16 in the workspace, then the dense projection's own tiles.
#include "gemm_core.h"
#include "internal.h"
#include "lin_epi.h"
#include "w4.h"

namespace moe {

// ---- quantisation ----
// Bound by memory: 16384 x 7168 bf16 80 to 89 us (3.3 to 3.7 TB/s), fp32 119 to 138 (3.9 to 4.5).
// One wave per row, one lane per 32 elements; a group's lanes (1, 2 or 4 neighbours) share its maximum.
template <typename T, int FMT>
__global__ __launch_bounds__(256) void k_quant_w4(const T* __restrict__ src, int64_t rows, int K, int group,
                                                  uint8_t* __restrict__ codes, void* __restrict__ scales) {
  constexpr int VEC = Vec<T>::N;
  const int lane = threadIdx.x & 63, nb = K / 32;
  for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < rows; row += (int64_t)gridDim.x * 4) {
    for (int b = lane; b < nb; b += 64) {
      const T* p = src + row * K + b * 32;
      float f[32];
#pragma unroll
      for (int c = 0; c < 32; c += VEC) unpack16<T>(ld16(p + c), f + c);
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(f[i]));
      uint32_t w[4] = {0, 0, 0, 0};
      if constexpr (FMT == W4_INT) {
        if (group >= 64) top = fmaxf(top, __shfl_xor(top, 1, WAVE));
        if (group >= 128) top = fmaxf(top, __shfl_xor(top, 2, WAVE));
        bf16 s = (bf16)(top / 7.0f);
        if ((float)s == 0.0f) s = (bf16)1.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float c = fminf(fmaxf(rintf(f[i] / (float)s), -7.0f), 7.0f);
          w[i >> 3] |= (uint32_t)((int)c + 8) << (4 * (i & 7));
        }
        if (b * 32 % group == 0) static_cast<bf16*>(scales)[(int64_t)(b * 32 / group) * rows + row] = s;
      } else {
        // the smallest power of two 2^k with top / 2^k <= 6 = 0.75 2^3
        int ex = 0;
        const float m = frexpf(top, &ex);
        const int k = top == 0.0f ? 0 : min(max(ex - 3 + (m > 0.75f ? 1 : 0), -127), 127);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float a = ldexpf(fabsf(f[i]), -k);
          // the nearest of 0 0.5 1 1.5 2 3 4 6, ties to the even code
          const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
          w[i >> 3] |= (c | (f[i] < 0.0f ? 8u : 0u)) << (4 * (i & 7));
        }
        static_cast<uint8_t*>(scales)[((int64_t)(b >> 2) * rows + row) * 4 + (b & 3)] = (uint8_t)(k + 127);
      }
      st16(codes + row * (K / 2) + b * 16, u32x4{w[0], w[1], w[2], w[3]});
    }
  }
}

// ---- expansion: a thread takes 8 codes of a word, so that a wave writes whole lines ----
// 16384 x 7168 to bf16 63 us with groups of 128 (4.7 TB/s), 82 to 89 with 32, whose scales lie in planes of their own.
template <typename T, int FMT>
__global__ __launch_bounds__(256) void k_expand_w4(const uint8_t* __restrict__ codes, const void* __restrict__ scales, int64_t rows,
                                                   int K, int group, T* __restrict__ out) {
  const int words = K / 8;  // of a row
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= words) return;
    const uint32_t w = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(codes + row * (K / 2)) + i);
    float f[8];
    if constexpr (FMT == W4_INT) {
      const float s = (float)static_cast<const bf16*>(scales)[(int64_t)(i * 8 / group) * rows + row];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = (float)((int)(w >> (4 * k) & 15) - 8) * s;
    } else {
      const int e = static_cast<const uint8_t*>(scales)[((int64_t)(i >> 4) * rows + row) * 4 + ((i >> 2) & 3)];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // twice the magnitude: 0 1 2 3 4 6 8 12
        const int c = (int)(w >> (4 * k)) & 15, m = c & 7, t = m < 4 ? m : (2 + (m & 1)) << ((m >> 1) - 1);
        f[k] = ldexpf((float)(c & 8 ? -t : t), e - 128);
      }
    }
#pragma unroll
    for (int u = 0; u < 8; u += Vec<T>::N) st16(out + row * K + i * 8 + u, pack16<T>(f + u));
  }
}

// ---- a few rows ----
enum { W4_OUT = 0, W4_GLU = 1, W4_PART = 2 };  // the epilogue; SwiGLU's; partial products of a slice

// One workgroup per 16 RT rows of W (SwiGLU: 8 RT columns, their gate rows in the first half of the tiles, the
// up rows in the second; with RT = 1 in the halves of one tile), NG groups of tokens and one slice of the
// reduction, which its waves share: blocks of 128 elements in contiguous runs.  The waves' results meet in LDS,
// [wave][RT][NG][token][16], are added in wave order, and the epilogue runs on four columns of a token a thread.
//
// Up to 4 tokens (NI = 1) each wave copies its run of X to LDS, so that the memory path carries little but
// codes.  With more, X (16 tokens of a block: 4 KB for a tile's 1 KB of
// codes) comes from L2 by whole lines, which bounds the kernel unless a wave takes several tiles of rows with each
// block of X: 13 x 14336 -> 4096 int4 took 17.3 us with RT = 1 and the whole reduction in a workgroup where RT = 4 and
// four slices took 11.2 (12 since a code goes in as two digits; joining the slices adds about 2).  What bounds it then is how short the work is: each wave has
// 3 or 4 blocks, so asking for the first (about 2 us) and the waves' sums are half of its time; two blocks more under way
// gave nothing.
//   One token: the codes alone.  7168 -> 2048 SwiGLU fp4 (15.6 MB) 6.6 us a call, 2.4 TB/s, 14336 columns (62 MB) 16.1,
// 3.9 TB/s: launch, first load and sums are some 3 us of either.
template <int FMT, int G, int NG, int RT, int NI, int XMODE, int U, int OUT>
__global__ __launch_bounds__(512) void k_w4_rows(const bf16* __restrict__ X, int64_t ldx, const uint8_t* __restrict__ codes,
                                                 const uint8_t* __restrict__ scales, int64_t plane, int m, int n, int K,
                                                 float* __restrict__ part, LinEpi<bf16> ep) {
  extern __shared__ __attribute__((aligned(16))) char w4_lds[];
  typedef W4Stream<FMT, G, NG, RT, NI, XMODE, U> Stream;
  constexpr bool XLDS = XMODE == W4_XLDS;
  constexpr int TOK = w4_tokens<NI>();
  constexpr bool GLU = OUT == W4_GLU;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W_ = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const int c0 = blockIdx.x * (GLU ? 8 : 16) * RT, t0 = blockIdx.y * TOK * NG;
  Stream ws;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    int row;  // (rows behind the last read it, unused)
    if constexpr (!GLU) row = min(c0 + 16 * r + r16, n - 1);
    else if constexpr (RT == 1) row = r16 < 8 ? c0 + r16 : n + c0 + r16 - 8;
    else row = (r < RT / 2 ? 0 : n) + min(c0 + 16 * (r % (RT / 2)) + r16, n - 1);
    ws.w[r] = codes + (int64_t)row * (K / 2) + 16 * q;
    ws.s[r] = scales + (FMT == W4_INT ? (int64_t)row * 2 : (int64_t)row * 4 + q);
  }
  ws.plane = plane;
  ws.K = K;
  const int nb = w4_blocks(K);
  const int z0 = (int)((int64_t)nb * blockIdx.z / gridDim.z), z1 = (int)((int64_t)nb * (blockIdx.z + 1) / gridDim.z);
  const int a = z0 + (z1 - z0) * wave / W_, b = z0 + (z1 - z0) * (wave + 1) / W_;
  bf16* xl = reinterpret_cast<bf16*>(w4_lds);
  const int xp = K + 8;  // LDS pitch of a token
  if constexpr (XLDS) {
    ws.x[0] = xl + min(w4_token(), m - 1) * xp + Stream::XQ * q;
  } else {
    ws.xb = reinterpret_cast<const char*>(X + (int64_t)t0 * ldx);
    ws.xs = w4_lds + wave * (NG * W4_XSLOT);
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i)  // (below 2^29)
        ws.xo[g][i] = (uint32_t)min(16 * g + 4 * i + q, m - 1 - t0) * (uint32_t)(ldx * 2) + 16 * r16;
  }
  W4Stage<2> first;
  if constexpr (XLDS) first.request(X, xl, a * W4_BLOCK, min(b * W4_BLOCK, K));
  f32x4 acc[RT][NG];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[r][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (a < b)
    ws.run(a, b, acc, [&] {
      if constexpr (XLDS) {
        first.write();
        for (int t = 1; t < m; ++t) {
          W4Stage<1> s;
          s.request(X + t * ldx, xl + t * xp, a * W4_BLOCK, min(b * W4_BLOCK, K));
          s.write();
        }
      }
    });
  // (the results take the tokens' place: with RT = 4 the wave's own)
  if constexpr (XLDS || RT < 4) __syncthreads();
  else w4_lds_order();
  float* res = reinterpret_cast<float*>(w4_lds);
  constexpr int TILE = TOK * 16;
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int g = 0; g < NG; ++g) w4_put<NI>(res + ((wave * RT + r) * NG + g) * TILE, acc[r][g]);
  __syncthreads();
  auto total = [&](int r, int g, int at) {
    const float* p = res + (r * NG + g) * TILE + at;
    f32x4 v = *reinterpret_cast<const f32x4*>(p);
    for (int w = 1; w < W_; ++w) v += *reinterpret_cast<const f32x4*>(p + w * RT * NG * TILE);
    return v;
  };
  constexpr int QUADS = GLU ? 2 * RT : 4 * RT;  // of a token's columns
  for (int it = threadIdx.x; it < NG * TOK * QUADS; it += blockDim.x) {
    const int quad = it % QUADS, tok = it / QUADS % TOK, g = it / QUADS / TOK;
    const int c = c0 + 4 * quad, t = t0 + g * TOK + tok;
    if (t >= m || c >= n) continue;
    const int r = quad >> 2, at = tok * 16 + 4 * (quad & 3);
    const f32x4 z = total(r, g, at);
    if constexpr (GLU) {
      const f32x4 up = RT == 1 ? total(0, g, at + 8) : total(r + RT / 2, g, at);
      lin_epi4(ep, (int64_t)t, c, n, true, z, up);
    } else if constexpr (OUT == W4_OUT) {
      lin_epi4(ep, (int64_t)t, c, n, false, z, z);
    } else {
      *reinterpret_cast<f32x4*>(part + ((int64_t)blockIdx.z * m + t) * n + c) = z;
    }
  }
}

// ---- some hundred rows ----
// X through LDS, W straight from its codes: a workgroup of four waves takes 128 tokens and 64 RT rows of W.  Blocks
// of 128 elements of the tokens (32 KB) arrive in two slots of LDS in turn by direct loads; each wave expands the codes
// of its own 16 RT rows into the products' B operand, where no other wave needs them, so that W never passes through
// LDS or memory as bf16.  INT4 values are rounded to bf16 here (half a step, 2^-9 of them; s (c - 8) itself is exact in
// fp32): eight token groups per tile leave no time for a scale per group and result.
//   X in LDS: [128 tokens][256 bytes], 16-byte chunk c of token t in slot c ^ (t & 15): the 16 tokens that are
// read together lie in different banks.  Each slot is an array of its own, so that the compiler sees that reading
// one does not wait for the loads into the other.
//   Bound by LDS: every wave reads the whole block of X, 32 KB against 64 MFMAs of 16 cycles (RT = 2).  Two
// workgroups a CU hide each other's waits: eight waves on a ring of four slots, one workgroup a CU, took 26 us where
// this takes 19 (256 x 2048 -> 7168).  777 x 2048 -> 7168 int4/32 40 us (570 TFLOP/s), int4/128 38, fp4 33.
constexpr int W4G_TOK = 128, W4G_NG = W4G_TOK / 16, W4G_WAVES = 4, W4G_SLOT = W4G_TOK * 256;
constexpr int W4G_DMA = W4G_SLOT / 1024 / W4G_WAVES;  // direct loads of a wave per block

template <int FMT>
__device__ __forceinline__ u32x4 w4_expand8(uint32_t w, float s, float s8) {
  if constexpr (FMT == W4_FP) {
    (void)s8;
    return w4_unpack_fp(w, s);
  } else {
    const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;  // elements 0 2 4 6 and 1 3 5 7
    u32x4 r;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      r[k] = pack_bf16x2(fmaf((float)((lo >> (8 * k)) & 255u), s, s8), fmaf((float)((hi >> (8 * k)) & 255u), s, s8));
    return r;
  }
}

template <int FMT, int RT, int OUT>
__global__ __launch_bounds__(W4G_WAVES * 64, 2) void k_w4_tile(const bf16* __restrict__ X, int64_t ldx,
                                                            const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                            int64_t plane, int group_shift, int m, int n, int K,
                                                            float* __restrict__ part, LinEpi<bf16> ep) {
  __shared__ __attribute__((aligned(1024))) char l0[W4G_SLOT], l1[W4G_SLOT];
  constexpr bool GLU = OUT == W4_GLU, INT = FMT == W4_INT;
  constexpr int COLS = GLU ? 8 * RT : 16 * RT;  // output columns of a wave
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane & 15, q = lane >> 4;
  const int c0 = (blockIdx.x * W4G_WAVES + wave) * COLS, t0 = blockIdx.y * W4G_TOK;
  const int nb = w4_blocks(K);
  const int b0 = (int)((int64_t)nb * blockIdx.z / gridDim.z), b1 = (int)((int64_t)nb * (blockIdx.z + 1) / gridDim.z);
  // the wave's rows of W (behind the last one: that one, unused): SwiGLU's tiles hold gate rows, then up rows
  const uint8_t *wp[RT], *sp[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int i = 16 * r + r16, col = GLU && i >= COLS ? i - COLS : i;
    const int64_t row = (GLU && i >= COLS ? n : 0) + min(c0 + col, n - 1);
    wp[r] = codes + row * (K / 2) + 16 * q;
    sp[r] = scales + (INT ? row * 2 : row * 4 + q);
  }
  // direct loads: instruction i of the wave fills tokens 16 i + 4 wave + 0 .. 3, lane l slot l % 16 of token l / 16
  const int tl = 4 * wave + (lane >> 4), chunk = (lane & 15) ^ (tl & 15);
  const char* xt = reinterpret_cast<const char*>(X + (int64_t)t0 * ldx);
  uint32_t xo[W4G_DMA];
#pragma unroll
  for (int i = 0; i < W4G_DMA; ++i) xo[i] = (uint32_t)min(16 * i + tl, m - 1 - t0) * (uint32_t)(ldx * 2);  // (below 2^31)
  u32x4 cw[2][RT];
  uint32_t cs[2][RT];
  auto fetch = [&](int b, char* slot, u32x4 (&c)[RT], uint32_t (&s)[RT]) {
    // (chunks behind the row repeat its last: they meet weights of zero)
    const uint32_t at = (uint32_t)b * 256u + 16u * (uint32_t)min(chunk, (K - b * W4_BLOCK) / 8 - 1);
#pragma unroll
    for (int i = 0; i < W4G_DMA; ++i) dma16(xt + xo[i] + at, slot + i * 4096 + wave * 1024);
    const bool in = b * W4_BLOCK + 32 * q < K;
    const int64_t pl = INT ? (b * W4_BLOCK + (in ? 32 * q : 0)) >> group_shift : b;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      c[r] = ld16(wp[r] + (int64_t)b * (W4_BLOCK / 2) - (in ? 0 : 16 * q));
      if constexpr (INT) s[r] = *reinterpret_cast<const uint16_t*>(sp[r] + pl * plane);
      else s[r] = sp[r][pl * plane];  // (a byte behind the row is not used)
    }
  };
  f32x4 acc[RT][W4G_NG];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int g = 0; g < W4G_NG; ++g) acc[r][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto products = [&](int b, const char* slot, const u32x4 (&c)[RT], const uint32_t (&s)[RT]) {
    const bool in = b * W4_BLOCK + 32 * q < K;
    const char* xb = slot + r16 * 256;
    float f[RT], f8[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      // (INT: a sixteenth of the scale, as 8 s may be beyond the range where 7 s is not; the end takes it back)
      if constexpr (INT) f[r] = in ? 0.0625f * __uint_as_float(s[r] << 16) : 0.0f;
      else f[r] = !in ? 1.0f : __uint_as_float(s[r] ? s[r] << 23 : 0x00400000u);
      f8[r] = -8.0f * f[r];
    }
    u32x4 x[2][W4G_NG];
    auto read = [&](int j) {
      const char* xj = xb + 16 * ((4 * q + j) ^ r16);
#pragma unroll
      for (int g = 0; g < W4G_NG; ++g) x[j & 1][g] = *reinterpret_cast<const u32x4*>(xj + g * 4096);
    };
    read(0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j < 3) read(j + 1);
      u32x4 w[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) w[r] = w4_expand8<FMT>(INT || in ? c[r][j] : 0u, f[r], f8[r]);
#pragma unroll
      for (int g = 0; g < W4G_NG; ++g)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r][g] = w4_mfma(x[j & 1][g], w[r], acc[r][g]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // block b from `slot`; the next one goes where the block before was (behind the last one: that one once more,
  // unread, so that the loop needs no case of its own)
  auto step = [&](int b, const char* slot, const u32x4 (&c)[RT], const uint32_t (&s)[RT], char* free, u32x4 (&cf)[RT], uint32_t (&sf)[RT]) {
    wait_vmcnt<0>();
    ring_barrier();
    fetch(min(b + 1, b1 - 1), free, cf, sf);
    products(b, slot, c, s);
  };
  if (b0 < b1) {
    fetch(b0, l0, cw[0], cs[0]);
    int b = b0;
    for (; b + 2 <= b1; b += 2) {
      step(b, l0, cw[0], cs[0], l1, cw[1], cs[1]);
      step(b + 1, l1, cw[1], cs[1], l0, cw[0], cs[0]);
    }
    if (b < b1) step(b, l0, cw[0], cs[0], l1, cw[1], cs[1]);
  }
  wait_vmcnt<0>();  // the direct loads still under way end before the slots are used again
  __syncthreads();
  // 16 tokens at a time through the wave's own part of LDS: [token][16 RT values], a lane takes a quarter of a
  // token's columns
  constexpr int PITCH = 16 * RT + 4, QUADS = COLS / 4;
  float* res = reinterpret_cast<float*>(l0) + wave * (16 * PITCH);
  const int tok = lane >> 2;
#pragma unroll
  for (int g = 0; g < W4G_NG; ++g) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) res[(4 * q + i) * PITCH + 16 * r + r16] = acc[r][g][i] * (INT ? 16.0f : 1.0f);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    __builtin_amdgcn_wave_barrier();
    const int t = t0 + 16 * g + tok;
#pragma unroll
    for (int k = 0; k < (QUADS + 3) / 4; ++k) {
      const int at = 4 * ((lane & 3) + 4 * k), c = c0 + at;
      if (at < COLS && t < m && c < n) {
        const f32x4 z = *reinterpret_cast<const f32x4*>(res + tok * PITCH + at);
        if constexpr (GLU) {
          const f32x4 up = *reinterpret_cast<const f32x4*>(res + tok * PITCH + COLS + at);
          lin_epi4(ep, (int64_t)t, c, n, true, z, up);
        } else if constexpr (OUT == W4_OUT) {
          lin_epi4(ep, (int64_t)t, c, n, false, z, z);
        } else {
          *reinterpret_cast<f32x4*>(part + ((int64_t)blockIdx.z * m + t) * n + c) = z;
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    __builtin_amdgcn_wave_barrier();
  }
}

constexpr int64_t W4_LDS = 65536;

// How a product is cut: by the shape alone, so that the workspace is known without the weights.
struct W4Plan {
  bool lds;         // up to 4 tokens, which lie in LDS
  int ng, rt;       // token groups of 16 and row tiles of a workgroup
  int slices, waves;
  double us;        // more than 16 rows: the model's time
};
static int w4_waves(int blocks) {  // of a workgroup: at least two blocks each
  int waves = 8;
  while (waves > 1 && blocks / waves < 2) waves /= 2;
  return waves;
}
static W4Plan w4_plan(const LinShape& s) {
  const bool glu = s.act == LIN_SWIGLU;
  const int64_t rows = glu ? 2 * s.N : s.N;
  const int blocks = w4_blocks((int)s.K);
  W4Plan p;
  p.lds = s.M <= 4 && s.M * (s.K + 8) * 2 <= W4_LDS;
  p.ng = s.M <= 16 ? 1 : 2;
  p.rt = 1;
  p.slices = 1;
  p.us = 0.0;
  if (p.lds) {
    // 8 waves where the grid would not fill the chip otherwise (2 x 2048 x 7168: 5.9 us, 6.6 with 4;
    // 2 x 14336 x 4096: 14.8, 14.0)
    const int64_t tiles = rows / 16;
    p.waves = 4;
    while (p.waves < 8 && tiles * p.waves < 2048) p.waves *= 2;
    while (p.waves > 1 && blocks / p.waves < 4) p.waves /= 2;
    return p;
  }
  const int64_t groups = cdiv(s.M, 16 * p.ng);
  if (p.ng == 1) {
    // X costs its bytes once per workgroup, at about 26 TB/s over all L2s; fewer, taller workgroups need slices to fill
    // the chip, and a second launch of about 2.5 us to join them
    const double x_us = 32.0 * s.K / 26e6;  // per row tile of a workgroup
    int best = 1;
    for (int rt : {4, 2}) {
      if (cdiv(rows, 16 * rt) >= 200) {
        best = rt;
        break;
      }
    }
    const double whole = x_us * cdiv(rows, 16 * best), sliced = x_us * cdiv(rows, 64) + 2.5;
    p.rt = best;
    if (best < 4 && sliced < whole) {
      p.rt = 4;
      while (p.slices < 8 && cdiv(rows, 64) * p.slices < 200 && blocks / (2 * p.slices) >= 8) p.slices *= 2;
      if (p.slices == 1) p.rt = best;
    }
    p.waves = w4_waves(blocks / p.slices);
    return p;
  }
  // 32 tokens a workgroup: by a model of measured times.  A round of 256 workgroups of eight waves, b blocks of 128 a
  // wave, takes 3 + 2 b us with four row tiles and 2.4 + 1.15 b with two; with one, where two workgroups share a
  // CU, each round adds 1.5 + 0.68 b to 2 + 0.42 b (96 x 7168 -> 2048 SwiGLU fp4 17.1, 21.8 and 22.7 us, 64 rows 16.8, 12.3
  // and 16.7, 32 rows 16.4, 12.0 and 10.6).
  for (int rt : {4, 2, 1})
    for (int slices = 1; slices <= (rt == 4 ? 8 : 1) && (slices == 1 || blocks / slices >= 16); slices *= 2) {
      const int waves = w4_waves(blocks / slices);
      const double b = (double)blocks / slices / 8.0;
      const double rounds = (double)cdiv(cdiv(rows, 16 * rt) * groups * slices * waves, 8 * 256);
      double us = rt == 4   ? 2.5 + rounds * (3.0 + 2.0 * b)
                  : rt == 2 ? 2.0 + rounds * (2.4 + 1.15 * b)
                            : 2.0 + 0.42 * b + rounds * (1.5 + 0.68 * b);
      if (slices > 1) us += 3.0 + (double)slices * (double)s.M * (double)rows * 8.0 / 4e6;  // joining them
      if (p.us == 0.0 || us < p.us) {
        p.us = us;
        p.rt = rt;
        p.slices = slices;
        p.waves = waves;
      }
    }
  return p;
}

struct W4TilePlan {
  int rt, slices;
  double us;
};
// Row tiles per wave and slices by a model of measured times: a block of the loop takes 1 us (RT = 2: 1.45) with one
// workgroup a CU and 1.7 (2.3) with two; joining slices takes 1.5 us and their bytes at 6 TB/s.
static W4TilePlan w4_tile_plan(const LinShape& s) {
  const int64_t rows = s.act == LIN_SWIGLU ? 2 * s.N : s.N, groups = cdiv(s.M, W4G_TOK), blocks = w4_blocks((int)s.K);
  W4TilePlan best{1, 1, 0.0};
  for (int rt = 1; rt <= 2; ++rt)
    for (int slices = 1; slices <= 4 && (slices == 1 || blocks / slices >= 2); slices *= 2) {
      const int64_t wgs = cdiv(rows, 16 * W4G_WAVES * rt) * groups * slices, rest = wgs % 512;
      const double one = rt == 1 ? 1.0 : 1.45, two = rt == 1 ? 1.7 : 2.3;
      double us = (double)cdiv(blocks, slices) * ((double)(wgs / 512) * two + (rest == 0 ? 0.0 : rest <= 256 ? one : two));
      us += 1.5;  // the launch and the first block
      if (slices > 1) us += 1.5 + (double)slices * (double)s.M * (double)rows * 8.0 / 6e6;
      if (best.us == 0.0 || us < best.us) best = W4TilePlan{rt, slices, us};
    }
  return best;
}

// Which way a product goes.  Up to 64 rows the codes are streamed; up to 1024 the quicker of streaming and tiles by the
// models above (256 x 1024 -> 1024 4.9 us, tiles 9.2; 256 x 2048 -> 7168 30 and 18); beyond, W is expanded (2048 x
// 2048 -> 7168 63 us, tiles 70; 1024 rows 45 and 38).
constexpr int W4_STREAM_ROWS = 64, W4_TILE_ROWS = 1024;
int linear_w4_plan(const LinShape& s) {
  if (s.M <= W4_STREAM_ROWS) return W4_STREAMED;
  if (s.M > W4_TILE_ROWS) return W4_EXPANDED;
  return w4_plan(s).us < w4_tile_plan(s).us ? W4_STREAMED : W4_TILED;
}
W4Cut linear_w4_cut(const LinShape& s) {
  const int way = linear_w4_plan(s);
  if (way == W4_EXPANDED || s.M == 0) return W4Cut{0, 0, 0};
  if (way == W4_TILED) {
    const W4TilePlan t = w4_tile_plan(s);
    return W4Cut{t.rt, W4G_NG, t.slices};
  }
  const W4Plan p = w4_plan(s);
  return W4Cut{p.rt, p.lds ? 0 : p.ng, p.slices};
}
template <int FMT, int RT>
static void w4_tile_rt(const LinShape& s, const W4TilePlan& p, const W4View& w, const bf16* X, const LinEpi<bf16>& ep, float* part,
                       hipStream_t st) {
  const bool glu = s.act == LIN_SWIGLU;
  const int64_t rows = glu ? 2 * s.N : s.N;
  const dim3 grid((unsigned)cdiv(rows, 16 * W4G_WAVES * RT), (unsigned)cdiv(s.M, W4G_TOK), (unsigned)p.slices);
  const uint8_t* sc = static_cast<const uint8_t*>(w.scales);
  const int64_t plane = rows * (FMT == W4_INT ? 2 : 4);
  const int m = (int)s.M, K = (int)s.K, shift = w.group == 32 ? 5 : w.group == 64 ? 6 : 7, T = W4G_WAVES * 64;
  if (p.slices > 1) k_w4_tile<FMT, RT, W4_PART><<<grid, T, 0, st>>>(X, s.ldx, w.codes, sc, plane, shift, m, (int)rows, K, part, ep);
  else if (glu) k_w4_tile<FMT, RT, W4_GLU><<<grid, T, 0, st>>>(X, s.ldx, w.codes, sc, plane, shift, m, (int)s.N, K, part, ep);
  else k_w4_tile<FMT, RT, W4_OUT><<<grid, T, 0, st>>>(X, s.ldx, w.codes, sc, plane, shift, m, (int)s.N, K, part, ep);
}
template <int FMT>
static hipError_t w4_tile(const LinShape& s, const W4View& w, const bf16* X, const LinEpi<bf16>& ep, float* part, hipStream_t st) {
  const W4TilePlan p = w4_tile_plan(s);
  if (p.rt == 2) w4_tile_rt<FMT, 2>(s, p, w, X, ep, part, st);
  else w4_tile_rt<FMT, 1>(s, p, w, X, ep, part, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.slices == 1) return e;
  return launch_lin_finish(part, p.slices, (int)s.M, (int)s.N, (int)(s.act == LIN_SWIGLU ? 2 * s.N : s.N), ep, st);
}

template <int FMT, int G, int NG, int RT, int NI, int XMODE, int U>
static void w4_rows(const LinShape& s, const W4Plan& p, const W4View& w, const bf16* X, const LinEpi<bf16>& ep, float* part,
                    hipStream_t st) {
  const bool glu = s.act == LIN_SWIGLU;
  const int64_t rows = glu ? 2 * s.N : s.N;
  constexpr int TOK = w4_tokens<NI>();
  size_t lds = (size_t)p.waves * RT * NG * TOK * 16 * sizeof(float);
  const size_t xl = XMODE == W4_XLDS ? (size_t)s.M * (s.K + 8) * sizeof(bf16) : (size_t)p.waves * NG * W4_XSLOT;
  if (xl > lds) lds = xl;
  const dim3 grid((unsigned)cdiv(rows, 16 * RT), (unsigned)cdiv(s.M, TOK * NG), (unsigned)p.slices);
  const uint8_t* sc = static_cast<const uint8_t*>(w.scales);
  const int64_t plane = rows * (FMT == W4_INT ? 2 : 4);
  const int m = (int)s.M, K = (int)s.K, threads = p.waves * 64;
  if (p.slices > 1) {
    if constexpr (RT == 4)
      k_w4_rows<FMT, G, NG, RT, NI, XMODE, U, W4_PART><<<grid, threads, lds, st>>>(X, s.ldx, w.codes, sc, plane, m, (int)rows, K, part, ep);
  } else if (glu) {
    k_w4_rows<FMT, G, NG, RT, NI, XMODE, U, W4_GLU><<<grid, threads, lds, st>>>(X, s.ldx, w.codes, sc, plane, m, (int)s.N, K, part, ep);
  } else {
    k_w4_rows<FMT, G, NG, RT, NI, XMODE, U, W4_OUT><<<grid, threads, lds, st>>>(X, s.ldx, w.codes, sc, plane, m, (int)s.N, K, part, ep);
  }
}
template <int FMT, int G, int NG>
static void w4_rows_rt(const LinShape& s, const W4Plan& p, const W4View& w, const bf16* X, const LinEpi<bf16>& ep, float* part,
                       hipStream_t st) {
  if (p.rt == 4) w4_rows<FMT, G, NG, 4, 4, W4_XLINE, 1>(s, p, w, X, ep, part, st);
  else if (p.rt == 2) w4_rows<FMT, G, NG, 2, 4, W4_XLINE, 1>(s, p, w, X, ep, part, st);
  else w4_rows<FMT, G, NG, 1, 4, W4_XLINE, 1>(s, p, w, X, ep, part, st);
}
template <int FMT, int G>
static hipError_t w4_stream(const LinShape& s, const W4View& w, const bf16* X, const LinEpi<bf16>& ep, float* part, hipStream_t st) {
  const W4Plan p = w4_plan(s);
  // (small groups leave no registers for two blocks a batch)
  if (p.lds) w4_rows<FMT, G, 1, 1, 1, W4_XLDS, FMT == W4_INT && G < 128 ? 1 : 2>(s, p, w, X, ep, part, st);
  else if (p.ng == 1) w4_rows_rt<FMT, G, 1>(s, p, w, X, ep, part, st);
  else w4_rows_rt<FMT, G, 2>(s, p, w, X, ep, part, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.slices == 1) return e;
  return launch_lin_finish(part, p.slices, (int)s.M, (int)s.N, (int)(s.act == LIN_SWIGLU ? 2 * s.N : s.N), ep, st);
}

static size_t w4_expanded_bytes(const LinShape& s) {
  return align_up((size_t)(s.act == LIN_SWIGLU ? 2 * s.N : s.N) * s.K * sizeof(bf16), 256);
}
size_t linear_w4_workspace_bytes(const LinShape& s) {
  const int way = linear_w4_plan(s);
  if (way == W4_EXPANDED) return w4_expanded_bytes(s) + linear_fwd_workspace_bytes(s);
  const int slices = way == W4_TILED ? w4_tile_plan(s).slices : s.M > 0 ? w4_plan(s).slices : 1;
  return slices > 1 ? (size_t)slices * s.M * (s.act == LIN_SWIGLU ? 2 * s.N : s.N) * sizeof(float) : 0;
}

hipError_t launch_quant_w4(const void* src, bool is_bf16, int format, int group, int64_t rows, int64_t K, uint8_t* codes,
                           void* scales, hipStream_t st) {
  if (rows <= 0) return hipSuccess;
  const int grid = (int)(cdiv(rows, 4) < (1 << 20) ? cdiv(rows, 4) : 1 << 20);
  const int k = (int)K;
  if (is_bf16) {
    const bf16* p = static_cast<const bf16*>(src);
    if (format == W4_INT) k_quant_w4<bf16, W4_INT><<<grid, 256, 0, st>>>(p, rows, k, group, codes, scales);
    else k_quant_w4<bf16, W4_FP><<<grid, 256, 0, st>>>(p, rows, k, group, codes, scales);
  } else {
    const float* p = static_cast<const float*>(src);
    if (format == W4_INT) k_quant_w4<float, W4_INT><<<grid, 256, 0, st>>>(p, rows, k, group, codes, scales);
    else k_quant_w4<float, W4_FP><<<grid, 256, 0, st>>>(p, rows, k, group, codes, scales);
  }
  return hipGetLastError();
}

hipError_t launch_expand_w4(const W4View& w, int64_t rows, int64_t K, bool is_bf16, void* out, hipStream_t st) {
  if (rows <= 0) return hipSuccess;
  const dim3 grid((unsigned)cdiv(K / 8, 256), (unsigned)(rows < 32768 ? rows : 32768));
  const int k = (int)K;
  if (is_bf16) {
    bf16* o = static_cast<bf16*>(out);
    if (w.format == W4_INT) k_expand_w4<bf16, W4_INT><<<grid, 256, 0, st>>>(w.codes, w.scales, rows, k, w.group, o);
    else k_expand_w4<bf16, W4_FP><<<grid, 256, 0, st>>>(w.codes, w.scales, rows, k, w.group, o);
  } else {
    float* o = static_cast<float*>(out);
    if (w.format == W4_INT) k_expand_w4<float, W4_INT><<<grid, 256, 0, st>>>(w.codes, w.scales, rows, k, w.group, o);
    else k_expand_w4<float, W4_FP><<<grid, 256, 0, st>>>(w.codes, w.scales, rows, k, w.group, o);
  }
  return hipGetLastError();
}

hipError_t launch_linear_w4(const LinShape& s, const void* X, const W4View& w, const float* bias, const void* residual, void* out,
                            void* ws, hipStream_t st) {
  if (s.M == 0) return hipSuccess;
  const int way = linear_w4_plan(s);
  if (way == W4_EXPANDED) {
    const hipError_t e = launch_expand_w4(w, s.act == LIN_SWIGLU ? 2 * s.N : s.N, s.K, true, ws, st);
    if (e != hipSuccess) return e;
    return launch_linear(s, X, ws, bias, residual, nullptr, out, static_cast<char*>(ws) + w4_expanded_bytes(s), st);
  }
  const LinEpi<bf16> ep{bias, static_cast<const bf16*>(residual), s.ldr, nullptr, 0, static_cast<bf16*>(out), s.ldy, s.act};
  const bf16* x = static_cast<const bf16*>(X);
  float* part = static_cast<float*>(ws);
  if (way == W4_TILED) return w.format == W4_FP ? w4_tile<W4_FP>(s, w, x, ep, part, st) : w4_tile<W4_INT>(s, w, x, ep, part, st);
  if (w.format == W4_FP) return w4_stream<W4_FP, 32>(s, w, x, ep, part, st);
  if (w.group == 32) return w4_stream<W4_INT, 32>(s, w, x, ep, part, st);
  if (w.group == 64) return w4_stream<W4_INT, 64>(s, w, x, ep, part, st);
  return w4_stream<W4_INT, 128>(s, w, x, ep, part, st);
}

}  // namespace moe
