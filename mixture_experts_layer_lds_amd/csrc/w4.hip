// 4-bit weights with group scales (w4.h has the formats): quantisation, expansion, and the dense
// projection on them, out = residual + act(X W^T + bias) with bf16 X.
//
// A few rows: one workgroup per 16 RT rows of W, its waves sharing the reduction, the codes streamed from
// memory straight into registers (k_w4_skinny); the waves' partial tiles meet in LDS and the epilogue runs in
// the same launch.  More rows: W expanded to bf16 in the workspace, then the dense projection's own tiles.
#include "internal.h"
#include "lin_epi.h"
#include "w4.h"

namespace moe {

// ---- quantisation ----
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

// ---- expansion: a thread takes 32 codes ----
template <typename T, int FMT>
__global__ __launch_bounds__(256) void k_expand_w4(const uint8_t* __restrict__ codes, const void* __restrict__ scales, int64_t rows,
                                                   int K, int group, T* __restrict__ out) {
  const int nb = K / 32;
  const int64_t items = rows * nb;
  for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (int64_t)gridDim.x * 256) {
    const int64_t row = it / nb;
    const int b = (int)(it - row * nb);
    const u32x4 w = ld16_nt(codes + row * (K / 2) + b * 16);
    float s = 0.0f;
    int e = 0;
    if constexpr (FMT == W4_INT) s = (float)static_cast<const bf16*>(scales)[(int64_t)(b * 32 / group) * rows + row];
    else e = static_cast<const uint8_t*>(scales)[((int64_t)(b >> 2) * rows + row) * 4 + (b & 3)];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (int)(w[j] >> (4 * i)) & 15;
        if constexpr (FMT == W4_INT) {
          f[i] = (float)(c - 8) * s;
        } else {
          // twice the magnitude: 0 1 2 3 4 6 8 12
          const int m = c & 7, t = m < 4 ? m : (2 + (m & 1)) << ((m >> 1) - 1);
          f[i] = ldexpf((float)(c & 8 ? -t : t), e - 128);
        }
      }
#pragma unroll
      for (int u = 0; u < 8; u += Vec<T>::N) st16(out + row * K + b * 32 + j * 8 + u, pack16<T>(f + u));
    }
  }
}

// ---- a few rows ----
// Dynamic LDS: [wave][RT][NG][64] partial tiles.
template <int FMT, int G, int NG, int RT, bool GLU>
__global__ __launch_bounds__(512) void k_w4_skinny(const bf16* __restrict__ X, int64_t ldx, const uint8_t* __restrict__ codes,
                                                   const uint8_t* __restrict__ scales, int64_t plane, int m, int n, int K,
                                                   LinEpi<bf16> ep) {
  extern __shared__ f32x4 sk_part[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W_ = blockDim.x >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  constexpr int TC = GLU ? 8 * RT : 16 * RT;  // output columns per tile
  constexpr bool INT = FMT == W4_INT;
  const int c0 = blockIdx.x * TC, t0 = blockIdx.y * 16 * NG;
  W4Stream<FMT, G, NG, RT, NG == 1 && RT == 1 ? 2 : 1> ws;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    // row i of the tile: (rows behind the last read valid ones, unused)
    auto row = [&](int i, int rows) {
      if constexpr (!GLU) return min(c0 + 16 * r + i, n - rows);
      else if constexpr (RT == 1) return i < 8 ? c0 + i : n + c0 + i - 8;
      else return r * n + min(c0 + i, n - rows);
    };
    ws.w[r] = codes + (int64_t)row(r16, 1) * (K / 2) + 16 * q;
    ws.s[r] = INT ? scales + (int64_t)row(4 * q, 4) * 2 : scales + (int64_t)row(r16, 1) * 4 + q;
  }
  ws.plane = plane;
  ws.K = K;
#pragma unroll
  for (int g = 0; g < NG; ++g) ws.x[g] = X + (int64_t)min(t0 + g * 16 + r16, m - 1) * ldx + (INT ? 8 : 32) * q;
  f32x4 acc[RT][NG];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[r][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int nb = w4_blocks(K), a = (int)((int64_t)nb * wave / W_), b = (int)((int64_t)nb * (wave + 1) / W_);
  if (a < b) ws.run(a, b, acc);
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[r][g] *= w4_factor<FMT>();
  lin_skinny_join<bf16, NG, RT, GLU>(acc, sk_part, ep, t0, m, n, c0);
}

// Rows up to which the codes are streamed; more go through an expanded copy of W.
constexpr int W4_STREAM_ROWS = 64;

template <int FMT, int G, int NG, int RT>
static void w4_skinny_rt(const LinShape& s, const W4View& w, const bf16* X, const LinEpi<bf16>& ep, hipStream_t st) {
  const bool glu = s.act == LIN_SWIGLU;
  const int64_t rows = glu ? 2 * s.N : s.N;
  const dim3 grid((unsigned)cdiv(s.N, (glu ? 8 : 16) * RT), (unsigned)cdiv(s.M, 16 * NG));
  const int blocks = w4_blocks((int)s.K);
  int waves = 1;
  while (waves < 8 && blocks / waves >= 4) waves *= 2;
  const size_t lds = (size_t)waves * RT * NG * 64 * sizeof(f32x4);
  const uint8_t* sc = static_cast<const uint8_t*>(w.scales);
  const int64_t plane = rows * (FMT == W4_INT ? 2 : 4);
  if (glu) k_w4_skinny<FMT, G, NG, RT, true><<<grid, waves * 64, lds, st>>>(X, s.ldx, w.codes, sc, plane, (int)s.M, (int)s.N, (int)s.K, ep);
  else k_w4_skinny<FMT, G, NG, RT, false><<<grid, waves * 64, lds, st>>>(X, s.ldx, w.codes, sc, plane, (int)s.M, (int)s.N, (int)s.K, ep);
}
template <int FMT, int G>
static void w4_skinny(const LinShape& s, const W4View& w, const bf16* X, const LinEpi<bf16>& ep, hipStream_t st) {
  if (s.M <= 16) w4_skinny_rt<FMT, G, 1, 1>(s, w, X, ep, st);
  else w4_skinny_rt<FMT, G, 2, 1>(s, w, X, ep, st);
}

static size_t w4_expanded_bytes(const LinShape& s) {
  return align_up((size_t)(s.act == LIN_SWIGLU ? 2 * s.N : s.N) * s.K * sizeof(bf16), 256);
}
size_t linear_w4_workspace_bytes(const LinShape& s) {
  return s.M <= W4_STREAM_ROWS ? 0 : w4_expanded_bytes(s) + linear_fwd_workspace_bytes(s);
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
  const int64_t need = cdiv(rows * (K / 32), 256);
  const int grid = (int)(need < (1 << 20) ? need : 1 << 20);
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
  if (s.M > W4_STREAM_ROWS) {
    const hipError_t e = launch_expand_w4(w, s.act == LIN_SWIGLU ? 2 * s.N : s.N, s.K, true, ws, st);
    if (e != hipSuccess) return e;
    return launch_linear(s, X, ws, bias, residual, nullptr, out, static_cast<char*>(ws) + w4_expanded_bytes(s), st);
  }
  const LinEpi<bf16> ep{bias, static_cast<const bf16*>(residual), s.ldr, nullptr, 0, static_cast<bf16*>(out), s.ldy, s.act};
  const bf16* x = static_cast<const bf16*>(X);
  if (w.format == W4_FP) w4_skinny<W4_FP, 32>(s, w, x, ep, st);
  else if (w.group == 32) w4_skinny<W4_INT, 32>(s, w, x, ep, st);
  else if (w.group == 64) w4_skinny<W4_INT, 64>(s, w, x, ep, st);
  else w4_skinny<W4_INT, 128>(s, w, x, ep, st);
  return hipGetLastError();
}

}  // namespace moe
